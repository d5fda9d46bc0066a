// chunk_weights.cu — the attention weights that a chunk of prompt queries gives to every key of an
// int8 paged K/V cache, summed over the queries and over the heads of each KV head.
//
// For query i (position history + i), head h of KV head kvh, key t <= history + i:
//   s[t] = softmax_scale log2(e) q . (k_code[t] k_scale[t]),  p = 2^(s[t] - M) / l,
//   acc[kvh][t] += sum over (i, h) of p.
// M and l belong to a row (i, h), the sum to a key, so the scores are needed twice; at 2048 queries x
// 24 heads x 32768 keys they would be 6.4 GB in fp32, which costs more to write and read back than the
// product Q K^T costs to do again.  Two passes over the same tiles, each a matrix product whose
// reduction runs along the accumulator's columns, so that it stays inside one thread:
//   row pass:    A = 128 query rows (held in tensor memory), B = key tiles streamed through shared
//                memory; thread = row, running maximum and sum over the columns (keys).
//   column pass: A = 128 keys (held in tensor memory), B = query-row tiles streamed; thread = key,
//                sum over the columns (rows) of 2^(s - M) / l.
// The rows of a KV head are r = i * G + g (G heads a group), so a row tile is a run of queries.
//
// Operands.  sm_103a has no integer tcgen05 kind, and the codes are exact in bf16 (|code| < 2^8), so both
// passes take the bf16 queries as they are and widen the codes to bf16: every product is exact and the
// sums are fp32.  A pass before them lays the queries out in the swizzled order of an operand tile, so
// that a tile is one bulk copy; when there are eight row tiles or more to read them, it does the same
// with the widened keys.  With fewer row tiles (WIDEN) that copy would be most of the call's traffic:
// then the pages come into a ring of their own as bytes, by bulk copies, and warps of the CTA widen them
// from there, into the B tile (row pass) or into tensor memory (column pass).
//
// Schedule.  One CTA per SM; the (A unit, B tile) pairs of all KV heads are one line, cut into equal
// runs, one per CTA, so that causal and ragged shapes balance to a tile.  An A unit is one 128-row tile
// (MT = 1) or two of them (MT = 2), which share every B tile: a 128 x 128 tile pair at head_dim 256
// takes 1024 cycles of the tensor core, in which one SM would have to take in 64 KB, more than all SMs
// together get out of L2; with two A tiles it is half of that.  With few row tiles the column pass keeps
// all of them in shared memory instead.  An A unit that two CTAs share leaves one partial each, and the
// partials are added in the order of the line: the same result every time.  Roles of a CTA's warps:
//   warps 0-15   softmax: thread = tensor-memory lane 32 (w % 4) + lane, two groups of eight warps with a
//                score tile each (the other group's is multiplied meanwhile), 64 of its columns a warp
//   warps 16-19  A loaders (128 threads): an A tile from shared memory to tensor memory; in the WIDEN column
//                pass, where they widen it, two groups (warps 16-23) take every second unit
//   WIDEN row pass: warps 20-27 B producers, thread = key, two groups with half of the dims each
//   the last warps: MMA issue, tile copies, page copies (WIDEN)
// Shared memory: a ring of tiles | WIDEN: a ring of pages.  A tiles take their turn before the first B tile of
// their unit in the ring of tiles, or (WIDEN row pass) as halves in the ring of pages; the WIDEN column
// pass's A tiles are the pages.  A wait on a barrier tells a phase only from the one before it, so every
// role that waits on a barrier visits all its phases in order: each ring is filled by one role, and A tiles
// that share a ring announce themselves on barriers of their own.
// Tensor memory: A tiles (head_dim / 2 columns each) | two score tiles, filled in turn.
//
// What bounds it.  Long chunks at head_dim 256: the tensor core (a 128 x 128 tile is 1024 cycles at 4096
// multiply-adds a cycle and SM, its 16384 exponentials 512 at 32 a cycle).  2048 queries after 30720 x 24 heads:
// 1100 us, the two products at 1.46 PFLOP/s, 76 % of what the library's bf16 product reaches; with a quarter of
// the multiplications 810 us, with a quarter of them and no exponentials 690 us.  Else the way of a score tile
// through tensor memory, registers and barriers, some 1500 cycles whatever the head_dim, and the five
// launches: a prompt of 2047 at head_dim 128 takes 77 us (row pass 35, column pass 32), 32 queries over 32768
// keys 54 us (20 and 22, of which 5 each are the pages out of memory).
// Measured both ways, us by row tiles of 128 after 16384 keys (head_dim 256, 4 KV heads | 128, 8 KV heads):
//   keys widened by every CTA | once:      4: 50 | 56, 6: 63 | 68, 8: 80 | 82, 12: 104 | 105, 16: 130 | 128, 32: 233 | 217
//                                          4: 60 | 63, 6: 82 | 81, 8: 101 | 96, 12: 140 | 126, 32: 344 | 287
//   (One rule from eight row tiles on: at head_dim 256 it costs 1 to 2 % up to 15.)
//   one A tile a unit | two (row pass):    2: 41 | 39, 4: 59 | 50, 6: 72 | 63 and 2: 47 | 41, 4: 74 | 60, 6: 100 | 82
#include <algorithm>

#include <cuda_bf16.h>

#include "kvq_dev.cuh"
#include "kvq_launch.h"
#include "tcgen05.cuh"
#include "tile_dev.cuh"

namespace kvq {

namespace {

constexpr int kSoftWarps = 16, kLoadWarp = 16, kProdWarp = 20;
constexpr int kParBufs = 4;    // column parameters, by B tile
// Column pass: key constants, by A unit.  The softmax warps can lag behind the A loaders by several units
// (of one B tile each), so the constants have more buffers than the A tiles, and barriers of their own,
// whose phases cannot pass the reader.
constexpr int kConstBufs = 8;
// Row pass: the reference that stands for a row's maximum is the largest score of the first chunk the row
// sees, and moves only when a chunk's sum of 2^(s - reference) reaches this: fp32 holds the sums as exactly
// whatever their exponent, and without a maximum to take a score costs one multiply-add, one
// exponential and one addition.
constexpr float kSumLimit = 1.8446744e19f;  // 2^64

// Parts that a run leaves of each A tile of its units: a tile's columns are halved between warps, and with one
// tile a unit its B tiles are halved between two groups of warps as well.
__host__ __device__ constexpr int parts_of_run(int a_tiles) { return a_tiles == 2 ? 2 : 4; }

template <int D, int PASS, int MT, bool WIDEN>
struct Cw {
  static constexpr bool kProduce = PASS == 1 && WIDEN;     // B tiles made by producer warps
  static constexpr bool kARing = !WIDEN;                   // A tiles come through the ring of tiles
  static constexpr int kLoadGroups = PASS == 2 && WIDEN ? 2 : 1;
  static constexpr int kMmaWarp = kProduce ? kProdWarp + 8 : kLoadWarp + 4 * kLoadGroups;
  static constexpr int kPageWarp = kMmaWarp + 1, kTileWarp = kMmaWarp + (WIDEN ? 2 : 1);
  static constexpr int kThreads = 32 * (kProduce ? kPageWarp + 1 : kTileWarp + 1);
  static constexpr int kRows = 128 * MT;                   // rows of an A unit
  static constexpr int kTileBytes = D * 256;               // one tile: 128 rows x D 16-bit values
  static constexpr int kStages = (WIDEN ? 131072 : 196608) / kTileBytes;  // tiles in the ring
  static constexpr int kPageBytes = 8 * (D * KVQ_BLOCK_SIZE + 64);        // a key tile's codes, then its scales
  static constexpr int kPages = WIDEN ? 65536 / (D * 128) : 1;            // key tiles in the ring of pages
  static constexpr uint32_t kACols = D / 2;                // tensor-memory columns of an A tile
  static constexpr uint32_t kSCol = 256;                   // score tiles at 256 and 384
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kABufs = MT * 2 * kACols <= kSCol ? 2 : 1;  // A units held at a time
  static constexpr int offPages = kStages * kTileBytes;
  static constexpr int offPar = offPages + (WIDEN ? kPages * kPageBytes : 0);  // [buf][2][128] fp32
  static constexpr int offConst = offPar + kParBufs * 2 * 128 * 4;
  static constexpr int offValid = offConst + kConstBufs * kRows * 4;  // [buf][4] key bits
  static constexpr int offPageOk = offValid + kParBufs * 16;          // [page ring] bits of the pages that exist
  // phase of the last bulk copy into each tile, parameter buffer and page slot, -1: none
  static constexpr int offLast = offPageOk + 16;
  // Copies of an A unit (kARing, kProduce), a barrier each; four sets of them, since a slow loader warp may be
  // waiting for a unit when the copies of the second one after it have landed.
  static constexpr int kAParts = kProduce ? 2 * MT : MT;
  static constexpr int kASets = 4;
  static constexpr int kLasts = kStages + kParBufs + kPages + kAParts;
  static constexpr int offBar = offLast + 20 * 4;
  static constexpr int kNumBars = 2 * kStages + 4 + 2 * kParBufs + 4 + kConstBufs + 2 * kPages + kASets * kAParts + 1;
  static_assert(offBar % 8 == 0, "barriers");
  static constexpr int offFlag = offBar + kNumBars * 8;    // abort flag, TMEM base
  static constexpr int kAlloc = offFlag + 16 + 1024;
  static_assert(MT * kABufs * kACols <= kSCol && kSCol + 256 <= kTmemCols, "tensor memory");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  static_assert(kPages <= 4 && kLasts <= 20, "page bits, last copies");
  static_assert(!kProduce || kTileBytes / 2 <= kPageBytes, "half an A tile fits in a page slot");
  static_assert(!WIDEN || (kStages % 2 == 0 && kPages % 2 == 0 && kParBufs % 2 == 0), "a column pass slot belongs to one loader group");
  // barriers: tiles, score tiles, column parameters, A units, key constants, pages
  static constexpr int full = 0, empty = full + kStages, sFull = empty + kStages, sFree = sFull + 2, parFull = sFree + 2,
                       parFree = parFull + kParBufs, aFull = parFree + kParBufs, aFree = aFull + 2, constFull = aFree + 2,
                       pageFull = constFull + kConstBufs, pageFree = pageFull + kPages, aTile = pageFree + kPages, drain = aTile + kASets * kAParts;
  // Place in the ring of tiles of B tile f of the run, in its at-th A unit; the unit's A tile i (kARing) comes
  // MT - i places before its first B tile.
  __device__ static int entry(int f, int at) { return f + (kARing ? MT * (at + 1) : 0); }
  // barrier and phase of copy i of the at-th A unit
  __device__ static int a_tile(int at, int i) { return aTile + (at % kASets) * kAParts + i; }
  __device__ static int a_phase(int at) { return at / kASets; }
  // WIDEN row pass: place in the ring of pages of the key tile of B tile f; half h of the unit's A tile i comes
  // 2 (MT - i) - h places before its first key tile.
  __device__ static int page_entry(int f, int at) { return f + (kProduce ? 2 * MT * (at + 1) : 0); }
};

// B tiles of A unit t, and the first of them.
template <int PASS>
__device__ __forceinline__ int b_first(const ChunkWeightsArgs& a, int t) {
  // column pass: rows before the first query that sees the unit's first key see none of it
  return PASS == 1 ? 0 : max(0, a.a_rows[1] * t - a.history_len) * a.group / 128;
}
template <int PASS>
__device__ __forceinline__ int b_count(const ChunkWeightsArgs& a, int t) {
  if (PASS == 1) return (a.history_len + min(a.a_rows[0] * (t + 1) - 1, a.n_rows - 1) / a.group) / 128 + 1;
  return a.row_tiles - b_first<2>(a, t);
}

// The CTA whose run holds pair f of the line (runs start at floor(c N / P)).
__device__ __forceinline__ int run_of(long long f, long long n, int p) {
  return static_cast<int>(((f + 1) * p - 1) / n);
}

// Position on the line: KV head, A unit, B tile (counted from the A unit's first).
struct Walk {
  int kvh, t, b, n;
};

// The pair at f: a warp-wide search of the prefix sums of b_count.
template <int PASS>
__device__ Walk walk_at(const ChunkWeightsArgs& a, long long f) {
  const int lane = threadIdx.x & 31;
  const long long per = a.line[PASS - 1];
  Walk w;
  w.kvh = static_cast<int>(f / per);
  long long rem = f - w.kvh * per;
  const int tiles = a.units[PASS - 1];
  w.t = w.b = 0;
  w.n = 1;
  for (int base = 0; base < tiles; base += 32) {
    const int n = base + lane < tiles ? b_count<PASS>(a, base + lane) : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    if (rem < total) {
      const int l = __ffs(__ballot_sync(0xffffffffu, incl > rem)) - 1;
      w.t = base + l;
      w.n = __shfl_sync(0xffffffffu, n, l);
      w.b = static_cast<int>(rem) - (__shfl_sync(0xffffffffu, incl, l) - w.n);
      break;
    }
    rem -= total;
  }
  return w;
}

template <int PASS>
__device__ __forceinline__ void step(const ChunkWeightsArgs& a, Walk& w) {
  if (++w.b < w.n) return;
  w.b = 0;
  if (++w.t == a.units[PASS - 1]) {
    w.t = 0;
    ++w.kvh;
  }
  w.n = b_count<PASS>(a, w.t);
}

// 16 int8 codes -> eight words of two bf16 each.  With 0x43 above it, the low seven bits of a code are
// the bf16 number 128 + (code & 127), and its sign bit alone is 128 or 256: their difference is
// the code, exactly.
__device__ __forceinline__ void widen16_bf16(const uint4& raw, uint32_t* out) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = __byte_perm(w[i >> 1], 0x43434343u, (i & 1) ? kSelB23 : kSelB01);
    const uint32_t lo = v & 0xFF7FFF7Fu, hi = v & 0xFF80FF80u;
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo), *reinterpret_cast<const __nv_bfloat162*>(&hi));
    out[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
}

// The page of key t: its (page * n_kv_heads + kvh), or -1 (past the context, or outside the pool).
__device__ __forceinline__ long long key_ph(const ChunkWeightsArgs& a, int kvh, int t) {
  if (t >= a.n_keys) return -1;
  const int page = __ldg(a.block_table_row + t / KVQ_BLOCK_SIZE);
  if (page < 0 || page >= a.num_blocks) {
    set_status(a.status, KVQ_DEV_BAD_BLOCK);
    return -1;
  }
  return static_cast<long long>(page) * a.n_kv_heads + kvh;
}

}  // namespace

// Operand tiles: the first blocks lay the query rows of a KV head out (a row is G heads of a query in turn),
// kRowParts blocks a tile, the blocks after them widen 128 keys and leave their score factors and which of them exist.
constexpr int kRowParts = 4;

template <int D>
__global__ void __launch_bounds__(256) chunk_tiles_kernel(ChunkWeightsArgs a) {
  const int kvh = blockIdx.y, tid = threadIdx.x;
  __shared__ long long ph_s[8];
  grid_dep_trigger();  // the row pass may take its place; it waits for this grid before it reads
  grid_dep_wait();
  if (static_cast<int>(blockIdx.x) < kRowParts * a.row_tiles) {
    const int t = blockIdx.x / kRowParts, part = blockIdx.x % kRowParts;
    uint8_t* tile = a.q_tiles + (static_cast<long long>(kvh) * a.row_tiles + t) * (D * 256);
    constexpr int W = D / 8;  // 16-byte words of a row
    static_assert(W / 2 % kRowParts == 0, "whole passes of the block");
#pragma unroll
    for (int x = part * (W / 2 / kRowParts); x < (part + 1) * (W / 2 / kRowParts); ++x) {
      const int i = tid + 256 * x, n = i / W, c = i % W, r = 128 * t + n, q = r / a.group;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < a.n_rows)
        v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                 (static_cast<long long>(q) * a.n_q_heads + kvh * a.group + (r - q * a.group)) * D) + c);
      sts128(tile + (c >> 3) * kPieceBytes + tc::sw128_off(n, c & 7), v);  // a global store
    }
    return;
  }
  const int j = blockIdx.x - kRowParts * a.row_tiles;
  if (tid < 8) ph_s[tid] = key_ph(a, kvh, 128 * j + KVQ_BLOCK_SIZE * tid);
  __syncthreads();
  const long long u = static_cast<long long>(kvh) * a.key_tiles + j;
  uint8_t* tile = a.k_tiles + u * (D * 256);
  uint4 raw[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {  // four adjacent lanes fill one 128-byte row of a piece
    const int i = tid + 256 * x, n = (i >> 2) & 127, c16 = ((i >> 9) << 2) | (i & 3);
    const long long ph = ph_s[n >> 4];
    raw[x] = make_uint4(0, 0, 0, 0);
    if (ph >= 0 && 128 * j + n < a.n_keys)
      raw[x] = __ldg(reinterpret_cast<const uint4*>(a.k + (ph * (D / 16) + c16) * 256 + (n & 15) * 16));
  }
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {
    const int i = tid + 256 * x, n = (i >> 2) & 127, c16 = ((i >> 9) << 2) | (i & 3);
    uint32_t h[8];
    widen16_bf16(raw[x], h);
    uint8_t* piece = tile + (c16 >> 2) * kPieceBytes;
    const int cc = (c16 & 3) * 2;
    sts128(piece + tc::sw128_off(n, cc), make_uint4(h[0], h[1], h[2], h[3]));  // global stores
    sts128(piece + tc::sw128_off(n, cc + 1), make_uint4(h[4], h[5], h[6], h[7]));
  }
  if (tid < 128) {
    const long long ph = ph_s[tid >> 4];
    const bool real = ph >= 0 && 128 * j + tid < a.n_keys;
    a.k_par[u * 128 + tid] = real ? a.k_scale[ph * KVQ_BLOCK_SIZE + (tid & 15)] * a.c2 : 0.f;
    const uint32_t bits = __ballot_sync(0xffffffffu, real);
    if ((tid & 31) == 0) a.k_valid[u * 4 + (tid >> 5)] = bits;
  }
}

template <int D, int PASS, int MT, bool WIDEN>
__global__ void __launch_bounds__(Cw<D, PASS, MT, WIDEN>::kThreads, 1) chunk_weights_kernel(ChunkWeightsArgs a) {
  using L = Cw<D, PASS, MT, WIDEN>;
  constexpr int NP = D / 64;  // 16 KB pieces of a B tile
  constexpr int ST = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  float* par = reinterpret_cast<float*>(sm + L::offPar);
  float* consts = reinterpret_cast<float*>(sm + L::offConst);
  uint32_t* valid = reinterpret_cast<uint32_t*>(sm + L::offValid);
  volatile int* last_copy = reinterpret_cast<volatile int*>(sm + L::offLast);
  volatile uint32_t* page_ok = reinterpret_cast<volatile uint32_t*>(sm + L::offPageOk);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::offBar);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::offFlag);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::offFlag + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // WIDEN column pass with all row tiles in the ring at once: B tile j stays in stage (and parameter buffer) j
  // for all A units of a KV head, an epoch
  const bool resident = PASS == 2 && WIDEN && a.row_tiles <= min(ST, kParBufs);
  const long long total = a.line[PASS - 1] * a.n_kv_heads;
  const int P = static_cast<int>(gridDim.x);
  const long long f0 = total * blockIdx.x / P, f1 = total * (blockIdx.x + 1) / P;
  const int n_tiles = static_cast<int>(f1 - f0);
  Walk w = walk_at<PASS>(a, f0);
  if (warp == L::kMmaWarp) tc::tmem_alloc(tmem_slot, L::kTmemCols);
  if (tid == 0) {
    // a lane of each warp arrives for its warp: a thread's arrival costs as much as a warp's
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bars[L::full + s], L::kProduce ? 8 : 1);
      mbar_init(&bars[L::empty + s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[L::sFull + s], 1);
      mbar_init(&bars[L::sFree + s], kSoftWarps / 2);
      mbar_init(&bars[L::aFull + s], 4);
      mbar_init(&bars[L::aFree + s], 1);
    }
    for (int s = 0; s < kParBufs; ++s) {
      mbar_init(&bars[L::parFull + s], L::kProduce ? 4 : 1);
      mbar_init(&bars[L::parFree + s], MT == 2 || resident ? kSoftWarps : kSoftWarps / 2);
    }
    for (int s = 0; s < kConstBufs; ++s) mbar_init(&bars[L::constFull + s], 4);
    for (int s = 0; s < L::kPages; ++s) {
      mbar_init(&bars[L::pageFull + s], 1);
      mbar_init(&bars[L::pageFree + s], L::kProduce ? 8 : 4);
    }
    mbar_init(&bars[L::drain], 1);
    for (int s = 0; s < L::kASets * L::kAParts; ++s) mbar_init(&bars[L::aTile + s], 1);
    for (int s = 0; s < L::kLasts; ++s) last_copy[s] = -1;
    *abort_flag = 0;
    mbar_fence_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();  // everything above depends on the arguments alone
  auto wait = [&](int bar, uint32_t parity) {
    return wait_or_abort(&bars[bar], parity & 1u, a.status, abort_flag, a.wait_budget);
  };
  auto wait_warp = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
  auto arrive_warp = [&](int bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[bar]);
  };
  if (warp < kSoftWarps) {
    // ================================================================ softmax
    // Score tile g of the run is group g % 2's: with two A tiles a unit, one of them is; else every second B tile.
    const int group = warp >> 3, half = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
    const int tile = MT == 2 ? group : 0, part = MT == 2 ? half : 2 * group + half;
    const uint32_t tm_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + L::kSCol + 128 * group + 64 * half;
    // where this CTA's partial of the A unit at the walk goes: slot 0 unless an earlier run began it
    int slot = w.b == 0 ? 0 : static_cast<int>(blockIdx.x) - run_of(f0 - w.b, total, P);
    auto out_index = [&](const Walk& x) {
      const long long u = (static_cast<long long>(x.kvh) * a.units[PASS - 1] + x.t) * MT + tile;
      return (u * a.n_part[PASS - 1] + parts_of_run(MT) * slot + part) * 128 + row;
    };
    bool ok = true;
    int at = -1;    // ordinal of the current A unit in this CTA
    int first = 0;  // its first B tile
    int epoch = 0;
    // Row pass: reference and sum of the row, its last visible key.  Column pass: the key's sum, its score
    // factor, the first row that sees it.
    float m = -INFINITY, l = 0.f, cst = 0.f;
    int bound = 0;
    for (int f = 0; f < n_tiles; ++f) {
      if (f == 0 || w.b == 0) {
        ++at;
        if (PASS == 2) {
          ok = wait_warp(L::constFull + at % kConstBufs, at / kConstBufs);
          if (!ok) break;
        }
        first = b_first<PASS>(a, w.t);
        const int r = L::kRows * w.t + 128 * tile + row;
        if (PASS == 2) cst = consts[(at % kConstBufs) * L::kRows + 128 * tile + row];
        m = -INFINITY;
        l = 0.f;
        bound = PASS == 1 ? (r < a.n_rows ? a.history_len + r / a.group : -1) : max(0, r - a.history_len) * a.group;
      }
      if (MT == 2 || (f & 1) == group) {
        const int pb = resident ? first + w.b : f % kParBufs;
        ok = wait_warp(L::parFull + pb, resident ? epoch : f / kParBufs) && wait_warp(L::sFull + group, MT == 2 ? f : f >> 1);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int c0 = 64 * half + 32 * c;
          const float4* p0 = reinterpret_cast<const float4*>(par + (pb * 2 + 0) * 128 + c0);
          const float4* p1 = reinterpret_cast<const float4*>(par + (pb * 2 + 1) * 128 + c0);
          uint32_t sv[32];
          tc::ld_32x32b_x32(tm_s + 32 * c, sv);
          // columns of the chunk that count, as bits
          const uint32_t exist = PASS == 1 ? valid[pb * 4 + (c0 >> 5)] : 0u;
          uint32_t vis;
          if (PASS == 1) {
            const int n = bound - 128 * w.b + 1 - c0;
            vis = (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u) & exist;
          } else {
            const int r0 = 128 * (first + w.b) + c0, lo = bound - r0, hi = a.n_rows - r0;
            vis = (lo <= 0 ? 0xffffffffu : lo >= 32 ? 0u : ~((1u << lo) - 1u)) &
                  (hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1u);
          }
          const bool masked = __any_sync(0xffffffffu, vis != 0xffffffffu);
          tc::wait_ld();
          if (c == 1) {
            tc::fence_before_sync();
            arrive_warp(L::sFree + group);  // this warp's part of the score tile is in registers
          }
          if (PASS == 1) {
            // sum of 2^(s - ref) over the chunk, s = S * (k_scale c2)
            auto sum_from = [&](float ref) {
              const f2 nm2 = mk2(-ref, -ref);
              f2 sa = mk2(0.f, 0.f), sb = mk2(0.f, 0.f);
#pragma unroll
              for (int n = 0; n < 32; n += 4) {
                const float4 k4 = p0[n >> 2];
                const f2 xa = fma2(mk2(__uint_as_float(sv[n]), __uint_as_float(sv[n + 1])), mk2(k4.x, k4.y), nm2);
                const f2 xb = fma2(mk2(__uint_as_float(sv[n + 2]), __uint_as_float(sv[n + 3])), mk2(k4.z, k4.w), nm2);
                sa = add2(sa, mk2(fast_exp2(lo2(xa)), fast_exp2(hi2(xa))));
                sb = add2(sb, mk2(fast_exp2(lo2(xb)), fast_exp2(hi2(xb))));
              }
              return (lo2(sa) + lo2(sb)) + (hi2(sa) + hi2(sb));
            };
            float s = 0.f;
            bool plain = !masked && !__any_sync(0xffffffffu, m == -INFINITY);
            if (plain) {
              s = sum_from(m);
              plain = !__any_sync(0xffffffffu, !(s < kSumLimit));  // true for NaN
            }
            if (!plain) {  // masks, a first chunk, or a score far above the reference: scores, maximum, sum
              const float* k1 = par + (pb * 2 + 0) * 128 + c0;
              float cm = -INFINITY;
#pragma unroll
              for (int n = 0; n < 32; ++n) {
                const float y = ((vis >> n) & 1u) ? __uint_as_float(sv[n]) * k1[n] : -INFINITY;
                sv[n] = __float_as_uint(y);
                cm = fmaxf(cm, y);
              }
              // a first chunk, or more than 2^32 above the reference: the reference moves up
              if (m == -INFINITY || cm > m + 32.f) {
                if (m != -INFINITY) l *= fast_exp2(m - cm);
                m = cm;
              }
              const float ref = m == -INFINITY ? 0.f : m;
              s = 0.f;
#pragma unroll
              for (int n = 0; n < 32; ++n) s += fast_exp2(__uint_as_float(sv[n]) - ref);
            }
            l += s;
          } else {
            const f2 c2 = mk2(cst, cst);
            float tile_sum = 0.f;
            if (!masked) {
              f2 sa = mk2(0.f, 0.f), sb = mk2(0.f, 0.f);
#pragma unroll
              for (int n = 0; n < 32; n += 4) {
                const float4 nm = p0[n >> 2], il = p1[n >> 2];
                const f2 xa = fma2(mk2(__uint_as_float(sv[n]), __uint_as_float(sv[n + 1])), c2, mk2(nm.x, nm.y));
                const f2 xb = fma2(mk2(__uint_as_float(sv[n + 2]), __uint_as_float(sv[n + 3])), c2, mk2(nm.z, nm.w));
                sa = fma2(mk2(fast_exp2(lo2(xa)), fast_exp2(hi2(xa))), mk2(il.x, il.y), sa);
                sb = fma2(mk2(fast_exp2(lo2(xb)), fast_exp2(hi2(xb))), mk2(il.z, il.w), sb);
              }
              tile_sum = (lo2(sa) + lo2(sb)) + (hi2(sa) + hi2(sb));
            } else {
              const float* nm = par + (pb * 2 + 0) * 128 + c0;
              const float* il = par + (pb * 2 + 1) * 128 + c0;
#pragma unroll
              for (int n = 0; n < 32; ++n) {
                const float p = fast_exp2(fmaf(__uint_as_float(sv[n]), cst, nm[n])) * il[n];
                tile_sum += ((vis >> n) & 1u) ? p : 0.f;  // a row that does not see the key adds nothing, NaN neither
              }
            }
            l += tile_sum;
          }
        }
        if (!resident) arrive_warp(L::parFree + pb);
      }
      if (w.b + 1 == w.n || f + 1 == n_tiles) {  // the A unit, or this CTA's part of it, is done
        if (PASS == 1) a.row_part[out_index(w)] = make_float2(m, l);
        else a.col_part[out_index(w)] = l;
        slot = 0;
      }
      const int kvh = w.kvh;
      step<PASS>(a, w);
      if (resident && (w.kvh != kvh || f + 1 == n_tiles)) {  // every tile of the epoch, seen by a unit or not
        for (int j = 0; ok && j < a.row_tiles; ++j) {
          ok = wait_warp(L::parFull + j, epoch);
          if (ok && w.kvh != kvh) arrive_warp(L::parFree + j);
        }
        ++epoch;
        if (!ok) break;
      }
    }
    if (!ok) {
      // A wait ran out (KVQ_DEV_TIMEOUT is set): the rows of the A units from here on are marked as having
      // no sum (l < 0), the keys' parts as zero.
      for (long long f = f0; f < f1;) {
        Walk x = walk_at<PASS>(a, f);  // warp-wide
        slot = x.b == 0 ? 0 : static_cast<int>(blockIdx.x) - run_of(f - x.b, total, P);
        const long long end = min(f1, f + (x.n - x.b));
        if (x.kvh > w.kvh || (x.kvh == w.kvh && x.t >= w.t)) {
          if (PASS == 1) a.row_part[out_index(x)] = make_float2(0.f, -1.f);
          else a.col_part[out_index(x)] = 0.f;
        }
        f = end;
      }
    }
  } else if (L::kProduce && warp >= kProdWarp && warp < kProdWarp + 8) {
    // ================================================================ B producers: thread = key of the tile
    const int n = (tid - 32 * kProdWarp) & 127, group = (warp - kProdWarp) >> 2;
    bool ok = true;
    int at = -1;
    uint32_t phases = 0;  // per page slot: parity of its next key tile
    for (int f = 0; f < n_tiles; ++f) {
      if (f == 0 || w.b == 0) ++at;
      const int pb = f % kParBufs, s = f % ST, x = L::page_entry(f, at), ps = x % L::kPages;
      ok = wait_warp(L::pageFull + ps, phases >> ps);
      phases ^= 1u << ps;
      if (ok && group == 0 && f >= kParBufs) ok = wait_warp(L::parFree + pb, f / kParBufs - 1);
      if (ok && f >= ST) ok = wait_warp(L::empty + s, f / ST - 1);
      if (!ok) break;
      const uint8_t* page = sm + L::offPages + ps * L::kPageBytes;
      const uint8_t* src = page + (n >> 4) * (D * KVQ_BLOCK_SIZE) + (n & 15) * 16;
      uint8_t* tile = sm + s * L::kTileBytes;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {  // this group's half of the dims
        const int i = group * (D / 32) + j;
        uint32_t h[8];
        widen16_bf16(*reinterpret_cast<const uint4*>(src + i * 256), h);
        uint8_t* piece = tile + (i >> 2) * kPieceBytes;
        sts128(piece + tc::sw128_off(n, 2 * (i & 3)), make_uint4(h[0], h[1], h[2], h[3]));
        sts128(piece + tc::sw128_off(n, 2 * (i & 3) + 1), make_uint4(h[4], h[5], h[6], h[7]));
      }
      const bool real = ((page_ok[ps] >> (n >> 4)) & 1u) && 128 * w.b + n < a.n_keys;
      const float ks = reinterpret_cast<const float*>(page + 8 * D * KVQ_BLOCK_SIZE)[n];
      tc::fence_proxy_async_smem();  // each writer's stores come before the tensor core's reads
      // test-only fault injection: CTA 0's first tile is never announced
      if (!(a.fault == 4 && blockIdx.x == 0 && f == 0)) arrive_warp(L::full + s);
      if (group == 0) {
        par[(pb * 2 + 0) * 128 + n] = real ? ks * a.c2 : 0.f;
        const uint32_t bits = __ballot_sync(0xffffffffu, real);
        if (lane == 0) valid[pb * 4 + (n >> 5)] = bits;
        arrive_warp(L::parFull + pb);
      }
      arrive_warp(L::pageFree + ps);
      step<1>(a, w);
    }
  } else if (WIDEN && warp == L::kPageWarp) {
    // ================================================================ page copies: lane = page of the key tile
    // the key tiles of the run's B tiles (row pass), each unit's A tiles before them, or of its A units (column pass)
    auto page_at = [&](const Walk& v) {
      return lane < 8 ? key_ph(a, v.kvh, 128 * (PASS == 1 ? v.b : v.t) + KVQ_BLOCK_SIZE * lane) : -1;
    };
    long long ph = page_at(w);
    bool ok = true;
    int x = 0, at = -1;   // entries of the ring filled, A unit
    uint32_t phases = 0;  // per page slot: parity of its next key tile
    auto slot_free = [&] { return x < L::kPages || wait_warp(L::pageFree + x % L::kPages, x / L::kPages - 1); };
    for (int f = 0; f < n_tiles;) {
      if (L::kProduce && (f == 0 || w.b == 0)) {
        ++at;
        for (int i = 0; ok && i < 2 * MT; ++i) {
          ok = slot_free();
          if (!ok) break;
          if (lane == 0) {
            const int ps = x % L::kPages;
            // the second tile of the last unit may not exist: any tile will do, its rows count for nothing
            const long long u = static_cast<long long>(w.kvh) * a.row_tiles + min(MT * w.t + i / 2, a.row_tiles - 1);
            last_copy[ST + kParBufs + L::kPages + i] = at;
            mbar_arrive_expect_tx(&bars[L::a_tile(at, i)], L::kTileBytes / 2);
            bulk_g2s(sm + L::offPages + ps * L::kPageBytes, a.q_tiles + u * L::kTileBytes + (i & 1) * (L::kTileBytes / 2),
                     L::kTileBytes / 2, &bars[L::a_tile(at, i)]);
          }
          __syncwarp();
          ++x;
        }
      }
      ok = ok && slot_free();
      if (!ok) break;
      const int ps = x % L::kPages;
      const uint32_t exist = __ballot_sync(0xffffffffu, ph >= 0);
      if (lane == 0) {
        page_ok[ps] = exist;
        last_copy[ST + kParBufs + ps] = (phases >> ps) & 1u;
        mbar_arrive_expect_tx(&bars[L::pageFull + ps], __popc(exist) * (D * KVQ_BLOCK_SIZE + 64));
      }
      __syncwarp();
      if (ph >= 0) {  // codes of pages that do not exist are whatever was there: finite once widened, and masked
        uint8_t* page = sm + L::offPages + ps * L::kPageBytes;
        bulk_g2s(page + lane * (D * KVQ_BLOCK_SIZE), a.k + ph * (D * KVQ_BLOCK_SIZE), D * KVQ_BLOCK_SIZE, &bars[L::pageFull + ps]);
        bulk_g2s(page + 8 * D * KVQ_BLOCK_SIZE + lane * 64, a.k_scale + ph * KVQ_BLOCK_SIZE, 64, &bars[L::pageFull + ps]);
      }
      phases ^= 1u << ps;
      ++x;
      f += PASS == 1 ? 1 : w.n - w.b;
      if (PASS == 2) w.b = w.n - 1;
      step<PASS>(a, w);
      if (f < n_tiles) ph = page_at(w);  // the next tile's pages, while this one's copies run
    }
  } else if (!L::kProduce && warp == L::kTileWarp) {
    // ================================================================ tile copies (one lane)
    if (lane == 0) {
      int e = 0;  // ring entries filled
      // test-only fault injection: CTA 0's first key tile is not copied
      const bool skip_one = PASS == 1 && !WIDEN && a.fault == 4 && blockIdx.x == 0;
      auto copy_tile = [&](int s, int bar, int last, int phase, const uint8_t* src) {
        last_copy[last] = phase;
        mbar_arrive_expect_tx(&bars[bar], L::kTileBytes);
        bulk_g2s(sm + s * L::kTileBytes, src, L::kTileBytes, &bars[bar]);
      };
      uint32_t phases = 0;  // per stage: parity of its next B tile
      // the next entry of the ring: A tile i of unit at, or (i < 0) a B tile
      auto put = [&](const uint8_t* src, int i, int at, bool skip) {
        const int s = e % ST;
        if (e >= ST && !wait(L::empty + s, e / ST - 1)) return false;
        if (i >= 0) {
          copy_tile(s, L::a_tile(at, i), ST + kParBufs + L::kPages + i, at, src);
        } else {
          if (!skip) copy_tile(s, L::full + s, s, (phases >> s) & 1u, src);
          phases ^= 1u << s;
        }
        ++e;
        return true;
      };
      auto copy_columns = [&](int pb, int phase, long long u) {
        last_copy[ST + pb] = phase;
        if (PASS == 1) {
          mbar_arrive_expect_tx(&bars[L::parFull + pb], 512 + 16);
          bulk_g2s(par + (pb * 2 + 0) * 128, a.k_par + u * 128, 512, &bars[L::parFull + pb]);
          bulk_g2s(valid + pb * 4, a.k_valid + u * 4, 16, &bars[L::parFull + pb]);
        } else {
          mbar_arrive_expect_tx(&bars[L::parFull + pb], 1024);
          bulk_g2s(par + (pb * 2 + 0) * 128, a.row_nm + u * 128, 512, &bars[L::parFull + pb]);
          bulk_g2s(par + (pb * 2 + 1) * 128, a.row_il + u * 128, 512, &bars[L::parFull + pb]);
        }
      };
      bool ok = true;
      if (resident) {
        int epoch = 0;
        for (int f = 0; ok && f < n_tiles; ++epoch) {
          for (int j = 0; j < a.row_tiles; ++j) {
            if (epoch > 0) ok = wait(L::parFree + j, epoch - 1) && wait(L::empty + j, epoch - 1);
            if (!ok) break;
            const long long u = static_cast<long long>(w.kvh) * a.row_tiles + j;
            copy_columns(j, epoch, u);
            copy_tile(j, L::full + j, j, epoch, a.q_tiles + u * L::kTileBytes);
          }
          for (const int kvh = w.kvh; f < n_tiles && w.kvh == kvh; ++f) step<PASS>(a, w);
        }
      } else {
        for (int f = 0, at = -1; ok && f < n_tiles; ++f) {
          if (L::kARing && (f == 0 || w.b == 0)) {
            ++at;
            const uint8_t* tiles = PASS == 1 ? a.q_tiles : a.k_tiles;
            const int n = PASS == 1 ? a.row_tiles : a.key_tiles;
            // the second tile of the last unit may not exist: any tile will do, its rows count for nothing
            for (int i = 0; ok && i < MT; ++i)
              ok = put(tiles + (static_cast<long long>(w.kvh) * n + min(MT * w.t + i, n - 1)) * L::kTileBytes, i, at, false);
          }
          if (!ok) break;
          const int pb = f % kParBufs;
          if (f >= kParBufs && !wait(L::parFree + pb, f / kParBufs - 1)) break;
          const long long u = PASS == 1 ? static_cast<long long>(w.kvh) * a.key_tiles + w.b
                                        : static_cast<long long>(w.kvh) * a.row_tiles + b_first<2>(a, w.t) + w.b;
          copy_columns(pb, f / kParBufs, u);
          ok = put((PASS == 1 ? a.k_tiles : a.q_tiles) + u * L::kTileBytes, -1, 0, skip_one && f == 0);
          step<PASS>(a, w);
        }
      }
    }
    __syncwarp();  // the lanes go to the CTA's barrier together
  } else if (warp >= kLoadWarp && warp < kLoadWarp + 4 * L::kLoadGroups) {
    // ================================================================ A loaders: thread = row n of each A tile
    const int n = (tid - 32 * kLoadWarp) & 127, group = (warp - kLoadWarp) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    for (int f = 0, at = 0; ok && f < n_tiles; ++at) {
      const int ab = at % L::kABufs;
      if (L::kLoadGroups == 2 && (at & 1) != group) {  // the other group's unit, buffer and page slot
        f += w.n - w.b;
        w.b = w.n - 1;
        step<PASS>(a, w);
        continue;
      }
#pragma unroll 1
      for (int i = 0; ok && i < MT; ++i) {
        const uint32_t tm_a = tmem + lane_base + (ab * MT + i) * L::kACols;
        float cst = 0.f;
        if (PASS == 2 && !WIDEN) {
          const int t = min(MT * w.t + i, a.key_tiles - 1);
          cst = __ldg(a.k_par + (static_cast<long long>(w.kvh) * a.key_tiles + t) * 128 + n);
        }
        // kARing: a tile of the ring.  Row pass: two halves of a tile in the ring of pages.  Column pass: pages.
        constexpr int kParts = L::kProduce ? 2 : 1;
#pragma unroll
        for (int half = 0; half < kParts; ++half) {
          const int e = L::entry(f, at) - MT + i;
          const int x = L::kProduce ? L::page_entry(f, at) - 2 * (MT - i) + half : at;
          const int s = L::kARing ? e % ST : x % L::kPages;
          ok = L::kARing      ? wait_warp(L::a_tile(at, i), L::a_phase(at))
               : L::kProduce ? wait_warp(L::a_tile(at, 2 * i + half), L::a_phase(at))
                             : wait_warp(L::pageFull + s, x / L::kPages);
          // the MMAs of the unit that held this buffer are done
          if (ok && i == 0 && half == 0 && at >= L::kABufs) ok = wait_warp(L::aFree + ab, at / L::kABufs - 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint8_t* src = L::kARing ? sm + s * L::kTileBytes : sm + L::offPages + s * L::kPageBytes;
#pragma unroll
          for (int p = 0; p < NP / kParts; ++p) {
            uint32_t h[32];
            if (PASS == 1 || !WIDEN) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint4 v = *reinterpret_cast<const uint4*>(src + p * kPieceBytes + tc::sw128_off(n, c));
                h[4 * c] = v.x;
                h[4 * c + 1] = v.y;
                h[4 * c + 2] = v.z;
                h[4 * c + 3] = v.w;
              }
            } else {
              const uint8_t* key = src + (n >> 4) * (D * KVQ_BLOCK_SIZE) + (n & 15) * 16;
#pragma unroll
              for (int c = 0; c < 4; ++c) widen16_bf16(*reinterpret_cast<const uint4*>(key + (4 * p + c) * 256), h + 8 * c);
            }
            tc::st_32x32b_x32(tm_a + 32 * (half * (NP / kParts) + p), h);
          }
          if (PASS == 2 && WIDEN) cst = reinterpret_cast<const float*>(src + 8 * D * KVQ_BLOCK_SIZE)[n] * a.c2;
          if (PASS == 2) consts[(at % kConstBufs) * L::kRows + 128 * i + n] = cst;
          arrive_warp(L::kARing ? L::empty + s : L::pageFree + s);
          if (L::kProduce && lane == 0) mbar_arrive(&bars[L::pageFree + s]);  // a key tile has eight readers
        }
      }
      tc::wait_st();  // also when a wait ran out: nothing is on its way to tensor memory when it is given back
      if (!ok) break;
      tc::fence_before_sync();
      arrive_warp(L::aFull + ab);
      if (PASS == 2) arrive_warp(L::constFull + at % kConstBufs);
      f += w.n - w.b;
      w.b = w.n - 1;
      step<PASS>(a, w);
    }
  } else if (warp == L::kMmaWarp) {
    // ================================================================ MMA issue
    const uint64_t rd0 = tc::sdesc_sw128(smem_u32(sm));
    constexpr uint32_t idesc = tc::idesc_bf16_f32(128, 128);
    bool ok = true;
    int at = -1, epoch = 0, first = 0;
    uint32_t phases = 0;  // per stage: parity of its next B tile
    for (int f = 0; ok && f < n_tiles; ++f) {
      if (f == 0 || w.b == 0) {
        ++at;
        first = b_first<PASS>(a, w.t);
        ok = wait_warp(L::aFull + at % L::kABufs, at / L::kABufs);
      }
      const int s = resident ? first + w.b : L::entry(f, at) % ST;
      if (ok) ok = wait_warp(L::full + s, resident ? epoch : phases >> s);
      phases ^= 1u << s;
      const bool last = w.b + 1 == w.n || f + 1 == n_tiles;
      const int kvh = w.kvh;
      step<PASS>(a, w);
      const bool epoch_end = resident && w.kvh != kvh;
      const uint64_t bd0 = rd0 + static_cast<uint64_t>((s * L::kTileBytes) >> 4);
#pragma unroll 1
      for (int i = 0; ok && i < MT; ++i) {
        const int g = MT * f + i, sg = g & 1;
        if (g >= 2) ok = wait_warp(L::sFree + sg, (g >> 1) - 1);
        if (!ok) break;
        if (elect_one()) {
          tc::fence_after_sync();
          const uint32_t tm_a = tmem + ((at % L::kABufs) * MT + i) * L::kACols, tm_s = tmem + L::kSCol + 128 * sg;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_f16_ts(tm_s, tm_a + 8 * k, bd0 + (k >> 2) * (kPieceBytes >> 4) + 2 * (k & 3), idesc, k ? 1u : 0u);
          tc::commit(&bars[L::sFull + sg]);
          if (i == MT - 1) {
            // a stage is released by four arrivals (an A tile's are the four loader warps): three now, the last one
            // when the MMAs are done
            if (!resident) {
              for (int x = 0; x < 3; ++x) mbar_arrive(&bars[L::empty + s]);
              tc::commit(&bars[L::empty + s]);
            }
            if (last) tc::commit(&bars[L::aFree + at % L::kABufs]);
          }
        }
        __syncwarp();
      }
      // the epoch's tiles that no unit of this run saw (their phases are visited all the same)
      if (resident && (epoch_end || f + 1 == n_tiles))
        for (int j = 0; ok && j < a.row_tiles; ++j) ok = wait_warp(L::full + j, epoch);
      if (ok && epoch_end && elect_one()) {
        for (int j = 0; j < a.row_tiles; ++j) {
          for (int x = 0; x < 3; ++x) mbar_arrive(&bars[L::empty + j]);
          tc::commit(&bars[L::empty + j]);
        }
      }
      __syncwarp();
      epoch += epoch_end;
    }
    if (elect_one()) {
      tc::commit(&bars[L::drain]);
      mbar_wait(&bars[L::drain], 0, a.status, a.wait_budget);
    }
    __syncwarp();
  }

  grid_dep_trigger();
  tc::fence_before_sync();
  __syncthreads();
  // After an abort copies may still be in flight: they land before the CTA exits (within microseconds, so the
  // waits are short).
  if (*abort_flag && tid == 0) {
    for (int s = 0; s < L::kLasts; ++s) {
      const int at = last_copy[s], i = s - ST - kParBufs - L::kPages;
      const int bar = s < ST                             ? L::full + s
                      : s < ST + kParBufs              ? L::parFull + (s - ST)
                      : s < ST + kParBufs + L::kPages ? L::pageFull + (s - ST - kParBufs)
                                                       : L::a_tile(max(at, 0), i);
      if (at >= 0) mbar_wait(&bars[bar], (i < 0 ? at : L::a_phase(at)) & 1, nullptr, 1000000);
      // (the A unit before that one too: its copies may be as young)
      if (i >= 0 && at > 0) mbar_wait(&bars[L::a_tile(at - 1, i)], L::a_phase(at - 1) & 1, nullptr, 1000000);
    }
  }
  if (warp == L::kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Runs that hold a part of A unit t of KV head kvh: the number of them (block-wide; the prefix of the
// units before it is summed by the block's threads, 256 at most).
template <int PASS>
__device__ int segments_of(const ChunkWeightsArgs& a, int kvh, int t) {
  __shared__ long long warp_sum[8];
  long long s = 0;
  for (int x = threadIdx.x; x < t; x += blockDim.x) s += b_count<PASS>(a, x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  const long long line = a.line[PASS - 1], total = line * a.n_kv_heads;
  const int runs = a.runs[PASS - 1];
  long long f = kvh * line;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) f += warp_sum[i];
  return run_of(f + b_count<PASS>(a, t) - 1, total, runs) - run_of(f, total, runs) + 1;
}

// Row statistics of the column pass: minus the reference and 1 / l, from the parts of the row pass.  A lane
// takes a row; WARPS warps share a row's parts (a row cut over a whole GPU has dozens) and a CTA of 8 warps
// has 8 / WARPS times 32 rows.
constexpr int kRowWarps = 8;
// Parts of a row up to which a warp takes them all.  2048 row tiles of a few parts each: 5.7 us against 10.2 with
// eight warps a row; 8 row tiles of 76 parts: 6.6 us with eight warps, one would read them one after another.
constexpr int kFewParts = 16;

template <int WARPS>
__global__ void __launch_bounds__(kRowWarps * 32) chunk_rows_kernel(ChunkWeightsArgs a) {
  __shared__ float2 part_s[kRowWarps][32];
  constexpr int kRows = kRowWarps / WARPS * 32;
  const int kvh = blockIdx.y, warp = threadIdx.x / 32 % WARPS, group = threadIdx.x / 32 / WARPS, lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x) * kRows / 128, n_all = static_cast<int>(blockIdx.x) * kRows + 32 * group + lane;
  const int mt = a.a_rows[0] / 128;
  grid_dep_trigger();
  const int parts = parts_of_run(mt) * segments_of<1>(a, kvh, t / mt);
  grid_dep_wait();
  const int tile = n_all / 128, n = n_all % 128;  // a CTA's rows are of one A unit
  if (tile >= a.row_tiles) return;
  const float2* p = a.row_part + (static_cast<long long>(kvh) * a.units[0] * mt + tile) * a.n_part[0] * 128 + n;
  // (m, l) of several (m, l): the largest m, the sums moved onto it; a sum below zero marks a dropped part.  A part
  // without a maximum has the sum 0 (no key) or NaN (every score is), and 2^-inf times it is the same.
  float m = -INFINITY, l = 0.f;
  bool dropped = false;
  auto merge = [&](const float2& v) {
    const float x = fmaxf(m, v.x), ref = x == -INFINITY ? 0.f : x;
    l = fmaf(v.y, fast_exp2(v.x - ref), l * fast_exp2(m - ref));
    m = x;
    dropped = dropped || v.y < 0.f;
  };
  for (int i0 = warp; i0 < parts; i0 += 8 * WARPS) {
    float2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = i0 + WARPS * i < parts ? p[(i0 + WARPS * i) * 128] : make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) merge(v[i]);
  }
  if (WARPS > 1) {
    static_assert(WARPS == 1 || WARPS == kRowWarps, "a block barrier joins one group");
    part_s[warp][lane] = make_float2(m, dropped ? -1.f : l);
    __syncthreads();
    if (warp != 0) return;
    for (int i = 1; i < WARPS; ++i) merge(part_s[i][lane]);
  }
  if (dropped) l = -1.f;
  // A row with no key gives no weight; nor does one without its sum, whatever its scores: 2^(s - inf) is 0, while 2^s
  // may be infinite.
  const long long r = (static_cast<long long>(kvh) * a.row_tiles + tile) * 128 + n;
  a.row_nm[r] = l < 0.f ? -INFINITY : m == -INFINITY ? 0.f : -m;
  a.row_il[r] = l < 0.f || l == 0.f ? 0.f : __fdiv_rn(1.0f, l);
}

// acc += the parts of the column pass, in the order of the line.
__global__ void __launch_bounds__(128) chunk_acc_kernel(ChunkWeightsArgs a) {
  const int t = blockIdx.x, kvh = blockIdx.y, n = threadIdx.x;
  const int mt = a.a_rows[1] / 128;
  const int parts = parts_of_run(mt) * segments_of<2>(a, kvh, t / mt);
  grid_dep_wait();
  const int key = 128 * t + n;
  if (key >= a.n_keys) return;
  const int page = a.block_table_row[key / KVQ_BLOCK_SIZE];
  if (page < 0 || page >= a.num_blocks) return;
  const float* p = a.col_part + (static_cast<long long>(kvh) * a.units[1] * mt + t) * a.n_part[1] * 128 + n;
  float s = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) s += p[i * 128];
  a.acc[kvh * a.acc_stride + key] += s;
}

ChunkWeightsPlan chunk_weights_plan(int n_tokens, int n_q_heads, int n_kv_heads, int history_len, int head_dim,
                                    int n_sms) {
  ChunkWeightsPlan p{};
  const long long G = n_q_heads / n_kv_heads;
  const long long rows = n_tokens * G, keys = static_cast<long long>(history_len) + n_tokens;
  p.row_tiles = static_cast<int>((rows + 127) / 128);
  p.key_tiles = static_cast<int>((keys + 127) / 128);
  // Two A tiles a unit share each B tile; one A tile a unit is loaded ahead of its use.  The row pass has
  // many B tiles a unit, so it takes two wherever there are two; the column pass does when the rows are
  // many enough to outweigh the loads.
  p.a_rows[0] = p.row_tiles > 1 ? 256 : 128;  // measured at the top of this file
  p.widen_once = p.row_tiles >= 8;
  p.a_rows[1] = p.widen_once ? 256 : 128;
  long long most[2] = {0, 0};
  p.units[0] = static_cast<int>((rows + p.a_rows[0] - 1) / p.a_rows[0]);
  p.units[1] = static_cast<int>((keys + p.a_rows[1] - 1) / p.a_rows[1]);
  for (long long t = 0; t < p.units[0]; ++t) {
    const long long n = (history_len + std::min(p.a_rows[0] * (t + 1) - 1, rows - 1) / G) / 128 + 1;
    p.line[0] += n;
    most[0] = std::max(most[0], n);
  }
  for (long long t = 0; t < p.units[1]; ++t) {
    const long long n = p.row_tiles - std::max(0LL, p.a_rows[1] * t - history_len) * G / 128;
    p.line[1] += n;
    most[1] = std::max(most[1], n);
  }
  long long part[2];
  for (int i = 0; i < 2; ++i) {
    const long long total = p.line[i] * n_kv_heads;
    p.runs[i] = static_cast<int>(std::min<long long>(total, n_sms));
    // an A unit of n pairs lies in at most ceil(n / floor(total / runs)) + 1 runs, and in no more than there are
    const long long shortest = total / p.runs[i];
    const long long seg = std::min<long long>(p.runs[i], (most[i] + shortest - 1) / shortest + 1);
    p.n_part[i] = parts_of_run(p.a_rows[i] / 128) * static_cast<int>(seg);
    part[i] = static_cast<long long>(n_kv_heads) * p.units[i] * p.a_rows[i] * p.n_part[i];
  }
  auto round = [](long long x) { return (x + 255) / 256 * 256; };
  const long long row_n = static_cast<long long>(n_kv_heads) * p.row_tiles * 128;
  p.off_nm = round(part[0] * 8);
  p.off_il = p.off_nm + round(row_n * 4);
  p.off_q = p.off_il + round(row_n * 4);
  p.off_col = p.off_q + row_n * head_dim * 2;
  p.bytes = p.off_col + part[1] * 4;
  if (p.widen_once) {
    const long long key_n = static_cast<long long>(n_kv_heads) * p.key_tiles * 128;
    p.off_k = round(p.bytes);
    p.off_kpar = p.off_k + key_n * head_dim * 2;
    p.off_kvalid = p.off_kpar + key_n * 4;
    p.bytes = p.off_kvalid + key_n / 8;
  }
  return p;
}

template <int D, int PASS, int MT, bool WIDEN>
static cudaError_t launch_pass(const ChunkWeightsArgs& a, cudaStream_t stream) {
  using L = Cw<D, PASS, MT, WIDEN>;
  auto kern = chunk_weights_kernel<D, PASS, MT, WIDEN>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), L::kAlloc, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.runs[PASS - 1]), dim3(L::kThreads), L::kAlloc, stream, a);
}

template <int D>
static cudaError_t launch_chunk_weights_d(const ChunkWeightsArgs& a, cudaStream_t stream) {
  const bool once = a.k_tiles != nullptr;
  cudaError_t e = launch_pdl(chunk_tiles_kernel<D>, dim3(kRowParts * a.row_tiles + (once ? a.key_tiles : 0), a.n_kv_heads), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  e = once                  ? launch_pass<D, 1, 2, false>(a, stream)
      : a.a_rows[0] == 256 ? launch_pass<D, 1, 2, true>(a, stream)
                           : launch_pass<D, 1, 1, true>(a, stream);
  if (e != cudaSuccess) return e;
  e = a.n_part[0] > kFewParts
          ? launch_pdl(chunk_rows_kernel<kRowWarps>, dim3(4 * a.row_tiles, a.n_kv_heads), dim3(kRowWarps * 32), 0, stream, a)
          : launch_pdl(chunk_rows_kernel<1>, dim3((a.row_tiles + 1) / 2, a.n_kv_heads), dim3(kRowWarps * 32), 0, stream, a);
  if (e != cudaSuccess) return e;
  e = once ? launch_pass<D, 2, 2, false>(a, stream) : launch_pass<D, 2, 1, true>(a, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_acc_kernel, dim3(a.key_tiles, a.n_kv_heads), dim3(128), 0, stream, a);
}

cudaError_t launch_chunk_weights(const ChunkWeightsArgs& a, cudaStream_t stream) {
  return a.head_dim == 256 ? launch_chunk_weights_d<256>(a, stream) : launch_chunk_weights_d<128>(a, stream);
}

}  // namespace kvq
