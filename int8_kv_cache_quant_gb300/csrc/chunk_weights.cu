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
// Operands.  sm_103a has no integer tcgen05 kind, and the codes are exact in 16 bits: the row pass widens
// K to fp16 and scales each query row by a power of two (exact for bf16 values within 2^29 of the row's
// largest); the column pass takes the bf16 queries as they are and widens the codes to bf16 (exact:
// |code| < 2^8).  Either way every product is exact and the sums are fp32.  The row pass widens in the
// producer warps, from global memory through registers into the swizzled shared-memory tile: the codes
// are read as bytes (half of what a widened copy would move) and no copy of K is ever written.  The
// queries, far smaller, are laid out once in the swizzled tile order by the row pass, on its way
// through them, so that the column pass brings a tile in with one bulk copy.
//
// Schedule.  One CTA per SM; the (A unit, B tile) pairs of all KV heads are one line, cut into equal
// runs, one per CTA, so that causal and ragged shapes balance to a tile.  An A unit is one 128-row tile
// (MT = 1, held twice: the next one loads while this one is in use) or two of them (MT = 2), which
// share every B tile: a 128 x 128 tile pair at head_dim 256 takes 1024 cycles of the tensor core, in
// which one SM would have to take in 64 KB of queries, more than all SMs together get out of L2;
// with two A tiles it is half of that.  An A unit that two CTAs share leaves one partial each, and the
// partials are added in the order of the line: the same result every time.  Roles of a CTA's warps:
//   warps 0-7    softmax: group w / 4 takes every second 128 x 128 tile of scores (MT = 2: its A tile's),
//                thread = tensor-memory lane 32 (w % 4) + lane
//   warps 8-11   row pass: B producers (128 threads); column pass: warp 8 issues the bulk copies, warp 9
//                the MMAs
//   warps 12-15  A loaders (128 threads)
//   warp 16      row pass: MMA issue
// Tensor memory: A tiles (head_dim / 2 columns each) | two score tiles, one a softmax group.
//
// What bounds it: at head_dim 256 the tensor core (1024 cycles a 128 x 128 tile at 4096 multiply-adds a
// cycle and SM; its 16384 exponentials take 512 at 32 a cycle), at head_dim 128 both alike.
#include <algorithm>

#include <cuda_bf16.h>

#include "kvq_dev.cuh"
#include "kvq_launch.h"
#include "tcgen05.cuh"
#include "tile_dev.cuh"

namespace kvq {

namespace {

constexpr int kSoftWarps = 8, kProdWarp = 8, kLoadWarp = 12;
constexpr int kParBufs = 4;    // column parameters, by B tile
// Row constants, by A unit.  A softmax group can lag behind the A loaders by five units (of one B tile
// each: the other group's tiles go on until the MMA needs this group's score tile), so the constants
// have more buffers than the A tiles, and barriers of their own, whose phases cannot pass the reader.
constexpr int kConstBufs = 8;
constexpr float kRefSlack = 8.0f;  // a running maximum stays until it is exceeded by 2^8

template <int D, int PASS, int MT>
struct Cw {
  static constexpr int kThreads = PASS == 1 ? 17 * 32 : 16 * 32;
  static constexpr int kMmaWarp = PASS == 1 ? 16 : 9;
  static constexpr int kRows = 128 * MT;                   // rows of an A unit
  static constexpr int kTileBytes = D * 256;               // one B tile: 128 rows x D 16-bit values
  static constexpr int kStages = 196608 / kTileBytes;      // 3 at head_dim 256, 6 at 128
  static constexpr uint32_t kACols = D / 2;                // tensor-memory columns of an A tile
  static constexpr uint32_t kSCol = 256;                   // score tiles at 256 and 384
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kABufs = MT * 2 * kACols <= kSCol ? 2 : 1;  // A units held at a time
  static constexpr int offPar = kStages * kTileBytes;      // [buf][2][128] fp32
  static constexpr int offConst = offPar + kParBufs * 2 * 128 * 4;
  static constexpr int offValid = offConst + kConstBufs * kRows * 4;  // [buf][4] key bits
  static constexpr int offBar = offValid + kParBufs * 16;
  static constexpr int kNumBars = 2 * kStages + 4 + 2 * kParBufs + 4 + kConstBufs + 1;
  static constexpr int offFlag = offBar + kNumBars * 8;    // abort flag, TMEM base
  static constexpr int kAlloc = offFlag + 16 + 1024;
  static_assert(MT * kABufs * kACols <= kSCol && kSCol + 256 <= kTmemCols, "tensor memory");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  // barriers: B stages, score tiles (one a softmax group), column parameters, A units
  static constexpr int full = 0, empty = full + kStages, sFull = empty + kStages, sFree = sFull + 2, parFull = sFree + 2,
                       parFree = parFull + kParBufs, aFull = parFree + kParBufs, aFree = aFull + 2, constFull = aFree + 2, drain = constFull + kConstBufs;
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

template <int D, int PASS, int MT>
__global__ void __launch_bounds__(Cw<D, PASS, MT>::kThreads, 1) chunk_weights_kernel(ChunkWeightsArgs a) {
  using L = Cw<D, PASS, MT>;
  constexpr int NP = D / 64;  // 16 KB pieces of a B tile
  constexpr int ST = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  float* par = reinterpret_cast<float*>(sm + L::offPar);
  float* consts = reinterpret_cast<float*>(sm + L::offConst);
  uint32_t* valid = reinterpret_cast<uint32_t*>(sm + L::offValid);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::offBar);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::offFlag);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::offFlag + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  grid_dep_wait();
  const long long total = a.line[PASS - 1] * a.n_kv_heads;
  const int P = static_cast<int>(gridDim.x);
  const long long f0 = total * blockIdx.x / P, f1 = total * (blockIdx.x + 1) / P;
  const int n_tiles = static_cast<int>(f1 - f0);
  Walk w = walk_at<PASS>(a, f0);
  if (warp == L::kMmaWarp) tc::tmem_alloc(tmem_slot, L::kTmemCols);
  if (tid == 0) {
    // a lane of each warp arrives for its warp: a thread's arrival costs as much as a warp's
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bars[L::full + s], PASS == 1 ? 4 : 1);
      mbar_init(&bars[L::empty + s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[L::sFull + s], 1);
      mbar_init(&bars[L::sFree + s], 4);
      mbar_init(&bars[L::aFull + s], 4);
      mbar_init(&bars[L::aFree + s], 1);
    }
    for (int s = 0; s < kParBufs; ++s) {
      mbar_init(&bars[L::parFull + s], PASS == 1 ? 4 : 1);
      mbar_init(&bars[L::parFree + s], 4 * MT);  // MT = 1: only the group whose tile it is reads them
    }
    for (int s = 0; s < kConstBufs; ++s) mbar_init(&bars[L::constFull + s], 4);
    mbar_init(&bars[L::drain], 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
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
    const int grp = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tm_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + L::kSCol + 128 * grp;
    // where this CTA's partial of the A unit at the walk goes: slot 0 unless an earlier run began it
    int slot = w.b == 0 ? 0 : static_cast<int>(blockIdx.x) - run_of(f0 - w.b, total, P);
    // parts of a 128-row tile: [slot] (MT = 2), or [slot][group] (MT = 1)
    auto out_index = [&](const Walk& x) {
      const long long u = (static_cast<long long>(x.kvh) * a.units[PASS - 1] + x.t) * MT + (MT == 2 ? grp : 0);
      return (u * a.n_part[PASS - 1] + (MT == 2 ? slot : 2 * slot + grp)) * 128 + row;
    };
    const int arow = (MT == 2 ? 128 * grp : 0) + row;  // row of the A unit
    bool ok = true;
    int at = -1;       // ordinal of the current A unit in this CTA
    int mine = 0;      // score tiles this group has taken
    float cst = 0.f;   // row pass: the row's score factor; column pass: the key's
    float m = -INFINITY, l = 0.f;
    int bound = 0;     // row pass: last visible key; column pass: first row that sees the key
    for (int f = 0; f < n_tiles; ++f) {
      if (f == 0 || w.b == 0) {
        ++at;
        ok = wait_warp(L::constFull + at % kConstBufs, at / kConstBufs);
        if (!ok) break;
        cst = consts[(at % kConstBufs) * L::kRows + arow];
        m = -INFINITY;
        l = 0.f;
        const int r = L::kRows * w.t + arow;
        if (PASS == 1) bound = r < a.n_rows ? a.history_len + r / a.group : -1;
        else bound = max(0, r - a.history_len) * a.group;
      }
      if (MT == 2 || (f & 1) == grp) {
        const int pb = f % kParBufs;
        ok = wait_warp(L::sFull + grp, mine) && wait_warp(L::parFull + pb, f / kParBufs);
        if (!ok) break;
        tc::fence_after_sync();
        float tile_sum = 0.f;
        uint32_t buf[2][32];
        tc::ld_32x32b_x32(tm_s, buf[0]);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t (&sv)[32] = buf[ch & 1];
          tc::wait_ld();
          if (ch < 3) {
            tc::ld_32x32b_x32(tm_s + 32 * (ch + 1), buf[(ch + 1) & 1]);  // on its way while this chunk is worked on
          } else {
            tc::fence_before_sync();
            arrive_warp(L::sFree + grp);  // the tile is in registers
          }
          const int c0 = 32 * ch;  // first column of the chunk
          const float4* p0 = reinterpret_cast<const float4*>(par + (pb * 2 + 0) * 128 + c0);
          const float4* p1 = reinterpret_cast<const float4*>(par + (pb * 2 + 1) * 128 + c0);
          // columns of the chunk that count, as bits
          uint32_t vis;
          if (PASS == 1) {
            const int n = bound - 128 * w.b + 1 - c0;
            vis = (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u) & valid[pb * 4 + ch];
          } else {
            const int r0 = 128 * (b_first<2>(a, w.t) + w.b) + c0;
            const int lo = bound - r0, hi = a.n_rows - r0;
            vis = (lo <= 0 ? 0xffffffffu : lo >= 32 ? 0u : ~((1u << lo) - 1u)) &
                  (hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1u);
          }
          const bool masked = __any_sync(0xffffffffu, vis != 0xffffffffu);
          if (PASS == 1) {
            float ym0 = -INFINITY, ym1 = -INFINITY;
#pragma unroll
            for (int n = 0; n < 32; n += 4) {
              const float4 k4 = p0[n >> 2];
              const f2 ya = mul2(mk2(__uint_as_float(sv[n]), __uint_as_float(sv[n + 1])), mk2(k4.x, k4.y));
              const f2 yb = mul2(mk2(__uint_as_float(sv[n + 2]), __uint_as_float(sv[n + 3])), mk2(k4.z, k4.w));
              sv[n] = __float_as_uint(lo2(ya));
              sv[n + 1] = __float_as_uint(hi2(ya));
              sv[n + 2] = __float_as_uint(lo2(yb));
              sv[n + 3] = __float_as_uint(hi2(yb));
              ym0 = fmax3(ym0, lo2(ya), hi2(ya));
              ym1 = fmax3(ym1, lo2(yb), hi2(yb));
            }
            float ym = fmaxf(ym0, ym1);
            if (masked) {
              ym = -INFINITY;
#pragma unroll
              for (int n = 0; n < 32; ++n) {
                if (!((vis >> n) & 1u)) sv[n] = 0xFF800000u;  // -inf
                ym = fmaxf(ym, __uint_as_float(sv[n]));
              }
            }
            const float cm = ym * cst;
            if (cm > m + kRefSlack) {
              l *= fast_exp2(m - cm);
              m = cm;
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const f2 c2 = mk2(cst, cst), nm2 = mk2(-ref, -ref);
            f2 s = mk2(0.f, 0.f);
#pragma unroll
            for (int n = 0; n < 32; n += 2) {
              const f2 x = fma2(mk2(__uint_as_float(sv[n]), __uint_as_float(sv[n + 1])), c2, nm2);
              s = add2(s, mk2(fast_exp2(lo2(x)), fast_exp2(hi2(x))));
            }
            l += lo2(s) + hi2(s);
          } else {
            const f2 c2 = mk2(cst, cst);
            f2 s = mk2(0.f, 0.f);
            if (!masked) {
#pragma unroll
              for (int n = 0; n < 32; n += 4) {
                const float4 nm = p0[n >> 2], il = p1[n >> 2];
                const f2 xa = fma2(mk2(__uint_as_float(sv[n]), __uint_as_float(sv[n + 1])), c2, mk2(nm.x, nm.y));
                const f2 xb = fma2(mk2(__uint_as_float(sv[n + 2]), __uint_as_float(sv[n + 3])), c2, mk2(nm.z, nm.w));
                s = fma2(mk2(fast_exp2(lo2(xa)), fast_exp2(hi2(xa))), mk2(il.x, il.y), s);
                s = fma2(mk2(fast_exp2(lo2(xb)), fast_exp2(hi2(xb))), mk2(il.z, il.w), s);
              }
              tile_sum += lo2(s) + hi2(s);
            } else {
              const float* nm = par + (pb * 2 + 0) * 128 + c0;
              const float* il = par + (pb * 2 + 1) * 128 + c0;
#pragma unroll
              for (int n = 0; n < 32; ++n) {
                const float p = fast_exp2(fmaf(__uint_as_float(sv[n]), cst, nm[n])) * il[n];
                tile_sum += ((vis >> n) & 1u) ? p : 0.f;  // a row that does not see the key adds nothing, NaN neither
              }
            }
          }
        }
        arrive_warp(L::parFree + pb);
        if (PASS == 2) l += tile_sum;
        ++mine;
      }
      if (w.b + 1 == w.n || f + 1 == n_tiles) {  // the A unit, or this CTA's part of it, is done
        if (PASS == 1) a.row_part[out_index(w)] = make_float2(m, l);
        else a.col_part[out_index(w)] = l;
        slot = 0;
      }
      step<PASS>(a, w);
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
  } else if (PASS == 1 && warp < kLoadWarp) {
    // ================================================================ row pass: B producers, thread = key of the tile
    const int n = tid - 32 * kProdWarp;
    constexpr int NI = D / 16;
    int4 raw[NI];  // the codes of the whole head dimension, one tile ahead
    float ks = 0.f;
    bool real = false, ok = true;
    const int8_t* src = nullptr;
    auto fetch = [&](const Walk& x) {
      const int t = 128 * x.b + n;
      const long long ph = key_ph(a, x.kvh, t);
      real = ph >= 0;
      src = a.k + (real ? ph : 0) * (D * KVQ_BLOCK_SIZE) + (t % KVQ_BLOCK_SIZE) * 16;
      ks = real ? __ldg(a.k_scale + ph * KVQ_BLOCK_SIZE + t % KVQ_BLOCK_SIZE) : 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        raw[i] = make_int4(0, 0, 0, 0);
        if (real) raw[i] = __ldg(reinterpret_cast<const int4*>(src + i * 256));
      }
    };
    fetch(w);
    for (int f = 0; f < n_tiles; ++f) {
      const int pb = f % kParBufs, s = f % ST;
      if (f >= kParBufs) ok = wait_warp(L::parFree + pb, f / kParBufs - 1);
      if (ok && f >= ST) ok = wait_warp(L::empty + s, f / ST - 1);
      if (!ok) break;
      par[(pb * 2 + 0) * 128 + n] = ks;
      const uint32_t bits = __ballot_sync(0xffffffffu, real);
      if (lane == 0) valid[pb * 4 + (n >> 5)] = bits;
      arrive_warp(L::parFull + pb);
      uint8_t* tile = sm + s * L::kTileBytes;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint4 c0, c1;
        widen16(raw[i], c0, c1);
        uint8_t* piece = tile + (i >> 2) * kPieceBytes;
        sts128(piece + tc::sw128_off(n, 2 * (i & 3)), c0);
        sts128(piece + tc::sw128_off(n, 2 * (i & 3) + 1), c1);
      }
      // test-only fault injection: CTA 0's first tile is never announced
      if (!(a.fault == 4 && blockIdx.x == 0 && f == 0)) arrive_warp(L::full + s);
      step<1>(a, w);
      if (f + 1 < n_tiles) fetch(w);
    }
  } else if (PASS == 2 && warp == kProdWarp) {
    // ================================================================ column pass: bulk copies (one lane)
    if (lane == 0) {
      int f = 0;
      for (; f < n_tiles; ++f) {
        const int pb = f % kParBufs, s = f % ST;
        if (f >= kParBufs && !wait(L::parFree + pb, f / kParBufs - 1)) break;
        if (f >= ST && !wait(L::empty + s, f / ST - 1)) break;
        const long long u = static_cast<long long>(w.kvh) * a.row_tiles + b_first<2>(a, w.t) + w.b;
        mbar_arrive_expect_tx(&bars[L::parFull + pb], 1024);
        bulk_g2s(par + (pb * 2 + 0) * 128, a.row_nm + u * 128, 512, &bars[L::parFull + pb]);
        bulk_g2s(par + (pb * 2 + 1) * 128, a.row_il + u * 128, 512, &bars[L::parFull + pb]);
        mbar_arrive_expect_tx(&bars[L::full + s], L::kTileBytes);
        bulk_g2s(sm + s * L::kTileBytes, a.q_tiles + u * L::kTileBytes, L::kTileBytes, &bars[L::full + s]);
        step<2>(a, w);
      }
      // copies still in flight (after an abort) land before the CTA exits
      for (int g = max(0, f - ST); g < f; ++g) mbar_wait(&bars[L::full + g % ST], (g / ST) & 1, a.status, a.wait_budget);
      for (int g = max(0, f - kParBufs); g < f; ++g)
        mbar_wait(&bars[L::parFull + g % kParBufs], (g / kParBufs) & 1, a.status, a.wait_budget);
    }
  } else if (warp >= kLoadWarp && warp < kLoadWarp + 4) {
    // ================================================================ A loaders: thread = row n of each A tile
    const int n = tid - 32 * kLoadWarp;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    for (int f = 0, at = 0; ok && f < n_tiles; ++at) {
      const int ab = at % L::kABufs;
#pragma unroll 1
      for (int i = 0; ok && i < MT; ++i) {
        const uint32_t tm_a = tmem + lane_base + (ab * MT + i) * L::kACols;
        float cst = 0.f;
        const int r = L::kRows * w.t + 128 * i + n;
        if (PASS == 1) {
          const bool real = r < a.n_rows;
          const int q = r / a.group;
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(a.q) +
              (real ? (static_cast<long long>(q) * a.n_q_heads + w.kvh * a.group + (r - q * a.group)) * D : 0));
          // the row's largest magnitude; on the way the run that begins the A unit lays the row out for the
          // column pass
          const int tile = MT * w.t + i;
          uint8_t* image = w.b == 0 && tile < a.row_tiles
                               ? a.q_tiles + (static_cast<long long>(w.kvh) * a.row_tiles + tile) * L::kTileBytes
                               : nullptr;
          float amax = 0.f;
#pragma unroll 8
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              amax = fmax3(amax, fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u)));
            if (image) sts128(image + (c >> 3) * kPieceBytes + tc::sw128_off(n, c & 7), v);  // a global store
          }
          float to_f16, back;
          pow2_scales(amax, to_f16, back);
          cst = real ? back * a.c2 : 0.f;
          if (i == 0 && at >= L::kABufs) ok = wait_warp(L::aFree + ab, at / L::kABufs - 1);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            uint32_t h[32];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint4 v = real ? __ldg(src + 8 * p + c) : make_uint4(0, 0, 0, 0);
              const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[4 * c + e] = pack_half2(__uint_as_float(x[e] << 16) * to_f16, __uint_as_float(x[e] & 0xFFFF0000u) * to_f16);
            }
            tc::st_32x32b_x32(tm_a + 32 * p, h);
          }
        } else {
          constexpr int NI = D / 16;
          const long long ph = key_ph(a, w.kvh, r);
          const uint4* src = reinterpret_cast<const uint4*>(a.k + (ph < 0 ? 0 : ph) * (D * KVQ_BLOCK_SIZE) +
                                                            (r % KVQ_BLOCK_SIZE) * 16);
          uint4 raw[NI];
#pragma unroll
          for (int c = 0; c < NI; ++c) raw[c] = ph < 0 ? make_uint4(0, 0, 0, 0) : __ldg(src + c * 16);
          cst = ph < 0 ? 0.f : __ldg(a.k_scale + ph * KVQ_BLOCK_SIZE + r % KVQ_BLOCK_SIZE) * a.c2;
          if (i == 0 && at >= L::kABufs) ok = wait_warp(L::aFree + ab, at / L::kABufs - 1);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            uint32_t h[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) widen16_bf16(raw[4 * p + c], h + 8 * c);
            tc::st_32x32b_x32(tm_a + 32 * p, h);
          }
        }
        consts[(at % kConstBufs) * L::kRows + 128 * i + n] = cst;
      }
      if (!ok) break;
      tc::wait_st();
      tc::fence_before_sync();
      arrive_warp(L::aFull + ab);
      arrive_warp(L::constFull + at % kConstBufs);
      // the next A unit of the run
      f += w.n - w.b;
      w.b = w.n - 1;
      step<PASS>(a, w);
    }
  } else if (warp == L::kMmaWarp) {
    // ================================================================ MMA issue
    const uint64_t rd0 = tc::sdesc_sw128(smem_u32(sm));
    constexpr uint32_t idesc = PASS == 1 ? tc::idesc_f16_f32(128, 128) : tc::idesc_bf16_f32(128, 128);
    bool ok = true;
    int at = -1;
    for (int f = 0; ok && f < n_tiles; ++f) {
      if (f == 0 || w.b == 0) {
        ++at;
        ok = wait_warp(L::aFull + at % L::kABufs, at / L::kABufs);
      }
      const int s = f % ST;
      if (ok) ok = wait_warp(L::full + s, f / ST);
      const bool last = w.b + 1 == w.n || f + 1 == n_tiles;
      const uint64_t bd0 = rd0 + static_cast<uint64_t>((s * L::kTileBytes) >> 4);
#pragma unroll 1
      for (int i = 0; ok && i < MT; ++i) {
        const int g = MT * f + i, sg = g & 1;  // score tile g belongs to softmax group g % 2
        if (g >= 2) ok = wait_warp(L::sFree + sg, g / 2 - 1);
        if (!ok) break;
        if (elect_one()) {
          // The producers' stores come before the tensor core's reads.  The fence is taken here, on the thread that
          // has acquired them, and not by the producers: there it would wait for every load they have in flight.
          if (PASS == 1 && i == 0) tc::fence_proxy_async_smem();
          tc::fence_after_sync();
          const uint32_t tm_a = tmem + ((at % L::kABufs) * MT + i) * L::kACols, tm_s = tmem + L::kSCol + 128 * sg;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_f16_ts(tm_s, tm_a + 8 * k, bd0 + (k >> 2) * (kPieceBytes >> 4) + 2 * (k & 3), idesc, k ? 1u : 0u);
          tc::commit(&bars[L::sFull + sg]);
          if (i == MT - 1) {
            tc::commit(&bars[L::empty + s]);
            if (last) tc::commit(&bars[L::aFree + at % L::kABufs]);
          }
        }
        __syncwarp();
      }
      step<PASS>(a, w);
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
  if (warp == L::kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Runs that hold a part of A unit t of KV head kvh: the number of them (block-wide; the prefix of the
// units before it is summed by the block's 128 threads).
template <int PASS>
__device__ int segments_of(const ChunkWeightsArgs& a, int kvh, int t) {
  __shared__ long long warp_sum[4];
  long long s = 0;
  for (int x = threadIdx.x; x < t; x += 128) s += b_count<PASS>(a, x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  const long long line = a.line[PASS - 1], total = line * a.n_kv_heads;
  const int runs = a.runs[PASS - 1];
  const long long f = kvh * line + warp_sum[0] + warp_sum[1] + warp_sum[2] + warp_sum[3];
  return run_of(f + b_count<PASS>(a, t) - 1, total, runs) - run_of(f, total, runs) + 1;
}

// Row statistics of the column pass: -M and 1 / l from the parts of the row pass.
__global__ void __launch_bounds__(128) chunk_rows_kernel(ChunkWeightsArgs a) {
  const int t = blockIdx.x, kvh = blockIdx.y, n = threadIdx.x;
  const int mt = a.a_rows[0] / 128;
  const int parts = segments_of<1>(a, kvh, t / mt) * (mt == 2 ? 1 : 2);
  grid_dep_wait();
  const float2* p = a.row_part + (static_cast<long long>(kvh) * a.units[0] * mt + t) * a.n_part[0] * 128 + n;
  float m = -INFINITY;
  bool dropped = false;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float2 v = p[i * 128];
    m = fmaxf(m, v.x);
    dropped |= v.y < 0.f;
  }
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float2 v = p[i * 128];
    if (v.x != -INFINITY) l += v.y * fast_exp2(v.x - ref);
  }
  // a row with no key (or without its sum) gives no weight
  const long long u = static_cast<long long>(kvh) * a.row_tiles + t;
  a.row_nm[u * 128 + n] = -ref;
  a.row_il[u * 128 + n] = dropped || l == 0.f ? 0.f : __fdiv_rn(1.0f, l);
}

// acc += the parts of the column pass, in the order of the line.
__global__ void __launch_bounds__(128) chunk_acc_kernel(ChunkWeightsArgs a) {
  const int t = blockIdx.x, kvh = blockIdx.y, n = threadIdx.x;
  const int mt = a.a_rows[1] / 128;
  const int parts = segments_of<2>(a, kvh, t / mt) * (mt == 2 ? 1 : 2);
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
  p.a_rows[0] = p.row_tiles > 1 ? 256 : 128;
  p.a_rows[1] = p.row_tiles >= 8 ? 256 : 128;
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
    const int mt = p.a_rows[i] / 128;
    p.n_part[i] = static_cast<int>(mt == 2 ? seg : 2 * seg);
    part[i] = static_cast<long long>(n_kv_heads) * p.units[i] * mt * p.n_part[i] * 128;
  }
  auto round = [](long long x) { return (x + 255) / 256 * 256; };
  const long long row_n = static_cast<long long>(n_kv_heads) * p.row_tiles * 128;
  p.off_nm = round(part[0] * 8);
  p.off_il = p.off_nm + round(row_n * 4);
  p.off_q = p.off_il + round(row_n * 4);
  p.off_col = p.off_q + row_n * head_dim * 2;
  p.bytes = p.off_col + part[1] * 4;
  return p;
}

template <int D, int PASS, int MT>
static cudaError_t launch_pass(const ChunkWeightsArgs& a, cudaStream_t stream) {
  using L = Cw<D, PASS, MT>;
  auto kern = chunk_weights_kernel<D, PASS, MT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.runs[PASS - 1]), dim3(L::kThreads), L::kAlloc, stream, a);
}

template <int D>
static cudaError_t launch_chunk_weights_d(const ChunkWeightsArgs& a, cudaStream_t stream) {
  cudaError_t e = a.a_rows[0] == 256 ? launch_pass<D, 1, 2>(a, stream) : launch_pass<D, 1, 1>(a, stream);
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(chunk_rows_kernel, dim3(a.row_tiles, a.n_kv_heads), dim3(128), 0, stream, a)) != cudaSuccess) return e;
  e = a.a_rows[1] == 256 ? launch_pass<D, 2, 2>(a, stream) : launch_pass<D, 2, 1>(a, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_acc_kernel, dim3(a.key_tiles, a.n_kv_heads), dim3(128), 0, stream, a);
}

cudaError_t launch_chunk_weights(const ChunkWeightsArgs& a, cudaStream_t stream) {
  return a.head_dim == 256 ? launch_chunk_weights_d<256>(a, stream) : launch_chunk_weights_d<128>(a, stream);
}

}  // namespace kvq
