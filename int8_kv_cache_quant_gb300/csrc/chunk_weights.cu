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
// are read as bytes (half of what a widened copy would move) and no copy of K is ever written.
//
// Schedule.  One CTA per SM; the (A tile, B tile) pairs of all KV heads are one line, cut into equal
// runs, one per CTA, so that causal and ragged shapes balance to a tile.  An A tile that two CTAs
// share leaves one partial each, and the partials are added in the order of the line: the same result
// every time.  Roles of a CTA's 17 warps:
//   warps 0-7    softmax: warp w has tensor-memory lanes 32 (w % 4) .., columns 64 (w / 4) .. of each S tile
//   warps 8-11   B producers (128 threads)
//   warps 12-15  A loaders (128 threads): the next A tile goes into the other A buffer
//   warp 16      MMA issue
// Tensor memory: A twice (head_dim / 2 columns each) | S tiles (two at head_dim 256, three at 128).
//
// What bounds it: at head_dim 256 the tensor core (a 128 x 128 x 256 tile takes 1024 cycles at 4096
// multiply-adds a cycle and SM) and the special-function unit (16384 exponentials at 16 a cycle: 1024
// cycles) alike; at head_dim 128 the exponentials alone.
#include <algorithm>

#include <cuda_bf16.h>

#include "kvq_dev.cuh"
#include "kvq_launch.h"
#include "tcgen05.cuh"
#include "tile_dev.cuh"

namespace kvq {

namespace {

constexpr int kSoftThreads = 256;
constexpr int kProdWarp = 8, kLoadWarp = 12, kCwMmaWarp = 16;
constexpr int kCwThreads = 17 * 32;
constexpr int kRing = 12;      // operand pieces of 16 KB
constexpr int kParBufs = 4;    // column parameters
constexpr int kConstBufs = 8;  // row constants: more than the softmax warps can lag behind the A loaders
constexpr int kLag = 4;        // column pass: pieces whose copies are in flight behind the one being issued
constexpr float kRefSlack = 8.0f;  // a running maximum stays until it is exceeded by 2^8

template <int D>
struct CwSmem {
  static constexpr int kS = D == 256 ? 2 : 3;              // S tiles
  static constexpr int offPar = kRing * kPieceBytes;       // [buf][2][128] fp32
  static constexpr int offConst = offPar + kParBufs * 2 * 128 * 4;
  static constexpr int offValid = offConst + kConstBufs * 128 * 4;  // [buf][4] key bits
  static constexpr int offBar = offValid + kParBufs * 16;
  static constexpr int kNumBars = 2 * kRing + 2 * kS + 2 * kParBufs + 5;
  static constexpr int offFlag = offBar + kNumBars * 8;    // abort flag, TMEM base
  static constexpr int kAlloc = offFlag + 16 + 1024;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kACols = D / 2;
  static constexpr uint32_t kSCol = 2 * kACols;
  static_assert(kSCol + kS * 128 <= kTmemCols, "tensor memory");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  // barriers
  static constexpr int full = 0, empty = full + kRing, sFull = empty + kRing, sFree = sFull + kS,
                       parFull = sFree + kS, parFree = parFull + kParBufs, aFull = parFree + kParBufs,
                       aFree = aFull + 2, drain = aFree + 2;
};

// B tiles of A tile t, and the first of them.
template <int PASS>
__device__ __forceinline__ int b_first(const ChunkWeightsArgs& a, int t) {
  // column pass: rows before the first query that sees the tile's first key see none of it
  return PASS == 1 ? 0 : max(0, 128 * t - a.history_len) * a.group / 128;
}
template <int PASS>
__device__ __forceinline__ int b_count(const ChunkWeightsArgs& a, int t) {
  if (PASS == 1) return (a.history_len + min(128 * t + 127, a.n_rows - 1) / a.group) / 128 + 1;
  return a.row_tiles - b_first<2>(a, t);
}

// The CTA whose run holds pair f of the line (runs start at floor(c N / P)).
__device__ __forceinline__ int run_of(long long f, long long n, int p) {
  return static_cast<int>(((f + 1) * p - 1) / n);
}

// Position on the line: KV head, A tile, B tile (counted from the A tile's first).
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
  const int tiles = PASS == 1 ? a.row_tiles : a.key_tiles;
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
  if (++w.t == (PASS == 1 ? a.row_tiles : a.key_tiles)) {
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;  // 0: the 16 bytes are zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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

template <int D, int PASS>
__global__ void __launch_bounds__(kCwThreads, 1) chunk_weights_kernel(ChunkWeightsArgs a) {
  using L = CwSmem<D>;
  constexpr int NP = D / 64;  // pieces per B tile
  constexpr int NS = L::kS;
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
  if (warp == kCwMmaWarp) tc::tmem_alloc(tmem_slot, L::kTmemCols);
  if (tid == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&bars[L::full + s], 4);  // a lane of each producer warp arrives: a thread's arrival costs as much as a warp's
      mbar_init(&bars[L::empty + s], 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars[L::sFull + s], 1);
      mbar_init(&bars[L::sFree + s], kSoftThreads / 32);
    }
    for (int s = 0; s < kParBufs; ++s) {
      mbar_init(&bars[L::parFull + s], 4);
      mbar_init(&bars[L::parFree + s], kSoftThreads / 32);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[L::aFull + s], 4);
      mbar_init(&bars[L::aFree + s], 1);
    }
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
  auto arrive_warp = [&](int bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[bar]);
  };
  auto wait_warp = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };

  if (warp < kProdWarp) {
    // ================================================================ softmax
    const int part = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tm_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + L::kSCol + 64 * part;
    const int nseg = a.n_seg[PASS - 1];
    // where this CTA's partial of the A tile at the walk goes: slot 0 unless an earlier run began it
    int slot = w.b == 0 ? 0 : static_cast<int>(blockIdx.x) - run_of(f0 - w.b, total, P);
    auto out_index = [&](const Walk& x) {
      const long long u = static_cast<long long>(x.kvh) * (PASS == 1 ? a.row_tiles : a.key_tiles) + x.t;
      return ((u * nseg + slot) * 2 + part) * 128 + row;
    };
    bool ok = true;
    int at = -1;       // ordinal of the current A tile in this CTA
    float cst = 0.f;   // row pass: the row's score factor; column pass: the key's
    float m = -INFINITY, l = 0.f;
    int bound = 0;     // row pass: last visible key; column pass: first row that sees the key
    for (int f = 0; f < n_tiles; ++f) {
      if (f == 0 || w.b == 0) {
        ++at;
        ok = wait_warp(L::aFull + (at & 1), at >> 1);
        if (!ok) break;
        cst = consts[(at % kConstBufs) * 128 + row];
        m = -INFINITY;
        l = 0.f;
        if (PASS == 1) {
          const int r = 128 * w.t + row;
          bound = r < a.n_rows ? a.history_len + r / a.group : -1;
        } else {
          bound = max(0, 128 * w.t + row - a.history_len) * a.group;
        }
      }
      const int sb = f % NS, pb = f % kParBufs;
      ok = wait_warp(L::sFull + sb, f / NS) && wait_warp(L::parFull + pb, f / kParBufs);
      if (!ok) break;
      tc::fence_after_sync();
      float tile_sum = 0.f;
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t sv[32];
        tc::ld_32x32b_x32(tm_s + sb * 128 + 32 * ch, sv);
        tc::wait_ld();
        if (ch == 1) {
          tc::fence_before_sync();
          arrive_warp(L::sFree + sb);  // this warp's part of S is in registers
        }
        const int c0 = 64 * part + 32 * ch;  // first column of the chunk
        const float4* p0 = reinterpret_cast<const float4*>(par + (pb * 2 + 0) * 128 + c0);
        const float4* p1 = reinterpret_cast<const float4*>(par + (pb * 2 + 1) * 128 + c0);
        // columns of the chunk that count, as bits
        uint32_t vis;
        if (PASS == 1) {
          const int n = bound - 128 * w.b + 1 - c0;
          vis = (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u) & valid[pb * 4 + 2 * part + ch];
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
      l += PASS == 2 ? tile_sum : 0.f;
      if (w.b + 1 == w.n || f + 1 == n_tiles) {  // the A tile, or this CTA's part of it, is done
        if (PASS == 1) a.row_part[out_index(w)] = make_float2(m, l);
        else a.col_part[out_index(w)] = l;
        slot = 0;
      }
      step<PASS>(a, w);
    }
    if (!ok) {
      // A wait ran out (KVQ_DEV_TIMEOUT is set): the rows of the A tiles from here on are marked as having
      // no sum (l < 0), the keys' parts as zero.
      for (long long f = f0; f < f1;) {
        Walk x = walk_at<PASS>(a, f);  // warp-wide
        slot = x.b == 0 ? 0 : static_cast<int>(blockIdx.x) - run_of(f - x.b, total, P);
        const long long end = min(f1, f + (x.n - x.b));
        const bool open = x.kvh > w.kvh || (x.kvh == w.kvh && x.t >= w.t);
        if (open) {
          if (PASS == 1) a.row_part[out_index(x)] = make_float2(0.f, -1.f);
          else a.col_part[out_index(x)] = 0.f;
        }
        f = end;
      }
    }
  } else if (warp < kLoadWarp) {
    // ================================================================ B producers
    const int n = tid - 32 * kProdWarp;  // 0 .. 127
    uint8_t* ring = sm;
    int fill = 0;  // pieces begun
    bool ok = true;
    if (PASS == 1) {
      // thread = key n of the tile: its codes of the whole head dimension are one tile ahead in registers
      constexpr int NI = D / 16;
      int4 raw[NI];
      float ks = 0.f;
      bool real = false;
      const int8_t* src = nullptr;
      auto seek = [&](const Walk& x) {
        const int t = 128 * x.b + n;
        const long long ph = key_ph(a, x.kvh, t);
        real = ph >= 0;
        src = a.k + (real ? ph : 0) * (D * KVQ_BLOCK_SIZE) + (t % KVQ_BLOCK_SIZE) * 16;
        ks = real ? __ldg(a.k_scale + ph * KVQ_BLOCK_SIZE + t % KVQ_BLOCK_SIZE) : 0.f;
      };
      auto fetch = [&](int i) {
        raw[i] = make_int4(0, 0, 0, 0);
        if (real) raw[i] = __ldg(reinterpret_cast<const int4*>(src + i * 256));
      };
      seek(w);
#pragma unroll
      for (int i = 0; i < NI; ++i) fetch(i);
      for (int f = 0; ok && f < n_tiles; ++f) {
        const int pb = f % kParBufs;
        if (f >= kParBufs) ok = wait_warp(L::parFree + pb, f / kParBufs - 1);
        if (!ok) break;
        par[(pb * 2 + 0) * 128 + n] = ks;
        const uint32_t bits = __ballot_sync(0xffffffffu, real);
        if (lane == 0) valid[pb * 4 + (n >> 5)] = bits;
        arrive_warp(L::parFull + pb);
        step<1>(a, w);
        const bool more = f + 1 < n_tiles;
        if (more) seek(w);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int s = fill % kRing;
          if (fill >= kRing && !wait_warp(L::empty + s, fill / kRing - 1)) {
            ok = false;
            break;
          }
          uint8_t* piece = ring + s * kPieceBytes;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 c0, c1;
            widen16(raw[4 * p + i], c0, c1);
            sts128(piece + tc::sw128_off(n, 2 * i), c0);
            sts128(piece + tc::sw128_off(n, 2 * i + 1), c1);
            if (more) fetch(4 * p + i);
          }
          // test-only fault injection: the first piece of CTA 0's second tile is never announced
          if (!(a.fault == 4 && blockIdx.x == 0 && f == 1 && p == 0)) arrive_warp(L::full + s);
          ++fill;
        }
      }
    } else {
      // 16-byte chunk n % 8 of rows n / 8 + 16 i; a piece is announced kLag pieces after its copies were issued
      const int cc = n & 7, r8 = n >> 3;
      int done = 0;
      auto announce = [&]() {
        arrive_warp(L::full + done % kRing);
        ++done;
      };
      auto stats = [&](const Walk& x, float& nm, float& il) {
        const long long r = static_cast<long long>(x.kvh) * a.row_tiles * 128 + 128 * (b_first<2>(a, x.t) + x.b) + n;
        nm = __ldg(a.row_nm + r);
        il = __ldg(a.row_il + r);
      };
      float nm, il;
      stats(w, nm, il);
      for (int f = 0; ok && f < n_tiles; ++f) {
        const int pb = f % kParBufs;
        if (f >= kParBufs) ok = wait_warp(L::parFree + pb, f / kParBufs - 1);
        if (!ok) break;
        par[(pb * 2 + 0) * 128 + n] = nm;
        par[(pb * 2 + 1) * 128 + n] = il;
        arrive_warp(L::parFull + pb);
        const int r0 = 128 * (b_first<2>(a, w.t) + w.b);
        const uint16_t* base = static_cast<const uint16_t*>(a.q) + static_cast<long long>(w.kvh) * a.group * D + 8 * cc;
        long long off[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + r8 + 16 * i, q = r / a.group;
          off[i] = r < a.n_rows ? (static_cast<long long>(q) * a.n_q_heads + (r - q * a.group)) * D : -1;
        }
        step<2>(a, w);
        if (f + 1 < n_tiles) stats(w, nm, il);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int s = fill % kRing;
          if (fill >= kRing && !wait_warp(L::empty + s, fill / kRing - 1)) {
            ok = false;
            break;
          }
          const uint32_t piece = smem_u32(ring + s * kPieceBytes);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            cp_async16(piece + tc::sw128_off(r8 + 16 * i, cc), base + (off[i] < 0 ? 0 : off[i]) + 64 * p, off[i] >= 0);
          cp_commit();
          ++fill;
          if (fill > kLag) {
            cp_wait<kLag>();
            announce();
          }
        }
      }
      cp_wait<0>();
      while (ok && done < fill) announce();
    }
  } else if (warp < kCwMmaWarp) {
    // ================================================================ A loaders: thread = row n of the A tile
    const int n = tid - 32 * kLoadWarp;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    for (int f = 0, at = 0; ok && f < n_tiles; ++at) {
      const uint32_t tm_a = tmem + lane_base + (at & 1) * L::kACols;
      float cst = 0.f;
      if (PASS == 1) {
        const int r = 128 * w.t + n;
        const bool real = r < a.n_rows;
        const int q = r / a.group;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) +
            (real ? (static_cast<long long>(q) * a.n_q_heads + w.kvh * a.group + (r - q * a.group)) * D : 0));
        float amax = 0.f;
#pragma unroll 8
        for (int i = 0; i < D / 8; ++i) {
          const uint4 v = __ldg(src + i);
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmax3(amax, fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u)));
        }
        float to_f16, back;
        pow2_scales(amax, to_f16, back);
        cst = real ? back * a.c2 : 0.f;
        if (at >= 2) ok = wait_warp(L::aFree + (at & 1), (at >> 1) - 1);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          uint32_t h[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 v = real ? __ldg(src + 8 * p + i) : make_uint4(0, 0, 0, 0);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[4 * i + e] = pack_half2(__uint_as_float(x[e] << 16) * to_f16, __uint_as_float(x[e] & 0xFFFF0000u) * to_f16);
          }
          tc::st_32x32b_x32(tm_a + 32 * p, h);
        }
      } else {
        constexpr int NI = D / 16;
        const int t = 128 * w.t + n;
        const long long ph = key_ph(a, w.kvh, t);
        const uint4* src = reinterpret_cast<const uint4*>(a.k + (ph < 0 ? 0 : ph) * (D * KVQ_BLOCK_SIZE) +
                                                          (t % KVQ_BLOCK_SIZE) * 16);
        uint4 raw[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) raw[i] = ph < 0 ? make_uint4(0, 0, 0, 0) : __ldg(src + i * 16);
        cst = ph < 0 ? 0.f : __ldg(a.k_scale + ph * KVQ_BLOCK_SIZE + t % KVQ_BLOCK_SIZE) * a.c2;
        if (at >= 2) ok = wait_warp(L::aFree + (at & 1), (at >> 1) - 1);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          uint32_t h[32];
#pragma unroll
          for (int i = 0; i < 4; ++i) widen16_bf16(raw[4 * p + i], h + 8 * i);
          tc::st_32x32b_x32(tm_a + 32 * p, h);
        }
      }
      tc::wait_st();
      consts[(at % kConstBufs) * 128 + n] = cst;
      tc::fence_before_sync();
      arrive_warp(L::aFull + (at & 1));
      // the next A tile of the run
      f += w.n - w.b;
      w.b = w.n - 1;
      step<PASS>(a, w);
    }
  } else {
    // ================================================================ MMA issue
    const uint64_t rd0 = tc::sdesc_sw128(smem_u32(sm));
    constexpr uint32_t idesc = PASS == 1 ? tc::idesc_f16_f32(128, 128) : tc::idesc_bf16_f32(128, 128);
    bool ok = true;
    int used = 0, at = -1;
    for (int f = 0; ok && f < n_tiles; ++f) {
      if (f == 0 || w.b == 0) {
        ++at;
        ok = wait_warp(L::aFull + (at & 1), at >> 1);
      }
      const int sb = f % NS;
      if (ok && f >= NS) ok = wait_warp(L::sFree + sb, f / NS - 1);
      const bool last = w.b + 1 == w.n || f + 1 == n_tiles;
      const uint32_t tm_a = tmem + (at & 1) * L::kACols, tm_s = tmem + L::kSCol + sb * 128;
      for (int p = 0; ok && p < NP; ++p) {
        const int s = used % kRing;
        ok = wait_warp(L::full + s, used / kRing);
        if (!ok) break;
        if (elect_one()) {
          // The producers' stores come before the tensor core's reads.  The fence is taken here, on the thread that
          // has acquired them, and not by the producers: there it waits for every load they have in flight.
          tc::fence_proxy_async_smem();
          tc::fence_after_sync();
          const uint64_t bd = rd0 + static_cast<uint64_t>((s * kPieceBytes) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) tc::mma_f16_ts(tm_s, tm_a + 32 * p + 8 * k, bd + 2 * k, idesc, (p | k) ? 1u : 0u);
          tc::commit(&bars[L::empty + s]);
          if (p == NP - 1) {
            tc::commit(&bars[L::sFull + sb]);
            if (last) tc::commit(&bars[L::aFree + (at & 1)]);
          }
        }
        __syncwarp();
        ++used;
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
  if (warp == kCwMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Runs that hold a part of A tile t of KV head kvh: the number of them (block-wide; the prefix of the
// tiles before it is summed by the block's 128 threads).
template <int PASS>
__device__ int segments_of(const ChunkWeightsArgs& a, int kvh, int t, int runs) {
  __shared__ long long warp_sum[4];
  long long s = 0;
  for (int x = threadIdx.x; x < t; x += 128) s += b_count<PASS>(a, x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  const long long line = a.line[PASS - 1], total = line * a.n_kv_heads;
  const long long f = kvh * line + warp_sum[0] + warp_sum[1] + warp_sum[2] + warp_sum[3];
  return run_of(f + b_count<PASS>(a, t) - 1, total, runs) - run_of(f, total, runs) + 1;
}

// Row statistics of the column pass: -M and 1 / l from the parts of the row pass.
__global__ void __launch_bounds__(128) chunk_rows_kernel(ChunkWeightsArgs a) {
  const int t = blockIdx.x, kvh = blockIdx.y, n = threadIdx.x;
  const int parts = 2 * segments_of<1>(a, kvh, t, a.runs[0]);
  grid_dep_wait();
  const long long u = static_cast<long long>(kvh) * a.row_tiles + t;
  const float2* p = a.row_part + u * a.n_seg[0] * 256 + n;
  float m = -INFINITY;
  bool dropped = false;
  for (int i = 0; i < parts; ++i) {
    const float2 v = p[i * 128];
    m = fmaxf(m, v.x);
    dropped |= v.y < 0.f;
  }
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int i = 0; i < parts; ++i) {
    const float2 v = p[i * 128];
    if (v.x != -INFINITY) l += v.y * fast_exp2(v.x - ref);
  }
  // a row with no key (or without its sum) gives no weight
  a.row_nm[u * 128 + n] = -ref;
  a.row_il[u * 128 + n] = dropped || l == 0.f ? 0.f : __fdiv_rn(1.0f, l);
}

// acc += the parts of the column pass, in the order of the line.
__global__ void __launch_bounds__(128) chunk_acc_kernel(ChunkWeightsArgs a) {
  const int t = blockIdx.x, kvh = blockIdx.y, n = threadIdx.x;
  const int parts = 2 * segments_of<2>(a, kvh, t, a.runs[1]);
  grid_dep_wait();
  const int key = 128 * t + n;
  if (key >= a.n_keys) return;
  const int page = a.block_table_row[key / KVQ_BLOCK_SIZE];
  if (page < 0 || page >= a.num_blocks) return;
  const float* p = a.col_part + (static_cast<long long>(kvh) * a.key_tiles + t) * a.n_seg[1] * 256 + n;
  float s = 0.f;
  for (int i = 0; i < parts; ++i) s += p[i * 128];
  a.acc[kvh * a.acc_stride + key] += s;
}

ChunkWeightsPlan chunk_weights_plan(int n_tokens, int n_q_heads, int n_kv_heads, int history_len, int n_sms) {
  ChunkWeightsPlan p{};
  const long long G = n_q_heads / n_kv_heads;
  const long long rows = n_tokens * G, keys = static_cast<long long>(history_len) + n_tokens;
  p.row_tiles = static_cast<int>((rows + 127) / 128);
  p.key_tiles = static_cast<int>((keys + 127) / 128);
  long long most[2] = {0, 0};
  for (long long t = 0; t < p.row_tiles; ++t) {
    const long long n = (history_len + std::min(128 * t + 127, rows - 1) / G) / 128 + 1;
    p.line[0] += n;
    most[0] = std::max(most[0], n);
  }
  for (long long t = 0; t < p.key_tiles; ++t) {
    const long long n = p.row_tiles - std::max(0LL, 128 * t - history_len) * G / 128;
    p.line[1] += n;
    most[1] = std::max(most[1], n);
  }
  for (int i = 0; i < 2; ++i) {
    const long long total = p.line[i] * n_kv_heads;
    p.runs[i] = static_cast<int>(std::min<long long>(total, n_sms));
    // an A tile of n pairs lies in at most ceil(n / floor(total / runs)) + 1 runs, and in no more than there are
    const long long shortest = total / p.runs[i];
    p.n_seg[i] = static_cast<int>(std::min<long long>(p.runs[i], (most[i] + shortest - 1) / shortest + 1));
  }
  auto round = [](long long x) { return (x + 255) / 256 * 256; };
  const long long row_n = static_cast<long long>(n_kv_heads) * p.row_tiles * 128;
  const long long key_n = static_cast<long long>(n_kv_heads) * p.key_tiles * 128;
  p.off_nm = round(row_n * p.n_seg[0] * 2 * 8);
  p.off_il = p.off_nm + round(row_n * 4);
  p.off_col = p.off_il + round(row_n * 4);
  p.bytes = p.off_col + key_n * p.n_seg[1] * 2 * 4;
  return p;
}

template <int D>
static cudaError_t launch_chunk_weights_d(const ChunkWeightsArgs& a, cudaStream_t stream) {
  using L = CwSmem<D>;
  cudaError_t e = cudaFuncSetAttribute(chunk_weights_kernel<D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(chunk_weights_kernel<D, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  const dim3 block(kCwThreads);
  if ((e = launch_pdl(chunk_weights_kernel<D, 1>, dim3(a.runs[0]), block, L::kAlloc, stream, a)) != cudaSuccess) return e;
  if ((e = launch_pdl(chunk_rows_kernel, dim3(a.row_tiles, a.n_kv_heads), dim3(128), 0, stream, a)) != cudaSuccess) return e;
  if ((e = launch_pdl(chunk_weights_kernel<D, 2>, dim3(a.runs[1]), block, L::kAlloc, stream, a)) != cudaSuccess) return e;
  return launch_pdl(chunk_acc_kernel, dim3(a.key_tiles, a.n_kv_heads), dim3(128), 0, stream, a);
}

cudaError_t launch_chunk_weights(const ChunkWeightsArgs& a, cudaStream_t stream) {
  return a.head_dim == 256 ? launch_chunk_weights_d<256>(a, stream) : launch_chunk_weights_d<128>(a, stream);
}

}  // namespace kvq
