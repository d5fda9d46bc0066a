// prefill_window.cu — attention of a chunk of prompt queries over the int8 paged K/V cache, with a sliding window and
// first tokens that stay visible.
//
// Query i (position p = history + i) sees the keys t <= p with t > p - W or t < S.  For a row (i, h) with scores in log2 units
// s[t] = softmax_scale log2(e) q . (k_code[t] k_scale[t]):
//     out = sum_t 2^s[t] v_scale[t] v_code[t] / sum_t 2^s[t].
// The V scale goes into the exponent: z[t] = s[t] + log2 v_scale[t], w[t] = 2^(z[t] - r) with one reference r a row, so that
//     out = sum_t w[t] v_code[t] / sum_t w[t] / v_scale[t],
// one exponential a score, weights that fit fp16 whatever the V scales are, and no second maximum.  r is the largest z
// of the row's first tile and moves only when a tile exceeds it by 2^8, so that the accumulator is hardly ever scaled again.
//
// Operands.  Codes are exact in 16-bit floats: the scores take the bf16 queries as they are and the K codes in bf16
// (every product exact, fp32 sums); the weights go in as fp16, rounded to 11 bits (2^-11 relative: the one rounding
// before the output's), against V codes in fp16.  A pass before the attention widens the tiles of 128 keys that any
// row sees, once for all row tiles and heads, into the byte image of the operands, and leaves each key's factors.
//
// Rows.  The rows of a KV head are r = i G + g (G heads a group): a tile of 128 rows is a run of 128 / G queries, so that
// it sees little more than a window of keys, all its heads share each K/V tile, and a short chunk fills tiles.
//
// Schedule.  The (row tile, key tile) pairs of all KV heads are one line, cut into equal runs, one a CTA and a CTA an SM.
// A row tile that two runs share leaves a part each (reference, sum, numerator) and a last launch joins the parts in
// the order of the line, so that the same call gives the same bits; one that lies within a run is written at once.
//
// A CTA's warps:
//   warps 0-7  softmax: thread = (row, half of the tile's keys); lanes 32 (w % 4) .. of tensor memory
//   warp 8     MMA issue and tensor-memory allocation
//   warp 9     tile copies: a ring of 16 KB pieces in the order the MMAs take them, and the keys' factors
// Tensor memory: S (128 columns) | P, two buffers of 64 | O (head_dim) | at head_dim 128 also Q (64).  S is one
// buffer: its threads hold it in registers and free it before they work on it, so that the next Q K^T runs meanwhile.
// P in tensor memory leaves the shared memory to the K/V tiles (and at head_dim 256 to Q).
#include <algorithm>

#include "kvq_dev.cuh"
#include "kvq_launch.h"
#include "tcgen05.cuh"
#include "tile_dev.cuh"

namespace kvq {

namespace {

constexpr int kWSoftWarps = 8, kWSoftThreads = 32 * kWSoftWarps, kWMmaWarp = kWSoftWarps;
constexpr int kWThreads = kWSoftThreads + 64;
constexpr int kWParBufs = 4;
constexpr float kWLazy = 8.0f;  // a tile may exceed its row's reference by 2^8
// V scales below this count as this: their codes' share of an output, at most 127 * 2^-100, is lost in any other
constexpr float kWMinScale = 7.8886091e-31f;  // 2^-100

template <int D>
struct Pw {
  static constexpr bool kQTmem = D == 128;
  static constexpr int kSlots = D == 256 ? 8 : 10;           // pieces in the ring
  static constexpr int kStageBytes = 128 * D * 2;            // the output tile in bf16; at head_dim 256 Q's place
  static constexpr int offRing = kStageBytes;
  static constexpr int offPar = offRing + kSlots * kPieceBytes;  // [buf][3][128] fp32
  static constexpr int offRed = offPar + kWParBufs * 3 * 128 * 4;  // [2][part][128] fp32
  static constexpr int offBar = offRed + 2 * 2 * 128 * 4;
  // barriers
  static constexpr int full = 0, empty = full + kSlots, parFull = empty + kSlots, parFree = parFull + kWParBufs,
                       sFull = parFree + kWParBufs, sFree = sFull + 1, pFull = sFree + 1, pvDone = pFull + 2,
                       qFull = pvDone + 2, oFree = qFull + 1, drain = oFree + 1, kNumBars = drain + 1;
  static constexpr int offFlag = offBar + kNumBars * 8;      // abort flag, TMEM base
  static constexpr int kAlloc = offFlag + 16 + 1024;
  static constexpr uint32_t kPCol = 128, kOCol = 256, kQCol = kOCol + 128, kTmemCols = 512;
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

// A barrier of COUNT threads that gives them all the OR of `pred`: they take the same way.
template <int COUNT>
__device__ __forceinline__ bool bar_or(int id, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, %3, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "r"(id), "n"(COUNT)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void soft_bar() { asm volatile("bar.sync 5, %0;" ::"n"(kWSoftThreads) : "memory"); }

}  // namespace

// Key tiles of row tile t of a KV head: sink tiles [0, sink), then tiles [low, low + n - sink).
struct RowTileKeys {
  int sink, low, n;
};
__host__ __device__ inline RowTileKeys row_tile_keys(int t, int n_rows, int group, int history, int window, int n_sink) {
  const int last = 128 * t + 127 < n_rows - 1 ? 128 * t + 127 : n_rows - 1;
  const int p_lo = history + 128 * t / group, p_hi = history + last / group;
  RowTileKeys r;
  r.low = p_lo - window + 1 > 0 ? (p_lo - window + 1) / 128 : 0;
  const int sink = n_sink / 128 + (n_sink % 128 != 0);
  r.sink = sink < r.low ? sink : r.low;
  r.n = r.sink + p_hi / 128 - r.low + 1;
  return r;
}

// Place on the line: KV head, row tile, key tile x of its n.
struct WindowWalk {
  int kvh, t, x;
  RowTileKeys keys;
  __device__ int tile() const { return x < keys.sink ? x : x - keys.sink + keys.low; }  // of the sequence
};
__device__ __forceinline__ RowTileKeys keys_of(const PrefillWindowArgs& a, int t) {
  return row_tile_keys(t, a.n_rows, a.group, a.history_len, a.window, a.n_sink);
}
__device__ __forceinline__ int stored_tile(const PrefillWindowArgs& a, int tile) {
  return tile < a.sink_tiles ? tile : tile - a.first_tile + a.sink_tiles;
}

// The pair at f: a warp-wide search of the prefix sums of the row tiles' counts.
__device__ __forceinline__ WindowWalk window_walk_at(const PrefillWindowArgs& a, long long f) {
  const int lane = threadIdx.x & 31;
  WindowWalk w;
  w.kvh = static_cast<int>(f / a.line);
  long long rem = f - w.kvh * a.line;
  w.t = w.x = 0;
  for (int base = 0; base < a.row_tiles; base += 32) {
    const int n = base + lane < a.row_tiles ? keys_of(a, base + lane).n : 0;
    long long incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    const long long total = __shfl_sync(0xffffffffu, incl, 31);
    if (rem < total) {
      const int l = __ffs(__ballot_sync(0xffffffffu, incl > rem)) - 1;
      w.t = base + l;
      w.x = static_cast<int>(rem - (__shfl_sync(0xffffffffu, incl, l) - __shfl_sync(0xffffffffu, n, l)));
      break;
    }
    rem -= total;
  }
  w.keys = keys_of(a, w.t);
  return w;
}
__device__ __forceinline__ void window_step(const PrefillWindowArgs& a, WindowWalk& w) {
  if (++w.x < w.keys.n) return;
  w.x = 0;
  if (++w.t == a.row_tiles) {
    w.t = 0;
    ++w.kvh;
  }
  w.keys = keys_of(a, w.t);
}
__device__ __forceinline__ long long run_start(const PrefillWindowArgs& a, int c, int runs) {
  return a.line * a.n_kv_heads * c / runs;
}

// ============================================================================ operand tiles
// One CTA per (stored tile, KV head): K codes to bf16, rows = keys, piece a = dims 64 a ..; V codes to fp16, rows = dims,
// piece kh (D / 128) + dh = keys 64 kh .. of dims 128 dh .. (the layouts of the prefill's operands); each key's factors.
// Pages that no row sees are not looked at.
template <int D>
__global__ void __launch_bounds__(256) window_tiles_kernel(const __grid_constant__ PrefillWindowArgs a) {
  const int kvh = blockIdx.y, tid = threadIdx.x;
  const int st = blockIdx.x, tile = st < a.sink_tiles ? st : st - a.sink_tiles + a.first_tile;
  __shared__ int page_s[8];
  grid_dep_wait();
  grid_dep_trigger();
  if (tid < 8) {
    const int key0 = 128 * tile + 16 * tid;
    int page = -1;
    if (key0 < a.n_keys && (key0 + 15 >= a.history_len - a.window + 1 || key0 < a.n_sink)) {
      page = a.block_table_row[key0 / KVQ_BLOCK_SIZE];
      if (page < 0 || page >= a.num_blocks) {
        set_status(a.status, KVQ_DEV_BAD_BLOCK);
        page = -1;
      }
    }
    page_s[tid] = page;
  }
  __syncthreads();
  const long long u = static_cast<long long>(kvh) * a.key_tiles + st;
  uint8_t* kdst = a.k_tiles + u * (D * 256);
  uint8_t* vdst = a.v_tiles + u * (D * 256);
  uint4 raw[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {  // four adjacent lanes fill one 128-byte row of a piece
    const int i = tid + 256 * x, n = (i >> 2) & 127, c16 = ((i >> 9) << 2) | (i & 3), page = page_s[n >> 4];
    raw[x] = make_uint4(0, 0, 0, 0);
    if (page >= 0 && 128 * tile + n < a.n_keys)
      raw[x] = __ldg(reinterpret_cast<const uint4*>(
          a.k + ((static_cast<long long>(page) * a.n_kv_heads + kvh) * (D / 16) + c16) * 256 + (n & 15) * 16));
  }
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {
    const int i = tid + 256 * x, n = (i >> 2) & 127, c16 = ((i >> 9) << 2) | (i & 3);
    uint32_t h[8];
    widen16_bf16(raw[x], h);
    uint8_t* piece = kdst + (c16 >> 2) * kPieceBytes;
    const int cc = (c16 & 3) * 2;
    sts128(piece + tc::sw128_off(n, cc), make_uint4(h[0], h[1], h[2], h[3]));  // global stores
    sts128(piece + tc::sw128_off(n, cc + 1), make_uint4(h[4], h[5], h[6], h[7]));
  }
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {
    const int i = tid + 256 * x, pl = ((i / (4 * D)) << 2) | (i & 3), d = (i >> 2) % D, page = page_s[pl];
    raw[x] = make_uint4(0, 0, 0, 0);
    if (page >= 0)
      raw[x] = __ldg(reinterpret_cast<const uint4*>(
          a.v + ((static_cast<long long>(page) * a.n_kv_heads + kvh) * D + d) * KVQ_BLOCK_SIZE));
  }
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {
    const int i = tid + 256 * x, pl = ((i / (4 * D)) << 2) | (i & 3), d = (i >> 2) % D;
    uint4 c0, c1;
    widen16(make_int4(raw[x].x, raw[x].y, raw[x].z, raw[x].w), c0, c1);
    uint8_t* piece = vdst + ((pl >> 2) * (D / 128) + (d >> 7)) * kPieceBytes;
    const int cc = (pl & 3) * 2;
    sts128(piece + tc::sw128_off(d & 127, cc), c0);
    sts128(piece + tc::sw128_off(d & 127, cc + 1), c1);
  }
  if (tid < 128) {
    const int page = page_s[tid >> 4];
    float kf = 0.f, lv = -INFINITY, iv = 0.f;  // a key that is not there: weight 0
    if (page >= 0 && 128 * tile + tid < a.n_keys) {
      const long long at = (static_cast<long long>(page) * a.n_kv_heads + kvh) * KVQ_BLOCK_SIZE + (tid & 15);
      kf = a.k_scale[at] * a.c2;
      float vs = a.v_scale[at];
      if (vs < kWMinScale) vs = kWMinScale;
      lv = log2f(vs);
      iv = 1.0f / vs;
    }
    float* par = a.par + u * 384;
    par[tid] = kf;
    par[128 + tid] = lv;
    par[256 + tid] = iv;
  }
}

// ============================================================================ attention
template <int D>
__global__ void __launch_bounds__(kWThreads, 1) window_attention_kernel(const __grid_constant__ PrefillWindowArgs a) {
  using L = Pw<D>;
  constexpr int NP = D / 64, OC = D / 2;  // pieces of a K or V tile; O columns of a softmax thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint8_t* stage = sm;
  uint8_t* ring = sm + L::offRing;
  float* par = reinterpret_cast<float*>(sm + L::offPar);
  float* red = reinterpret_cast<float*>(sm + L::offRed);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::offBar);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::offFlag);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::offFlag + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int runs = static_cast<int>(gridDim.x), run = static_cast<int>(blockIdx.x);
  const long long f0 = run_start(a, run, runs);
  const int n_tiles = static_cast<int>(run_start(a, run + 1, runs) - f0);
  WindowWalk w = window_walk_at(a, f0);

  if (warp == kWMmaWarp) tc::tmem_alloc(tmem_slot, L::kTmemCols);
  if (tid == 0) {
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(&bars[L::full + s], 1);
      mbar_init(&bars[L::empty + s], 1);
    }
    for (int s = 0; s < kWParBufs; ++s) {
      mbar_init(&bars[L::parFull + s], 1);
      mbar_init(&bars[L::parFree + s], kWSoftWarps);
    }
    mbar_init(&bars[L::sFull], 1);
    mbar_init(&bars[L::sFree], kWSoftWarps);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[L::pFull + s], kWSoftWarps);
      mbar_init(&bars[L::pvDone + s], 1);
    }
    mbar_init(&bars[L::qFull], kWSoftWarps);
    mbar_init(&bars[L::oFree], kWSoftWarps);
    mbar_init(&bars[L::drain], 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();  // the tiles come from the kernel before
  grid_dep_trigger();

  if (warp < kWSoftWarps) {
    // ================================================================ softmax warps
    const int row = (warp & 3) * 32 + lane, part = warp >> 2, gbar = 1 + (warp & 3);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tm_o = tmem + lane_base + L::kOCol + part * OC;
    const uint32_t tm_p = tmem + lane_base + L::kPCol + part * 32;
    bool failed = false;
    float2* ml = a.part_ml + static_cast<long long>(run) * 256;
    if (part == 0) {  // until they are written: dropped
      ml[row] = make_float2(-INFINITY, -1.0f);
      ml[128 + row] = make_float2(-INFINITY, -1.0f);
    }
    int f = 0;
    while (f < n_tiles) {
      // ---- a unit: the key tiles of row tile w.t that belong to this run
      const bool first_of_run = f == 0, from_start = w.x == 0;
      const int n_unit = min(w.keys.n - w.x, n_tiles - f);
      const bool to_end = w.x + n_unit == w.keys.n;
      const int r = 128 * w.t + row, qi = r / a.group;
      const int pos = a.history_len + qi;
      const int last_row = a.n_rows - 128 * w.t;  // rows of this tile: row < last_row
      // ---- Q
      if constexpr (L::kQTmem) {
        uint32_t qw[32];  // this thread's 64 dims
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) +
            (static_cast<long long>(qi) * a.n_q_heads + w.kvh * a.group + (r - qi * a.group)) * D + part * 64);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = row < last_row ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
          qw[4 * i] = v.x;
          qw[4 * i + 1] = v.y;
          qw[4 * i + 2] = v.z;
          qw[4 * i + 3] = v.w;
        }
        tc::st_32x32b_x32(tmem + lane_base + L::kQCol + part * 32, qw);
        tc::wait_st();
      } else {
        // a warp takes 16 rows, a row at a time: lane = 16-byte chunk
        uint4 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int n = warp * 16 + i, rr = 128 * w.t + n, q2 = rr / a.group;
          v[i] = make_uint4(0, 0, 0, 0);
          if (n < last_row)
            v[i] = __ldg(reinterpret_cast<const uint4*>(
                             static_cast<const uint16_t*>(a.q) +
                             (static_cast<long long>(q2) * a.n_q_heads + w.kvh * a.group + (rr - q2 * a.group)) * D) + lane);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sts128(stage + (lane >> 3) * kPieceBytes + tc::sw128_off(warp * 16 + i, lane & 7), v[i]);
        tc::fence_proxy_async_smem();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::qFull]);

      float ref = -INFINITY, l = 0.0f;
      for (int j = 0; j < n_unit; ++j, ++f) {
        const int b = f & 1, pb = f % kWParBufs;
        const int k0 = 128 * w.tile();
        failed |= !wait_or_abort(&bars[L::sFull], f & 1, a.status, abort_flag, a.wait_budget);
        tc::fence_after_sync();
        uint32_t s0[32], s1[32];
        tc::ld_32x32b_x32(tmem + lane_base + 64 * part, s0);
        tc::ld_32x32b_x32(tmem + lane_base + 64 * part + 32, s1);
        failed |= !wait_or_abort(&bars[L::parFull + pb], (f / kWParBufs) & 1, a.status, abort_flag, a.wait_budget);
        tc::wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::sFree]);
        const float4* kf = reinterpret_cast<const float4*>(par + pb * 384 + 64 * part);
        const float4* lv = kf + 32;
        const float4* iv = kf + 64;
        f2 z[32];
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const float4 k4 = kf[n], l4 = lv[n];
          const uint32_t* s = n < 8 ? s0 + 4 * n : s1 + 4 * (n - 8);
          z[2 * n] = fma2(mk2(__uint_as_float(s[0]), __uint_as_float(s[1])), mk2(k4.x, k4.y), mk2(l4.x, l4.y));
          z[2 * n + 1] = fma2(mk2(__uint_as_float(s[2]), __uint_as_float(s[3])), mk2(k4.z, k4.w), mk2(l4.z, l4.w));
          m0 = fmax3(m0, lo2(z[2 * n]), hi2(z[2 * n]));
          m1 = fmax3(m1, lo2(z[2 * n + 1]), hi2(z[2 * n + 1]));
        }
        // keys of this thread's half that the row sees: n < hi, and n >= lo or n < sk
        const int kk = k0 + 64 * part, hi = pos + 1 - kk, lo = pos - a.window + 1 - kk, sk = a.n_sink - kk;
        const bool whole = hi >= 64 && (lo <= 0 || sk >= 64);
        if (!whole) {
          m0 = m1 = -INFINITY;
#pragma unroll
          for (int n = 0; n < 32; ++n) {
            const bool v0 = 2 * n < hi && (2 * n >= lo || 2 * n < sk);
            const bool v1 = 2 * n + 1 < hi && (2 * n + 1 >= lo || 2 * n + 1 < sk);
            z[n] = mk2(v0 ? lo2(z[n]) : -INFINITY, v1 ? hi2(z[n]) : -INFINITY);
            m0 = fmax3(m0, lo2(z[n]), hi2(z[n]));
          }
        }
        red[(b * 2 + part) * 128 + row] = fmaxf(m0, m1);
        if (bar_or<64>(gbar, failed)) break;  // both halves of these rows leave together
        const float m = fmaxf(red[b * 256 + row], red[b * 256 + 128 + row]);
        float scale = 1.0f;
        if (j == 0) {
          ref = m;
        } else if (m > ref + kWLazy) {
          scale = ref == -INFINITY ? 0.0f : fast_exp2(ref - m);
          l *= scale;
          ref = m;
        }
        const float nr = ref == -INFINITY ? 0.0f : -ref;
        const f2 nr2 = mk2(nr, nr);
        uint32_t p[32];
        f2 la = mk2(0.f, 0.f), lb = mk2(0.f, 0.f);
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const float4 i4 = iv[n];
          const f2 xa = add2(z[2 * n], nr2), xb = add2(z[2 * n + 1], nr2);
          const f2 wa = mk2(fast_exp2(lo2(xa)), fast_exp2(hi2(xa))), wb = mk2(fast_exp2(lo2(xb)), fast_exp2(hi2(xb)));
          p[2 * n] = pack_half2(lo2(wa), hi2(wa));
          p[2 * n + 1] = pack_half2(lo2(wb), hi2(wb));
          f2 ia = mk2(i4.x, i4.y), ib = mk2(i4.z, i4.w);
          if (!whole) {  // a hidden key may have any scale
            ia = mk2(lo2(wa) == 0.f ? 0.f : i4.x, hi2(wa) == 0.f ? 0.f : i4.y);
            ib = mk2(lo2(wb) == 0.f ? 0.f : i4.z, hi2(wb) == 0.f ? 0.f : i4.w);
          }
          la = fma2(wa, ia, la);
          lb = fma2(wb, ib, lb);
        }
        const f2 ls = add2(la, lb);
        l += lo2(ls) + hi2(ls);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::parFree + pb]);
        // this buffer of P was read by the product of tile f - 2
        if (f >= 2) failed |= !wait_or_abort(&bars[L::pvDone + b], ((f >> 1) - 1) & 1, a.status, abort_flag, a.wait_budget);
        if (__any_sync(0xffffffffu, scale != 1.0f)) {
          // O holds the products up to tile f - 1 (of this unit: j > 0)
          failed |= !wait_or_abort(&bars[L::pvDone + (b ^ 1)], ((f - 1) >> 1) & 1, a.status, abort_flag, a.wait_budget);
          tc::fence_after_sync();
          const f2 sc2 = mk2(scale, scale);
#pragma unroll 1
          for (int c = 0; c < OC / 32; ++c) {
            uint32_t o[32];
            tc::ld_32x32b_x32(tm_o + 32 * c, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const f2 x = mul2(mk2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), sc2);
              o[e] = __float_as_uint(lo2(x));
              o[e + 1] = __float_as_uint(hi2(x));
            }
            tc::st_32x32b_x32(tm_o + 32 * c, o);
          }
        }
        tc::fence_after_sync();
        tc::st_32x32b_x32(tm_p + b * 64, p);
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::pFull + b]);
        if (j + 1 < n_unit) window_step(a, w);
      }
      if (!failed)
        failed = !wait_or_abort(&bars[L::pvDone + ((f - 1) & 1)], ((f - 1) >> 1) & 1, a.status, abort_flag, a.wait_budget);
      tc::fence_after_sync();
      red[part * 128 + row] = l;
      if (bar_or<kWSoftThreads>(5, failed)) break;  // all softmax warps leave together
      l = red[row] + red[128 + row];
      if (from_start && to_end) {
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        const int h = w.kvh * a.group + (r - qi * a.group);
        if (a.out_bf16) {
          // through shared memory, 16-byte chunk c of a row at c ^ (row % 8); Q's place is free, the unit's products done
#pragma unroll 1
          for (int c = 0; c < OC / 32; ++c) {
            uint32_t o[32];
            tc::ld_32x32b_x32(tm_o + 32 * c, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t hw[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(o[8 * e + 2 * y]) * inv,
                                                               __uint_as_float(o[8 * e + 2 * y + 1]) * inv);
                hw[y] = *reinterpret_cast<const uint32_t*>(&x);
              }
              const int chunk = part * (OC / 8) + 4 * c + e;
              sts128(stage + row * (2 * D) + ((chunk ^ (row & 7)) << 4), make_uint4(hw[0], hw[1], hw[2], hw[3]));
            }
          }
          tc::fence_before_sync();
          soft_bar();
          if (lane == 0) mbar_arrive(&bars[L::oFree]);
          constexpr int PER = 256 / D;  // rows a warp copies at a time (D / 8 chunks each)
#pragma unroll
          for (int i = 0; i < 16 / PER; ++i) {
            const int n = warp * 16 + i * PER + lane / (D / 8), chunk = lane % (D / 8);
            if (n < last_row) {
              const int rr = 128 * w.t + n, q2 = rr / a.group;
              reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                       (static_cast<long long>(q2) * a.n_q_heads + w.kvh * a.group + (rr - q2 * a.group)) * D)[chunk] =
                  *reinterpret_cast<const uint4*>(stage + n * (2 * D) + ((chunk ^ (n & 7)) << 4));
            }
          }
          soft_bar();  // the stage is read before the next unit's Q takes its place
        } else {
          float* dst = static_cast<float*>(a.out) + (static_cast<long long>(qi) * a.n_q_heads + h) * D + part * OC;
#pragma unroll 1
          for (int c = 0; c < OC / 32; ++c) {
            uint32_t o[32];
            tc::ld_32x32b_x32(tm_o + 32 * c, o);
            tc::wait_ld();
            if (row < last_row) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(dst + 32 * c + e) =
                    make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            }
          }
          tc::fence_before_sync();
          soft_bar();
          if (lane == 0) mbar_arrive(&bars[L::oFree]);
        }
      } else {
        // a part: the numerator four columns of all rows at a time
        const int slot = 2 * run + (first_of_run ? 0 : 1);
        float4* dst = a.part + (static_cast<long long>(slot) * (D / 4) + part * (OC / 4)) * 128 + row;
#pragma unroll 1
        for (int c = 0; c < OC / 32; ++c) {
          uint32_t o[32];
          tc::ld_32x32b_x32(tm_o + 32 * c, o);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[(8 * c + e) * 128] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                 __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        }
        if (part == 0) ml[(slot & 1) * 128 + row] = make_float2(ref, l);
        tc::fence_before_sync();
        soft_bar();
        if (lane == 0) mbar_arrive(&bars[L::oFree]);
      }
      window_step(a, w);
    }
  } else if (warp == kWMmaWarp) {
    // ================================================================ MMA issue
    const uint64_t qd0 = tc::sdesc_sw128(smem_u32(stage)), rd0 = tc::sdesc_sw128(smem_u32(ring));
    constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(128, 128), idesc_pv = tc::idesc_f16_f32(128, D);
    int slot = 0, unit = 0;
    uint32_t ph = 0;
    bool ok = true;
    auto await = [&](int bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, wait_or_abort(&bars[bar], parity, a.status, abort_flag, a.wait_budget));
      return ok;
    };
    auto next_slot = [&]() {
      if (++slot == L::kSlots) {
        slot = 0;
        ph ^= 1u;
      }
    };
    auto scores = [&](int f, bool first) {  // S = Q K_f^T
      if (first && !await(L::qFull, unit & 1)) return;
      if (f >= 1 && !await(L::sFree, (f - 1) & 1)) return;
      for (int qa = 0; qa < NP; ++qa) {
        if (!await(L::full + slot, ph)) return;
        if (elect_one()) {
          tc::fence_after_sync();
          const uint64_t kd = rd0 + static_cast<uint64_t>((slot * kPieceBytes) >> 4);
          const uint64_t qd = qd0 + static_cast<uint64_t>((qa * kPieceBytes) >> 4);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if constexpr (L::kQTmem)
              tc::mma_f16_ts(tmem, tmem + L::kQCol + 32 * qa + 8 * s, kd + 2 * s, idesc_qk, (qa | s) ? 1u : 0u);
            else
              tc::mma_f16_ss(tmem, qd + 2 * s, kd + 2 * s, idesc_qk, (qa | s) ? 1u : 0u);
          }
          tc::commit(&bars[L::empty + slot]);
          if (qa == NP - 1) tc::commit(&bars[L::sFull]);
        }
        __syncwarp();
        next_slot();
      }
    };
    auto values = [&](int f, bool first, int of_unit) {  // O (+)= P_f V_f
      const int b = f & 1;
      if (!await(L::pFull + b, (f >> 1) & 1)) return;
      if (first && of_unit > 0 && !await(L::oFree, (of_unit - 1) & 1)) return;
      for (int kh = 0; kh < 2; ++kh) {
        const int s0 = slot;
        for (int dh = 0; dh < D / 128; ++dh) {
          if (!await(L::full + slot, ph)) return;
          next_slot();
        }
        if (elect_one()) {
          tc::fence_after_sync();
          const uint64_t vd = rd0 + static_cast<uint64_t>((s0 * kPieceBytes) >> 4);
#pragma unroll
          for (int s = 0; s < 4; ++s)
            tc::mma_f16_ts(tmem + L::kOCol, tmem + L::kPCol + 64 * b + 32 * kh + 8 * s, vd + 2 * s, idesc_pv,
                           (first && kh == 0 && s == 0) ? 0u : 1u);
#pragma unroll
          for (int dh = 0; dh < D / 128; ++dh) tc::commit(&bars[L::empty + s0 + dh]);
          if (kh == 1) tc::commit(&bars[L::pvDone + b]);
        }
        __syncwarp();
      }
    };
    // Q K^T runs a tile ahead of P V within a unit; at a unit's end P V comes first (the next Q waits for it)
    bool was_first = false;
    for (int f = 0; ok && f < n_tiles; ++f) {
      const bool first = f == 0 || w.x == 0;
      if (first && f > 0) {
        values(f - 1, was_first, unit);
        if (!ok) break;
        ++unit;
      }
      scores(f, first);
      if (!ok) break;
      if (!first) values(f - 1, was_first, unit);
      was_first = first;
      window_step(a, w);
    }
    if (ok) values(n_tiles - 1, was_first, unit);
    // every MMA this warp issued has completed before the CTA releases tensor memory
    if (elect_one()) {
      tc::commit(&bars[L::drain]);
      mbar_wait(&bars[L::drain], 0, a.status, a.wait_budget);
    }
    __syncwarp();
  } else {
    // ================================================================ tile copies
    int slot = 0, fills = 0, par_fills = 0;
    uint32_t ph = 0;
    bool ok = true;
    const bool skip_one = a.fault == 5 && blockIdx.x == 0;  // test-only: the fourth piece is never copied
    if (lane == 0) {
      auto push = [&](const uint8_t* src) {
        for (int i = 0; i < NP; ++i) {
          if (fills >= L::kSlots && !wait_or_abort(&bars[L::empty + slot], ph ^ 1u, a.status, abort_flag, a.wait_budget)) {
            ok = false;
            return;
          }
          if (!(skip_one && fills == 3)) {
            mbar_arrive_expect_tx(&bars[L::full + slot], kPieceBytes);
            bulk_g2s(ring + slot * kPieceBytes, src + i * kPieceBytes, kPieceBytes, &bars[L::full + slot]);
          }
          ++fills;
          if (++slot == L::kSlots) {
            slot = 0;
            ph ^= 1u;
          }
        }
      };
      auto push_par = [&](long long u) {
        const int pb = par_fills % kWParBufs;
        if (par_fills >= kWParBufs &&
            !wait_or_abort(&bars[L::parFree + pb], (par_fills / kWParBufs - 1) & 1, a.status, abort_flag, a.wait_budget)) {
          ok = false;
          return;
        }
        mbar_arrive_expect_tx(&bars[L::parFull + pb], 1536);
        bulk_g2s(par + pb * 384, a.par + u * 384, 1536, &bars[L::parFull + pb]);
        ++par_fills;
      };
      long long before = 0;
      for (int f = 0; ok && f < n_tiles; ++f) {
        const bool first = f == 0 || w.x == 0;
        const long long u = static_cast<long long>(w.kvh) * a.key_tiles + stored_tile(a, w.tile());
        if (first && f > 0) push(a.v_tiles + before * (D * 256));
        if (ok) push_par(u);
        if (ok) push(a.k_tiles + u * (D * 256));
        if (ok && !first) push(a.v_tiles + before * (D * 256));
        before = u;
        window_step(a, w);
      }
      if (ok) push(a.v_tiles + before * (D * 256));
      // copies still in flight (only after an abort) land before the CTA exits
      for (int i = max(0, fills - L::kSlots); i < fills; ++i)
        if (!(skip_one && i == 3))
          mbar_wait(&bars[L::full + i % L::kSlots], (i / L::kSlots) & 1, a.status, a.wait_budget);
      for (int i = max(0, par_fills - kWParBufs); i < par_fills; ++i)
        mbar_wait(&bars[L::parFull + i % kWParBufs], (i / kWParBufs) & 1, a.status, a.wait_budget);
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kWMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ============================================================================ joining the parts
// Block (run, 16 rows).  The run in which a cut row tile ends joins its parts, from the run in which it begins on.
constexpr int kJoinRows = 16;

template <int D>
__global__ void __launch_bounds__(256) window_join_kernel(const __grid_constant__ PrefillWindowArgs a, int runs) {
  grid_dep_wait();
  grid_dep_trigger();
  const int run = blockIdx.x;
  const long long f0 = run_start(a, run, runs), f1 = run_start(a, run + 1, runs);
  const WindowWalk w = window_walk_at(a, f0);
  if (w.x == 0 || f0 - w.x + w.keys.n > f1) return;
  const long long start = f0 - w.x;
  int first = run - 1;  // the run in which the row tile begins
  while (run_start(a, first, runs) > start) --first;
  const int first_slot = 2 * first + (run_start(a, first, runs) < start ? 1 : 0);
  // thread = (row, columns): rows of a warp's lanes side by side, as the parts lie
  const int row = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, r = 128 * w.t + row;
  if (r >= a.n_rows) return;
  float m = -INFINITY;
  bool dropped = false;
  for (int c = first; c <= run; ++c) {
    const float2 v = a.part_ml[static_cast<long long>(c == first ? first_slot : 2 * c) * 128 + row];
    m = fmaxf(m, v.x);
    dropped |= v.y < 0.0f;
  }
  if (dropped) return;
  const int qi = r / a.group, h = w.kvh * a.group + (r - qi * a.group);
  const long long at = (static_cast<long long>(qi) * a.n_q_heads + h) * D;
  float l = 0.0f;
  for (int c = first; c <= run; ++c) {
    const float2 v = a.part_ml[static_cast<long long>(c == first ? first_slot : 2 * c) * 128 + row];
    if (v.x != -INFINITY || v.y != 0.0f) l += v.y * (v.x == -INFINITY ? 1.0f : fast_exp2(v.x - m));
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  for (int c4 = threadIdx.x / kJoinRows; c4 < D / 4; c4 += 256 / kJoinRows) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = first; c <= run; ++c) {
      const long long slot = c == first ? first_slot : 2 * c;
      const float2 v = a.part_ml[slot * 128 + row];
      if (v.x == -INFINITY && v.y == 0.0f) continue;  // no key of this part is seen
      const float s = v.x == -INFINITY ? 1.0f : fast_exp2(v.x - m);
      const float4 x = a.part[(slot * (D / 4) + c4) * 128 + row];
      o.x = fmaf(x.x, s, o.x);
      o.y = fmaf(x.y, s, o.y);
      o.z = fmaf(x.z, s, o.z);
      o.w = fmaf(x.w, s, o.w);
    }
    if (a.out_bf16) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv), y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at + 4 * c4) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + 4 * c4) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
  }
}

// ============================================================================ host
// The most CTAs a call runs: more than any GPU the library is built for has SMs, so that the workspace's size does not
// depend on the GPU.
constexpr int kWMaxRuns = 160;

PrefillWindowPlan prefill_window_plan(int n_tokens, int n_q_heads, int n_kv_heads, int history_len, int window,
                                      int n_sink, int head_dim, int n_sms) {
  PrefillWindowPlan p{};
  const int group = n_q_heads / n_kv_heads, n_rows = n_tokens * group;
  p.row_tiles = (n_rows + 127) / 128;
  p.first_tile = std::max(0, history_len - window + 1) / 128;
  p.sink_tiles = std::min(n_sink / 128 + (n_sink % 128 != 0), p.first_tile);
  p.key_tiles = p.sink_tiles + (history_len + n_tokens - 1) / 128 - p.first_tile + 1;
  for (int t = 0; t < p.row_tiles; ++t) p.line += row_tile_keys(t, n_rows, group, history_len, window, n_sink).n;
  const long long pairs = p.line * n_kv_heads;
  p.runs = static_cast<int>(std::min<long long>(pairs, std::min(n_sms, kWMaxRuns)));
  const long long max_runs = std::min<long long>(pairs, kWMaxRuns), tiles = static_cast<long long>(n_kv_heads) * p.key_tiles;
  p.off_v = tiles * head_dim * 256;
  p.off_par = 2 * p.off_v;
  p.off_ml = p.off_par + tiles * 1536;
  p.off_part = p.off_ml + max_runs * 2 * 128 * 8;
  p.bytes = p.off_part + max_runs * 2 * 128 * head_dim * 4;
  return p;
}

template <int D>
static cudaError_t launch_prefill_window_d(const PrefillWindowArgs& a, int runs, cudaStream_t stream) {
  using L = Pw<D>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(window_attention_kernel<D>), L::kAlloc, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(window_tiles_kernel<D>, dim3(a.key_tiles, a.n_kv_heads), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(window_attention_kernel<D>, dim3(runs), dim3(kWThreads), L::kAlloc, stream, a);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(runs, 128 / kJoinRows);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_join_kernel<D>, a, runs);
}

cudaError_t launch_prefill_window(const PrefillWindowArgs& a, int head_dim, int runs, cudaStream_t stream) {
  return head_dim == 256 ? launch_prefill_window_d<256>(a, runs, stream) : launch_prefill_window_d<128>(a, runs, stream);
}

}  // namespace kvq
