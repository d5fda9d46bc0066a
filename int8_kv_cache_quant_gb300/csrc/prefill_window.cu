// prefill_window.cu — attention of a chunk of prompt queries over the int8 paged K/V cache, with a sliding window and
// first tokens that stay visible.
//
// Query i (position p = history + i) sees the keys t <= p with t > p - W or t < S.  For a row (i, h) with scores in log2 units
// s[t] = softmax_scale log2(e) q . (k_code[t] k_scale[t]):
//     out = sum_t 2^s[t] v_scale[t] v_code[t] / sum_t 2^s[t].
// The V scale goes into the exponent: z[t] = s[t] + log2 v_scale[t], w[t] = 2^(z[t] - r) with one reference r a row, so that
//     out = sum_t w[t] v_code[t] / sum_t w[t] / v_scale[t],
// one exponential a score, weights that fit fp16 whatever the V scales are, and no second maximum.  r is 7 less than the largest z
// of the row's first tile and moves only when a tile's z is more than 15 above it, so that the accumulator is hardly ever scaled
// again: a row's largest weight is between 2^7 and 2^15, within fp16's 2^16 and far from where its numbers become subnormal.
// The one statistic has a price.  Factors of two to the -126 and less are 0, in the sum too, where a weight stands for w / v_scale: a
// key whose V scale is 2^-k of another's is lost from 126 - k octaves below that one's score on.  So V scales count as 2^-60
// at least (rows of zeros have 0), and past 2^40 they are reported: between the two, a key that is lost has less than
// 2^-26 of the largest probability.  A second statistic, of the scores alone, would be a second exponential a score.
//
// Operands.  Codes are exact in 16-bit floats: the scores take the bf16 queries as they are and the K codes in bf16
// (every product exact, fp32 sums); the weights go in as fp16, rounded to 11 bits (2^-11 relative, or 2^-25 where they are
// below 2^-14, which is 2^-32 of a row's largest: the one rounding before the output's), against V codes in fp16.  A pass before the attention widens the tiles of 128 keys that any
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
//   warps 0-15   softmax: rows 32 (w % 4) .. of the tile (the lanes of tensor memory that the warp can reach), a quarter of
//                its keys
//   warp 16      MMA issue and tensor-memory allocation
//   warp 17      tile copies, a ring of half tiles in the order the MMAs take them, and the keys' factors
//   warps 18-19  the next row tile's queries, while the last tiles of this one are worked on
// Tensor memory: three score tiles of 128 columns (two at head_dim 256) and O.  P takes its score tile's place, so that shared
// memory is left to Q and the K/V tiles and the scores run two tiles ahead of the values (one at head_dim 256).
// A softmax thread holds four rows x 8 keys (tcgen05.ld.16x256b), not one row x 32: a row a thread would need all keys'
// factors in every thread.  The scores stay in registers from the maximum to the weights; whether a row's maximum exceeds its
// reference is one barrier of the row's four warps, and only then do they exchange maxima.
//
// What bounds it, and what it was measured at.  2048 queries behind 30720 keys, W = 4096, 24 / 4 heads of 256: 177 us (206 GFLOP:
// 1.16 PFLOP/s), the tensor cores busy for 60 % of the attention's 161 us.  A tile has 2048 cycles of products and takes 3660
// (86 tiles a CTA): its P waits for its scores and these for the values two tiles before, since O leaves tensor memory
// room for two score tiles; and its operands are 128 KB, whose copies from L2 weigh as well (half of the bytes, the rest
// zeros: 165 us against 179 in the same build).  2047 queries, W = 1024, 32 / 8 heads of 128: 58.1 us (30 GFLOP), 27.4
// tiles and 3.4 row tiles' ends a CTA: the softmax and those ends, about 5000 cycles each for the last values, the output and the
// next queries; half of the bytes is no faster there (60.9 against 58.9).  33 queries, 24 / 4 heads of 256: 17.5 us, three
// launches of latencies.
// Instruction fetch decides more than arithmetic here: 20 warps in six roles run from the same caches.  2047 queries, us:
// with a softmax tile unrolled twice 71 against 63; product and copy code in one place each instead of three 59 against 63;
// the queries' loop eight times unrolled 64, four times 62; the MMA warp's operands not provably uniform 69 against 63.
// Other shapes that were built and were slower, us (2047 queries | 32K chunk): eight softmax warps and one score tile
// 104 | 314; two groups of eight that take turns at the tiles 58.6 | 193; scores and values issued by two warps 81 | 238 against
// 74 | 220; pairs of CTAs that share an MMA (cta_group::2, each half of a tile's K and V) 70 | 235 against 64 | 197; parts
// joined by whoever writes the second 63 | 183 against 59 | 181.
#include <algorithm>

#include "kvq_dev.cuh"
#include "kvq_launch.h"
#include "tcgen05.cuh"
#include "tile_dev.cuh"

namespace kvq {

namespace {

constexpr int kWSoftWarps = 16, kWMmaWarp = kWSoftWarps, kWCopyWarp = kWMmaWarp + 1, kWQWarp = kWCopyWarp + 1, kWQWarps = 2;
constexpr int kWThreads = 32 * (kWQWarp + kWQWarps);
constexpr int kWParBufs = 4;
// A row's largest weight when its reference is set, and what a later tile's may come to before it moves, in octaves: within
// fp16's 2^16, and as far from where weights become subnormal, 2^-14, as that leaves.
constexpr float kWLift = 7.0f, kWMost = kWLift + 8.0f;
// The V scales that a weight and its sum take (above).
constexpr float kWMinScale = 0x1p-60f, kWMaxScale = 0x1p40f;

template <int D>
struct Pw {
  static constexpr int kHalf = D * 128;                      // bytes of half a K tile (of its dims) or V tile (of its keys)
  static constexpr int kTiles = D == 256 ? 2 : 5;            // K or V tiles in the ring
  static constexpr int kScoreBufs = D == 256 ? 2 : 3;        // score tiles
  static constexpr int kQBytes = 128 * D * 2;                // Q in pieces of 16 KB
  static constexpr int offRing = kQBytes;
  static constexpr int offPar = offRing + 2 * kTiles * kHalf;      // [buf][3][128] fp32
  static constexpr int offRed = offPar + kWParBufs * 3 * 128 * 4;  // [maximum, sum][quarter of the keys][128] a row's four warps
  static constexpr int offBar = offRed + 2 * 4 * 128 * 4;
  // barriers: of the ring's tiles, their halves, ..; a score buffer's tiles have theirs
  static constexpr int full = 0, empty = full + kTiles, parFull = empty + 2 * kTiles, parFree = parFull + kWParBufs,
                       sFull = parFree + kWParBufs, pFull = sFull + kScoreBufs, pvDone = pFull + kScoreBufs, qFull = pvDone + kScoreBufs,
                       qFree = qFull + 1, oFree = qFree + 1, drain = oFree + 1, kNumBars = drain + 1;
  static constexpr int offFlag = offBar + kNumBars * 8;      // abort flag, TMEM base
  static constexpr int kAlloc = offFlag + 16 + 1024;
  // Tensor memory: score tiles and O.  A P tile takes the first half of its score tile's place.
  static constexpr uint32_t kOCol = 128 * kScoreBufs, kTmemCols = 512;
  static_assert(kOCol + D <= kTmemCols, "tensor memory");
  static_assert(offBar % 8 == 0, "alignment");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

// A barrier of four warps that gives them the OR of `pred`: they take the same way.
__device__ __forceinline__ bool rows_or(int id, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
}

// 16 bytes to shared memory without passing through registers; zeros where `real` is false.
__device__ __forceinline__ void cp_async16(uint8_t* dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// wait_or_abort in few instructions, since a dozen copies of it stand in the loops: the CTA's end reports the timeout.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long budget) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (*abort_flag || clock64() - t0 > budget) {
      *abort_flag = 1;
      return false;
    }
  return true;
}

// x / d for x and d below 2^15, with inv = ceil(2^32 / d), or 0 for d = 1.
__device__ __forceinline__ int small_div(int x, uint32_t inv) {
  return inv ? static_cast<int>(__umulhi(static_cast<uint32_t>(x), inv)) : x;
}

// Four lanes (c = lane % 4) of four words each: word k of lane c becomes word c of lane k.
__device__ __forceinline__ void lanes4_transpose(int c, uint32_t (&p)[4]) {
#pragma unroll
  for (int b = 1; b < 4; b *= 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(i & b)) {
        const bool up = (c & b) != 0;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? p[i] : p[i | b], b);
        if (up) p[i] = got;
        else p[i | b] = got;
      }
  }
}

// The lowest min(max(n, 0), 32) bits.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return __funnelshift_rc(0xffffffffu, 0u, 32u - static_cast<uint32_t>(min(n, 32)));
}

// Row of a quadrant that register pair j of a thread's fragment belongs to (tcgen05.cuh, two loads of 16 lanes).
__device__ __forceinline__ int frag_row(int lane, int j) { return (j >> 1) * 16 + (j & 1) * 8 + (lane >> 2); }

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

// Whether the scores of tile fs, the x-th of its row tile, come before the values of tile f: a tile ahead, two with three score
// tiles, but none where they wait for new queries, since a row tile's result waits for the values.
template <int D>
__device__ __forceinline__ bool scores_next(int fs, int f, int n_tiles, int x) {
  return fs < n_tiles && fs < f + (x == 0 ? 1 : 2 + (Pw<D>::kScoreBufs > 2));
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
// Blocks (stored tile, KV head, quarter), two quarters for K and two for V: K codes to bf16, rows = keys, piece a = dims 64 a ..; V codes to fp16, rows = dims,
// piece kh (D / 128) + dh = keys 64 kh .. of dims 128 dh .. (the layouts of the prefill's operands); each key's factors.
// Pages that no row sees are not looked at.
template <int D>
__global__ void __launch_bounds__(256) window_tiles_kernel(const __grid_constant__ PrefillWindowArgs a) {
  const int kvh = blockIdx.y, tid = threadIdx.x;
  const int st = blockIdx.x, tile = st < a.sink_tiles ? st : st - a.sink_tiles + a.first_tile;
  __shared__ int page_s[8];
  // The wait stays ahead of the trigger: the attention kernel's query warps read q without a wait of their own, and what the
  // stream did before this launch is there by then only because every block of it has waited.
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
  constexpr int N = D / 64;  // 16-byte loads of a thread
  const int i0 = tid + 256 * N * (blockIdx.z & 1);
  uint4 raw[N];
  if (blockIdx.z < 2) {
#pragma unroll
    for (int x = 0; x < N; ++x) {  // four adjacent lanes fill one 128-byte row of a piece
      const int i = i0 + 256 * x, n = (i >> 2) & 127, c16 = ((i >> 9) << 2) | (i & 3), page = page_s[n >> 4];
      raw[x] = make_uint4(0, 0, 0, 0);
      if (page >= 0 && 128 * tile + n < a.n_keys)
        raw[x] = __ldg(reinterpret_cast<const uint4*>(
            a.k + ((static_cast<long long>(page) * a.n_kv_heads + kvh) * (D / 16) + c16) * 256 + (n & 15) * 16));
    }
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int i = i0 + 256 * x, n = (i >> 2) & 127, c16 = ((i >> 9) << 2) | (i & 3);
      uint32_t h[8];
      widen16_bf16(raw[x], h);
      uint8_t* piece = kdst + (c16 >> 2) * kPieceBytes;
      const int cc = (c16 & 3) * 2;
      sts128(piece + tc::sw128_off(n, cc), make_uint4(h[0], h[1], h[2], h[3]));  // global stores
      sts128(piece + tc::sw128_off(n, cc + 1), make_uint4(h[4], h[5], h[6], h[7]));
    }
    if (blockIdx.z == 1) return;
  } else {
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int i = i0 + 256 * x, pl = ((i / (4 * D)) << 2) | (i & 3), d = (i >> 2) % D, page = page_s[pl];
      raw[x] = make_uint4(0, 0, 0, 0);
      if (page >= 0)
        raw[x] = __ldg(reinterpret_cast<const uint4*>(
            a.v + ((static_cast<long long>(page) * a.n_kv_heads + kvh) * D + d) * KVQ_BLOCK_SIZE));
    }
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int i = i0 + 256 * x, pl = ((i / (4 * D)) << 2) | (i & 3), d = (i >> 2) % D;
      uint4 c0, c1;
      widen16(make_int4(raw[x].x, raw[x].y, raw[x].z, raw[x].w), c0, c1);
      uint8_t* piece = vdst + ((pl >> 2) * (D / 128) + (d >> 7)) * kPieceBytes;
      const int cc = (pl & 3) * 2;
      sts128(piece + tc::sw128_off(d & 127, cc), c0);
      sts128(piece + tc::sw128_off(d & 127, cc + 1), c1);
    }
    return;
  }
  if (tid < 128) {
    const int page = page_s[tid >> 4];
    float kf = 0.f, lv = -INFINITY, iv = 0.f;  // a key that is not there: weight 0
    if (page >= 0 && 128 * tile + tid < a.n_keys) {
      const long long at = (static_cast<long long>(page) * a.n_kv_heads + kvh) * KVQ_BLOCK_SIZE + (tid & 15);
      kf = a.k_scale[at] * a.c2;
      float vs = a.v_scale[at];
      const int key = 128 * tile + tid;
      if (vs > kWMaxScale && (key > a.history_len - a.window || key < a.n_sink)) set_status(a.status, KVQ_DEV_BAD_SCALE);
      if (vs < kWMinScale) vs = kWMinScale;
      lv = log2f(vs);
      // (finite: 0 times it is 0 for the rows that do not see the key; the others have its infinity or NaN from lv)
      iv = vs < INFINITY ? 1.0f / vs : 0.0f;
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint8_t* ring = sm + L::offRing;
  float* par = reinterpret_cast<float*>(sm + L::offPar);
  float* red = reinterpret_cast<float*>(sm + L::offRed);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::offBar);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::offFlag);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::offFlag + 4);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (the same in its lanes, for the compiler too)
  const int runs = static_cast<int>(gridDim.x), run = static_cast<int>(blockIdx.x);
  const long long f0 = run_start(a, run, runs);
  const int n_tiles = static_cast<int>(run_start(a, run + 1, runs) - f0);
  WindowWalk w = window_walk_at(a, f0);

  if (warp == kWMmaWarp) tc::tmem_alloc(tmem_slot, L::kTmemCols);
  if (tid == 0) {
    for (int s = 0; s < L::kTiles; ++s) mbar_init(&bars[L::full + s], 2);
    for (int s = 0; s < 2 * L::kTiles; ++s) mbar_init(&bars[L::empty + s], 1);
    for (int s = 0; s < kWParBufs; ++s) {
      mbar_init(&bars[L::parFull + s], 1);
      mbar_init(&bars[L::parFree + s], kWSoftWarps);
    }
    for (int s = 0; s < L::kScoreBufs; ++s) {
      mbar_init(&bars[L::sFull + s], 1);
      mbar_init(&bars[L::pFull + s], kWSoftWarps);
      mbar_init(&bars[L::pvDone + s], 1);
    }
    mbar_init(&bars[L::qFull], kWQWarps);
    mbar_init(&bars[L::qFree], 1);
    mbar_init(&bars[L::oFree], kWSoftWarps);
    mbar_init(&bars[L::drain], 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  constexpr uint32_t tmem = 0;  // all columns: from the first

  if (warp < kWSoftWarps) {
    // ================================================================ softmax warps
    // A warp has the rows 32 quad .. and a quarter of a tile's keys, 32: a thread four rows, frag_row(lane, j), and eight keys,
    // 8 i + 2 c and the one after it.
    const int quad = warp & 3, part = warp >> 2, c = lane & 3, rows_id = 1 + quad;
    const uint32_t lanes0 = static_cast<uint32_t>(quad * 32) << 16, lanes1 = lanes0 + (16u << 16);
    bool failed = false;
    auto await = [&](int bar, uint32_t parity) {
      failed |= !wait_on(&bars[bar], parity, abort_flag, a.wait_budget);
    };
    auto arrive = [&](int bar) {  // for the warp
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bar]);
    };
    auto pick = [&](const float (&x)[4]) { return c < 2 ? (c == 0 ? x[0] : x[1]) : (c == 2 ? x[2] : x[3]); };  // x[c]
    float* red_max = red + quad * 32 + frag_row(lane, c);  // of a row of the thread's; its quarters 128 apart
    auto all_max = [&](int j) {                            // of the four warps
      const float* r = red + quad * 32 + frag_row(lane, j);
      return fmaxf(fmaxf(r[0], r[128]), fmaxf(r[256], r[384]));
    };
    grid_dep_wait();  // the tiles come from the kernel before
    grid_dep_trigger();
    float2* ml = a.part_ml + static_cast<long long>(run) * 256;
    if (warp < 4) {  // until they are written: dropped
      ml[quad * 32 + lane] = make_float2(-INFINITY, -1.0f);
      ml[128 + quad * 32 + lane] = make_float2(-INFINITY, -1.0f);
    }
    int f_unit = 0;
    while (f_unit < n_tiles) {
      // ---- a unit: the key tiles of row tile w.t that belong to this run
      const int n_unit = min(w.keys.n - w.x, n_tiles - f_unit);
      const bool whole_unit = w.x == 0 && n_unit == w.keys.n;
      const int r0 = 128 * w.t + quad * 32, q0 = r0 / a.group, g0 = r0 - q0 * a.group;  // the warp's first row: query, head
      auto query = [&](int row) { return q0 + small_div(g0 + row, a.group_inv); };       // of the warp's row
      float ref[4];
      f2 l[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ref[j] = -INFINITY;
        l[j] = mk2(0.f, 0.f);
      }
      for (int u = 0; u < n_unit; ++u) {
        const int f = f_unit + u, pb = f % kWParBufs, x = w.x + u, sb = f % L::kScoreBufs;
        const int k0 = 128 * (x < w.keys.sink ? x : x - w.keys.sink + w.keys.low) + 32 * part;  // the warp's first key
        const uint32_t tm_s = tmem + 128 * sb + 32 * part, tm_p = tmem + 128 * sb + 16 * part;
        const float2* kf = reinterpret_cast<const float2*>(par + pb * 384 + 32 * part) + c;
        await(L::parFull + pb, (f / kWParBufs) & 1);
        await(L::sFull + sb, (f / L::kScoreBufs) & 1);
        tc::fence_after_sync();
        uint32_t y[32];
        tc::ld_16x256b_x4(tm_s + lanes0, y);
        tc::ld_16x256b_x4(tm_s + lanes1, y + 16);
        tc::wait_ld();
        // z
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 k2 = kf[4 * i], l2 = kf[64 + 4 * i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t* s = y + (j >> 1) * 16 + 4 * i + 2 * (j & 1);
            const f2 z = fma2(mk2(__uint_as_float(s[0]), __uint_as_float(s[1])), mk2(k2.x, k2.y), mk2(l2.x, l2.y));
            s[0] = __float_as_uint(lo2(z));
            s[1] = __float_as_uint(hi2(z));
          }
        }
        // hidden keys: a row at position p sees n < hi, and n >= lo or n < sk, counted from the first of these keys
        const int sk = a.n_sink - k0, hi0 = a.history_len + q0 + 1 - k0;
        if (__builtin_expect(hi0 < 32 || (a.history_len + query(31) + 1 - a.window > k0 && sk < 32), 0)) {  // the same in the warp
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int hi = a.history_len + query(frag_row(lane, j)) + 1 - k0;
            const uint32_t seen = (low_bits(hi) & (low_bits(sk) | ~low_bits(hi - a.window))) >> (2 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (!(seen & (1u << (8 * (e >> 1) + (e & 1)))))
                y[(j >> 1) * 16 + 4 * (e >> 1) + 2 * (j & 1) + (e & 1)] = 0xff800000u;  // -infinity
          }
        }
        float m[4];
        bool over = failed || u == 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          m[j] = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t* s = y + (j >> 1) * 16 + 4 * i + 2 * (j & 1);
            m[j] = fmax3(m[j], __uint_as_float(s[0]), __uint_as_float(s[1]));
          }
          over |= m[j] > ref[j] + kWMost;
        }
        // All scores are in registers, and P may take their place; and does a row's maximum exceed its reference?
        tc::fence_before_sync();
        over = rows_or(rows_id, over);
        tc::fence_after_sync();
        if (__builtin_expect(over, 0)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 1));
            m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 2));
          }
          red_max[128 * part] = pick(m);
          if (rows_or(rows_id, failed)) {
            failed = true;
            break;
          }
          bool moved = false;
          float scale[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            m[j] = all_max(j);
            scale[j] = 1.0f;
            if (u == 0 || m[j] > ref[j] + kWMost) {
              m[j] -= kWLift;
              // (from -infinity there is nothing in l and O, but NaN, which stays)
              if (ref[j] != -INFINITY) {
                scale[j] = fast_exp2(ref[j] - m[j]);
                moved = true;
              }
              ref[j] = m[j];
              l[j] = mul2(l[j], mk2(scale[j], scale[j]));
            }
          }
          rows_or(rows_id, false);  // the maxima are read
          if (__any_sync(0xffffffffu, moved)) {
            // O holds the products up to tile f - 1 (of this unit: u > 0); a quarter of its columns
            await(L::pvDone + (f - 1) % L::kScoreBufs, ((f - 1) / L::kScoreBufs) & 1);
            tc::fence_after_sync();
#pragma unroll 1
            for (int o = 0; o < D / 64; ++o) {  // 16 lanes, 32 columns
              const uint32_t at = tmem + (o & 1 ? lanes1 : lanes0) + L::kOCol + part * (D / 4) + 32 * (o >> 1);
              const float sa = o & 1 ? scale[2] : scale[0], sb2 = o & 1 ? scale[3] : scale[1];
              uint32_t t[16];
              tc::ld_16x256b_x4(at, t);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) t[e] = __float_as_uint(__uint_as_float(t[e]) * (e & 2 ? sb2 : sa));
              tc::st_16x256b_x4(at, t);
            }
          }
        }
        uint32_t p0[8], p1[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 i2 = kf[128 + 4 * i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t* s = y + (j >> 1) * 16 + 4 * i + 2 * (j & 1);
            const float nr = ref[j] == -INFINITY ? 0.0f : -ref[j];
            const f2 v = add2(mk2(__uint_as_float(s[0]), __uint_as_float(s[1])), mk2(nr, nr));
            const float w0 = fast_exp2(lo2(v)), w1 = fast_exp2(hi2(v));
            l[j] = fma2(mk2(w0, w1), mk2(i2.x, i2.y), l[j]);
            (j < 2 ? p0 : p1)[2 * i + (j & 1)] = pack_half2(w0, w1);
          }
        }
        tc::st_16x128b_x4(tm_p + lanes0, p0);
        tc::st_16x128b_x4(tm_p + lanes1, p1);
        tc::wait_st();
        tc::fence_before_sync();
        arrive(L::pFull + sb);
        arrive(L::parFree + pb);
      }
      if (rows_or(rows_id, failed)) break;
      // ---- the unit's sums: this warp's, then all four's
      float sum[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[j] = lo2(l[j]) + hi2(l[j]);
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
      }
      red_max[512 + 128 * part] = pick(sum);
      rows_or(rows_id, false);
      const int slot = 2 * run + (f_unit == 0 ? 0 : 1);
      float inv[4];
      int at_row[4];  // where the thread's rows stand in the output, from its query's first on
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = frag_row(lane, j), qs = small_div(g0 + row, a.group_inv);
        const float* r = red + 512 + quad * 32 + row;
        sum[j] = (r[0] + r[128]) + (r[256] + r[384]);
        inv[j] = sum[j] > 0.0f || sum[j] != sum[j] ? __frcp_rn(sum[j]) : 0.0f;
        at_row[j] = r0 + row < a.n_rows ? (qs * a.n_q_heads + g0 + row - qs * a.group) * D : -1;
      }
      const long long out0 = (static_cast<long long>(q0) * a.n_q_heads + w.kvh * a.group) * D + part * (D / 4);
      // O once its last product is there.  (Few instructions: what runs once a row tile comes from far out of the
      // instruction caches.)
      const int last = f_unit + n_unit - 1;
      await(L::pvDone + last % L::kScoreBufs, (last / L::kScoreBufs) & 1);
      if (rows_or(rows_id, failed)) break;
      tc::fence_after_sync();
      if (!whole_unit && part == 0) ml[(slot & 1) * 128 + quad * 32 + frag_row(lane, c)] = make_float2(pick(ref), pick(sum));
#pragma unroll 1
      for (int o = 0; o < D / 128; ++o) {  // 32 columns of the four rows
        const uint32_t at = tmem + L::kOCol + part * (D / 4) + 32 * o;
        uint32_t y[32];
        tc::ld_16x256b_x4(at + lanes0, y);
        tc::ld_16x256b_x4(at + lanes1, y + 16);
        tc::wait_ld();
        if (o == D / 128 - 1) {  // the next unit's first product may write O
          tc::fence_before_sync();
          arrive(L::oFree);
        }
        if (!whole_unit) {  // a part: the numerator as the threads hold it
          float4* dst = a.part + (((static_cast<long long>(slot) * 4 + quad) * 4 + part) * (D / 128) + o) * (8 * 32) + lane;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e * 32] = make_float4(__uint_as_float(y[4 * e]), __uint_as_float(y[4 * e + 1]), __uint_as_float(y[4 * e + 2]),
                                      __uint_as_float(y[4 * e + 3]));
          continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t* v = y + (j >> 1) * 16 + 2 * (j & 1);  // (columns 8 i + 2 c, + 1 at 4 i)
          auto x = [&](int e) { return __uint_as_float(v[e]) * inv[j]; };
          if (a.out_bf16) {
            // four lanes have 8 columns together, four times: each takes one eight, and a row's 64 bytes are written at once
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(x(4 * i), x(4 * i + 1));
              p[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            lanes4_transpose(c, p);
            if (at_row[j] >= 0)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + out0 + at_row[j] + 32 * o + 8 * c) =
                  make_uint4(p[0], p[1], p[2], p[3]);
          } else if (at_row[j] >= 0) {
            float* d = static_cast<float*>(a.out) + out0 + at_row[j] + 32 * o + 2 * c;
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(d + 8 * i) = make_float2(x(4 * i), x(4 * i + 1));
          }
        }
      }
      f_unit += n_unit;
      w.x += n_unit - 1;
      window_step(a, w);
    }
  } else if (warp == kWMmaWarp) {
    // ================================================================ MMA issue
    grid_dep_wait();
    grid_dep_trigger();
    const uint64_t qd0 = tc::sdesc_sw128(smem_u32(sm)), rd0 = tc::sdesc_sw128(smem_u32(ring));
    constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(128, 128), idesc_pv = tc::idesc_f16_f32(128, D);
    int tile = 0;  // of the ring's fills
    bool ok = true;
    auto await = [&](int bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, wait_on(&bars[bar], parity, abort_flag, a.wait_budget));
      return ok;
    };
    // The next tile, before what it is multiplied with, which comes later.  (A tile cut short passes too, after the flag is set.)
    auto await_tile = [&]() {
      ok = __all_sync(0xffffffffu, wait_on(&bars[L::full + tile % L::kTiles], (tile / L::kTiles) & 1, abort_flag, a.wait_budget) &&
                                       !*abort_flag);
      return ok;
    };
    // S = Q K_f^T, in the place of the P of kScoreBufs tiles before, once that is multiplied
    WindowWalk ws = w;  // of the scores
    int fs = 0, s_unit = -1;
    auto scores = [&]() {
      const int b = fs % L::kScoreBufs, slot = tile % L::kTiles * 2;
      if (!await_tile()) return;
      if (fs == 0 || ws.x == 0) {
        ++s_unit;
        if (!await(L::qFull, s_unit & 1)) return;
      }
      if (fs >= L::kScoreBufs && !await(L::pvDone + b, (fs / L::kScoreBufs - 1) & 1)) return;
      const bool last = ws.x + 1 == ws.keys.n;  // of its row tile: Q's place is free then
      if (elect_one()) {
        tc::fence_after_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < D / 128; ++i) {  // 64 dims
            const uint64_t kd = rd0 + static_cast<uint64_t>(((slot + h) * L::kHalf + i * kPieceBytes) >> 4);
            const uint64_t qd = qd0 + static_cast<uint64_t>((h * L::kHalf + i * kPieceBytes) >> 4);
#pragma unroll
            for (int s = 0; s < 4; ++s) tc::mma_f16_ss(tmem + 128 * b, qd + 2 * s, kd + 2 * s, idesc_qk, (h | i | s) ? 1u : 0u);
          }
          tc::commit(&bars[L::empty + slot + h]);
        }
        tc::commit(&bars[L::sFull + b]);
        if (last) tc::commit(&bars[L::qFree]);
      }
      __syncwarp();
      ++tile;
      ++fs;
      window_step(a, ws);
    };
    int v_unit = -1;
    auto values = [&](int f) {  // O (+)= P_f V_f
      const int b = f % L::kScoreBufs, slot = tile % L::kTiles * 2;
      const bool first = f == 0 || w.x == 0;
      if (!await_tile()) return;
      if (first) ++v_unit;
      if (first && v_unit > 0 && !await(L::oFree, (v_unit - 1) & 1)) return;  // the row tile before has been read
      if (!await(L::pFull + b, (f / L::kScoreBufs) & 1)) return;
      if (elect_one()) {
        tc::fence_after_sync();
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          const uint64_t vd = rd0 + static_cast<uint64_t>(((slot + kh) * L::kHalf) >> 4);
#pragma unroll
          for (int s = 0; s < 4; ++s)
            tc::mma_f16_ts(tmem + L::kOCol, tmem + 128 * b + 32 * kh + 8 * s, vd + 2 * s, idesc_pv,
                           (first && kh == 0 && s == 0) ? 0u : 1u);
          tc::commit(&bars[L::empty + slot + kh]);
        }
        tc::commit(&bars[L::pvDone + b]);
      }
      __syncwarp();
      ++tile;
      window_step(a, w);
    };
    // The scores run ahead of the values, one tile with two score tiles and two with three (scores_next): while the softmax
    // warps are at tile f, the scores of the next are made, and the values of the one before.
    for (int f = 0; ok && f < n_tiles;) {
      if (scores_next<D>(fs, f, n_tiles, ws.x)) scores();
      else values(f++);
    }
    // every MMA this warp issued has completed before the CTA releases tensor memory
    if (elect_one()) {
      tc::commit(&bars[L::drain]);
      mbar_wait(&bars[L::drain], 0, a.status, a.wait_budget);
    }
    __syncwarp();
  } else if (warp == kWCopyWarp) {
    // ================================================================ tile copies, in the order of the products
    grid_dep_wait();
    grid_dep_trigger();
    const bool skip_one = a.fault == 5 && blockIdx.x == 0;  // test-only: the second tile is never copied
    WindowWalk wk = w;                                      // of the scores
    int tile = 0, fk = 0, cut = 0;
    bool ok = true;
    auto await = [&](int bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, wait_on(&bars[bar], parity, abort_flag, a.wait_budget));
      return ok;
    };
    for (int f = 0; ok && f < n_tiles; ++tile) {
      const bool is_k = scores_next<D>(fk, f, n_tiles, wk.x);
      WindowWalk& at = is_k ? wk : w;
      const long long u = static_cast<long long>(at.kvh) * a.key_tiles + stored_tile(a, at.tile());
      window_step(a, at);
      if (is_k) {
        const int pb = fk % kWParBufs;
        if (fk >= kWParBufs && !await(L::parFree + pb, (fk / kWParBufs - 1) & 1)) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars[L::parFull + pb], 1536);
          bulk_g2s(par + pb * 384, a.par + u * 384, 1536, &bars[L::parFull + pb]);
        }
        __syncwarp();
        ++fk;
      } else {
        ++f;
      }
      const uint8_t* src = (is_k ? a.k_tiles : a.v_tiles) + u * (2 * L::kHalf);
      const int slot = tile % L::kTiles * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (tile >= L::kTiles && !await(L::empty + slot + h, (tile / L::kTiles - 1) & 1)) {
          cut = h;  // the tile has one half
          break;
        }
        if (!(skip_one && tile == 1) && elect_one()) {
          mbar_arrive_expect_tx(&bars[L::full + slot / 2], L::kHalf);
          bulk_g2s(ring + (slot + h) * L::kHalf, src + h * L::kHalf, L::kHalf, &bars[L::full + slot / 2]);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    // Copies still in flight (only after an abort) land before the CTA exits, those of a tile cut short too.
    if (lane == 0) {
      if (cut) mbar_arrive(&bars[L::full + tile++ % L::kTiles]);
      for (int i = max(0, tile - L::kTiles); i < tile; ++i)
        if (!(skip_one && i == 1)) mbar_wait(&bars[L::full + i % L::kTiles], (i / L::kTiles) & 1, a.status, a.wait_budget);
      for (int i = max(0, fk - kWParBufs); i < fk; ++i)
        mbar_wait(&bars[L::parFull + i % kWParBufs], (i / kWParBufs) & 1, a.status, a.wait_budget);
    }
    __syncwarp();
  } else {
    // ================================================================ queries: a row tile's when its place is free
    const int t0 = tid - 32 * kWQWarp;
    constexpr int CH = D / 8, ROWS = 32 * kWQWarps / CH;  // 16-byte chunks of a row, rows at a time
    const int ch = t0 % CH;
    int units = 0;
    for (int f = 0; f < n_tiles; ++units) {
      if (units > 0 && !__all_sync(0xffffffffu, wait_on(&bars[L::qFree], (units - 1) & 1, abort_flag, a.wait_budget))) break;
      // every row's address for itself, four rows of a thread on their way: two warps alone have nothing else to fill the
      // latencies with
      const int r0 = 128 * w.t, q0 = r0 / a.group, g0 = r0 - q0 * a.group, rows = min(a.n_rows - r0, 128);
      const uint16_t* src = static_cast<const uint16_t*>(a.q) +
                            (static_cast<long long>(q0) * a.n_q_heads + w.kvh * a.group) * D + 8 * ch;
      uint8_t* dst = sm + (ch >> 3) * kPieceBytes;
#pragma unroll 4
      for (int n = t0 / CH; n < 128; n += ROWS) {
        const int q = small_div(g0 + n, a.group_inv), g = g0 + n - q * a.group;
        const bool real = n < rows;
        cp_async16(dst + tc::sw128_off(n, ch & 7), real ? src + (q * a.n_q_heads + g) * D : src, real);
      }
      cp_async_wait();
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::qFull]);
      // The first queries come from before the kernel that makes the tiles, which waits for them before it lets this one
      // start (window_tiles_kernel); this grid's own wait is the other warps'.
      const int n_unit = min(w.keys.n - w.x, n_tiles - f);
      f += n_unit;
      w.x += n_unit - 1;
      window_step(a, w);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(a.status, KVQ_DEV_TIMEOUT);
  if (warp == kWMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ============================================================================ joining the parts
// Block (run, 32 columns).  The run in which a cut row tile ends joins its parts, from the run in which it
// begins on; threads take the places of the attention kernel's softmax threads, as the parts lie, two threads for the four
// rows of one.  Two parts are fetched at once, five blocks an SM; one part after the other 28 us for ten parts, four at once and
// three blocks an SM 4 us more for the chunk of 32K.
template <int D>
__global__ void __launch_bounds__(256, 5) window_join_kernel(const __grid_constant__ PrefillWindowArgs a, int runs) {
  const int run = blockIdx.x, o = blockIdx.y, quad = (threadIdx.x >> 5) & 3, h = threadIdx.x >> 7, lane = threadIdx.x & 31;
  const long long f0 = run_start(a, run, runs), f1 = run_start(a, run + 1, runs);
  const WindowWalk w = window_walk_at(a, f0);
  const long long start = f0 - w.x;
  // the last run c with run_start(c) <= start: the row tile begins in it
  const int first = static_cast<int>(((start + 1) * runs - 1) / (a.line * a.n_kv_heads));
  const int first_slot = 2 * first + (run_start(a, first, runs) < start ? 1 : 0);
  grid_dep_wait();
  grid_dep_trigger();
  if (w.x == 0 || start + w.keys.n > f1) return;
  const int c = lane & 3, row0 = quad * 32 + frag_row(lane, 2 * h);  // the thread's rows: row0, row0 + 8
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  bool dropped[2] = {false, false};
  float4 acc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = first; i0 <= run; i0 += 2) {
    float2 v[2][2];
    float4 x[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const long long slot = i0 + t == first ? first_slot : 2 * (i0 + t);
      const float4* src = a.part + ((slot * 4 + quad) * (D / 32) + o) * (8 * 32) + (4 * h) * 32 + lane;  // (o: half of the columns, then 32)
      const bool real = i0 + t <= run;
#pragma unroll
      for (int j = 0; j < 2; ++j) v[t][j] = real ? a.part_ml[slot * 128 + row0 + 8 * j] : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[t][e] = real ? src[e * 32] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float s[2][2];
    bool none[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float was = m[j];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        m[j] = fmaxf(m[j], v[t][j].x);
        dropped[j] |= v[t][j].y < 0.0f;
      }
      const float s0 = was == m[j] || was == -INFINITY ? 1.0f : fast_exp2(was - m[j]);
      l[j] *= s0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        (j ? acc[e].z : acc[e].x) *= s0;
        (j ? acc[e].w : acc[e].y) *= s0;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        none[t][j] = v[t][j].x == -INFINITY && v[t][j].y == 0.0f;  // the row sees no key of this part
        s[t][j] = v[t][j].x == -INFINITY ? 1.0f : fast_exp2(v[t][j].x - m[j]);  // (a part of NaN alone has no maximum)
        if (!none[t][j]) l[j] = fmaf(v[t][j].y, s[t][j], l[j]);
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!none[t][0]) {
          acc[e].x = fmaf(x[t][e].x, s[t][0], acc[e].x);
          acc[e].y = fmaf(x[t][e].y, s[t][0], acc[e].y);
        }
        if (!none[t][1]) {
          acc[e].z = fmaf(x[t][e].z, s[t][1], acc[e].z);
          acc[e].w = fmaf(x[t][e].w, s[t][1], acc[e].w);
        }
      }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int rr = 128 * w.t + row0 + 8 * j, q2 = rr / a.group;
    if (rr >= a.n_rows || dropped[j]) continue;
    const float inv = l[j] > 0.0f || l[j] != l[j] ? 1.0f / l[j] : 0.0f;
    const long long at = (static_cast<long long>(q2) * a.n_q_heads + w.kvh * a.group + (rr - q2 * a.group)) * D + 32 * o + 2 * c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 u = acc[e];
      const float x = (j ? u.z : u.x) * inv, y = (j ? u.w : u.y) * inv;
      if (a.out_bf16) *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(a.out) + at + 8 * e) = __floats2bfloat162_rn(x, y);
      else *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + 8 * e) = make_float2(x, y);
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
  // (two tiles a run at least: a part costs more to write and to join than a tile; 80 pairs, one | two | three a run: 21.0 |
  // 18.6 | 22.2 us)
  p.runs = static_cast<int>(std::min<long long>(std::max(1LL, pairs / 2), std::min(n_sms, kWMaxRuns)));
  const long long max_runs = std::min<long long>(std::max(1LL, pairs / 2), kWMaxRuns), tiles = static_cast<long long>(n_kv_heads) * p.key_tiles;
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
  e = launch_pdl(window_tiles_kernel<D>, dim3(a.key_tiles, a.n_kv_heads, 4), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(window_attention_kernel<D>, dim3(runs), dim3(kWThreads), L::kAlloc, stream, a);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(runs, D / 32);
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
