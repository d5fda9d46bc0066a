// decode_accum.cu — the decode step that also adds up the attention weight of every key.
//
// An eviction by accumulated weight needs, per (sequence, KV head, key), the sum of the softmax
// weights that the queries gave it:
//   acc[b][kvh][t] += sum over the query rows i and the heads h of the KV head's group of
//                     p[b][i][h][t] = 2^(s[t] - M) / l,
// with s the scores in log2 units, M and l the row's maximum and sum over all its keys.  M and l are
// known only when the whole row has been walked, so stage 1 (decode_stage1.cuh, with SCORES) leaves
// its scores behind, 4 bytes per (query row, key) against the 2 * head_dim + 8 bytes of the key's K
// and V, and step_tail_kernel turns them into weights, in the launch that merges the splits.  Its reads
// mostly hit L2: the scores of a call were just written.  A thread owns four keys and sums the rows in
// a fixed order: no atomics, the same result every time.
//
// Bound: bytes for a large batch (64 sequences of up to 16384, 32 heads on 8 of 128: 242 us, stage 1 215 at
// 5.3 TB/s of K and V, the tail 31); few sequences are latency and the row arithmetic of stage 1 (1 x 1024: 8.5 us; 4
// new tokens after 32763, 24 rows a KV head: 40 us, stage 1 36, tail 10 alone and part of it behind stage 1).
// One launch for merge and weights: 11.8 -> 8.5 us at 1 x 1024 against a launch each.
#include <atomic>
#include <cstdint>

#include "decode_merge.cuh"
#include "decode_stage1.cuh"

namespace kvq {

namespace {

constexpr int kAccumThreads = 256;
constexpr int kKeysPerThread = 4;
constexpr int kAccumKeys = kKeysPerThread * kAccumThreads;  // keys per CTA
constexpr int kRowsAhead = 8;                               // rows whose scores a thread loads before their statistics are known
constexpr int kRowLanes = 8;                                // lanes that share a row's statistics
static_assert(kAccumThreads == kMergeThreads && kAccumThreads == 256, "one launch does both");

// The weights of kAccumKeys keys of one (sequence, KV head).
__device__ __forceinline__ void accum_block(const StepAccumArgs& sa, int chunk, int kvh, int b) {
  const DecodeArgs& a = sa.d;
  __shared__ float row_m[KVQ_VERIFY_MAX_ROWS], row_il[KVQ_VERIFY_MAX_ROWS];
  const int tid = threadIdx.x;
  const int Hq = a.n_q_heads, G = Hq / a.n_kv_heads, nq = a.nq, R = G * nq;
  grid_dep_wait();
  const int raw = a.ctx_lens[b];
  const int cap = min(a.max_blocks_per_seq * KVQ_BLOCK_SIZE, a.max_ctx);
  const int ctx = max(0, min(raw, cap));
  if (chunk * kAccumKeys >= ctx) return;
  const int t = chunk * kAccumKeys + kKeysPerThread * tid;
  const int n = min(a.n_split, (ctx + a.split_rows - 1) / a.split_rows);
  // rows of scores start on 16 bytes and hold whole groups of 16 keys
  const float* sc = a.scores + (static_cast<long long>(b) * a.n_kv_heads + kvh) * R * a.scores_stride + t;
  float4 ahead[kRowsAhead];
#pragma unroll
  for (int r = 0; r < kRowsAhead; ++r)
    if (r < R && t < ctx) ahead[r] = __ldcg(reinterpret_cast<const float4*>(sc + r * a.scores_stride));
  const long long at = (static_cast<long long>(b) * a.n_kv_heads + kvh) * sa.acc_stride + t;
  const int first_new = a.k_new != nullptr && raw >= nq && raw <= cap ? ctx - nq : ctx;  // new tokens start from zero
  const bool whole = t + kKeysPerThread <= first_new && (reinterpret_cast<uintptr_t>(sa.acc + at) & 15) == 0;
  float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
  if (whole) old = *reinterpret_cast<const float4*>(sa.acc + at);
  // each row's maximum and 1 / l over the splits' statistics, in one pass of eight lanes
  for (int r = tid / kRowLanes; r < (R + 3) / 4 * 4; r += kAccumThreads / kRowLanes) {  // whole warps
    const int rr = min(r, R - 1);
    const long long orow = (static_cast<long long>(b) * nq + rr / G) * Hq + kvh * G + rr % G;
    const float4* st = reinterpret_cast<const float4*>(a.part_stats) + orow * a.n_split;
    float m = -INFINITY, l = 0.f;
    auto join = [&](float om, float ol) {
      // without a maximum a sum is 0 (no key) or NaN (every score is), and 2^-inf times it is the same
      const float top = fmaxf(m, om), ref = top == -INFINITY ? 0.f : top;
      l = l * fast_exp2(m - ref) + ol * fast_exp2(om - ref);
      m = top;
    };
    for (int s0 = tid % kRowLanes; s0 < n; s0 += 4 * kRowLanes) {
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = s0 + i * kRowLanes < n ? st[s0 + i * kRowLanes] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) join(v[i].x, v[i].w);
    }
#pragma unroll
    for (int off = kRowLanes / 2; off > 0; off >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, off), ol = __shfl_xor_sync(0xffffffffu, l, off);
      join(om, ol);
    }
    if (tid % kRowLanes == 0 && r < R) {
      row_m[r] = m == -INFINITY ? 0.f : m;
      row_il[r] = l == 0.f ? 0.f : __fdiv_rn(1.0f, l);  // a row with no key gives no weight
    }
  }
  __syncthreads();
  if (t >= ctx) return;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](const float4& s4, int r) {
    const float m = row_m[r], il = row_il[r];
    w[0] = fmaf(fast_exp2(s4.x - m), il, w[0]);
    w[1] = fmaf(fast_exp2(s4.y - m), il, w[1]);
    w[2] = fmaf(fast_exp2(s4.z - m), il, w[2]);
    w[3] = fmaf(fast_exp2(s4.w - m), il, w[3]);
  };
  for (int r0 = 0; r0 < R; r0 += kRowsAhead) {
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      if (r0 + i < R) add(ahead[i], r0 + i);
      if (r0 + kRowsAhead + i < R)
        ahead[i] = __ldcg(reinterpret_cast<const float4*>(sc + static_cast<long long>(r0 + kRowsAhead + i) * a.scores_stride));
    }
  }
  if (w[0] != w[0]) {
    // A row that is not finite has made every sum NaN.  Again, row by row: it gives NaN to the keys it sees and nothing
    // to the others, where 0 * NaN is neither.  (A branch in the loop above cost 6 of 40 us at 24 rows.)
    const int page = a.block_table[static_cast<long long>(b) * a.max_blocks_per_seq + t / KVQ_BLOCK_SIZE];
    w[0] = w[1] = w[2] = w[3] = 0.f;
    for (int r = 0; r < R; ++r) {
      const float il = row_il[r];
      if (il == il) {
        add(__ldcg(reinterpret_cast<const float4*>(sc + r * a.scores_stride)), r);
      } else if (page >= 0 && page < a.num_blocks) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t + i <= ctx - nq + r / G) w[i] = il;
      }
    }
  }
  if (whole) {
    *reinterpret_cast<float4*>(sa.acc + at) = make_float4(old.x + w[0], old.y + w[1], old.z + w[2], old.w + w[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (t + i < first_new) {
      sa.acc[at + i] += w[i];
    } else if (t + i < ctx) {
      sa.acc[at + i] = w[i];
      if (sa.slot_pos) sa.slot_pos[at + i] = sa.pos[b] + (t + i - first_new);
    }
  }
}

}  // namespace

// Stage 2: the first CTAs merge the splits into the output, the others make the weights.  Both need
// stage 1 alone, so they share a launch.  Three CTAs an SM: 242 us at 64 x 16384, 252 with two, and 239 with
// four, which costs 0.5 us at 1 x 1024; the warps' merge at head_dim 256 would spill at three.
template <int D, bool WARPS>
__global__ void __launch_bounds__(kAccumThreads, D == 256 && WARPS ? 2 : 3) step_tail_kernel(StepAccumArgs sa) {
  extern __shared__ float wts[];  // [n_split], of a merging CTA
  int x = blockIdx.x;
  if (x < sa.merge_blocks) {
    if (WARPS) {
      decode_merge_warps<D>(sa.d, x);
    } else {
      constexpr int kCols = D / kMergeCols;
      decode_merge_block<D>(sa.d, x / kCols % sa.d.n_q_heads, x / kCols / sa.d.n_q_heads, x % kCols, wts);
    }
    return;
  }
  x -= sa.merge_blocks;
  const int unit = x / sa.key_blocks;
  accum_block(sa, x % sa.key_blocks, unit % sa.d.n_kv_heads, unit / sa.d.n_kv_heads);
}

// CTAs of the tail: those that merge, those of keys per (sequence, KV head), all.
struct TailGrid {
  bool warps;
  long long merge, keys, all;
};
static TailGrid tail_grid(const DecodeArgs& d) {
  const long long rows = static_cast<long long>(d.batch) * d.nq * d.n_q_heads, units = static_cast<long long>(d.batch) * d.n_kv_heads;
  TailGrid g;
  g.warps = decode_merge_by_warps(d);
  g.merge = g.warps ? (rows + 7) / 8 : rows * (d.head_dim / kMergeCols);
  g.keys = (static_cast<long long>(d.max_ctx) + kAccumKeys - 1) / kAccumKeys;
  g.all = g.merge + units * g.keys;
  return g;
}

bool step_accum_grid_ok(const DecodeArgs& d) { return tail_grid(d).all <= INT32_MAX; }

// Stage 1 writes the new tokens, so whatever can be refused is asked for before it.
template <int D>
static cudaError_t prepare_tail(const DecodeArgs& d, const TailGrid& g) {
  static std::atomic<uint64_t> done{0};
  if (g.warps || d.n_split * sizeof(float) <= kMergeSmem) return cudaSuccess;
  return allow_smem(reinterpret_cast<const void*>(step_tail_kernel<D, false>), kMaxSplits * sizeof(float), done);
}

template <int D>
static cudaError_t launch_tail(StepAccumArgs a, const TailGrid& g, cudaStream_t stream) {
  a.merge_blocks = static_cast<int>(g.merge);
  a.key_blocks = static_cast<int>(g.keys);
  const dim3 grid(static_cast<unsigned>(g.all));
  return g.warps ? launch_pdl(step_tail_kernel<D, true>, grid, dim3(kAccumThreads), 0, stream, a)
                 : launch_pdl(step_tail_kernel<D, false>, grid, dim3(kAccumThreads), a.d.n_split * sizeof(float), stream, a);
}

template <int D>
static cudaError_t launch_stage1_scores(const DecodeArgs& a, dim3 grid, cudaStream_t stream) {
  if (a.nq == 1 && a.n_q_heads / a.n_kv_heads <= 8) {
    if (a.k_new) return launch_stage1<D, 1, true, false, true, true>(a, grid, stream);
    return launch_stage1<D, 1, true, false, false, true>(a, grid, stream);
  }
  const int rows = (a.n_q_heads / a.n_kv_heads) * a.nq;
  switch ((rows + 7) / 8) {
    case 1: return launch_stage1<D, 1, true, true, true, true>(a, grid, stream);
    case 2: return launch_stage1<D, 2, true, true, true, true>(a, grid, stream);
    case 3: return launch_stage1<D, 3, true, true, true, true>(a, grid, stream);
    case 4: return launch_stage1<D, 4, true, true, true, true>(a, grid, stream);
    case 5: return launch_stage1<D, 5, true, true, true, true>(a, grid, stream);
    case 6: return launch_stage1<D, 6, true, true, true, true>(a, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_step_accum(const StepAccumArgs& a, cudaStream_t stream, int* launched) {
  *launched = 2;
  const TailGrid g = tail_grid(a.d);
  cudaError_t e = a.d.head_dim == 256 ? prepare_tail<256>(a.d, g) : prepare_tail<128>(a.d, g);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.d.n_split, a.d.n_kv_heads, a.d.batch);
  e = a.d.head_dim == 256 ? launch_stage1_scores<256>(a.d, grid, stream) : launch_stage1_scores<128>(a.d, grid, stream);
  if (e != cudaSuccess) return e;
  return a.d.head_dim == 256 ? launch_tail<256>(a, g, stream) : launch_tail<128>(a, g, stream);
}

}  // namespace kvq
