// decode_accum.cu — the decode step that also adds up the attention weight of every key.
//
// An eviction by accumulated weight needs, per (sequence, KV head, key), the sum of the softmax
// weights that the queries gave it:
//   acc[b][kvh][t] += sum over the query rows i and the heads h of the KV head's group of
//                     p[b][i][h][t] = 2^(s[t] - M) / l,
// with s the scores in log2 units, M and l the row's maximum and sum over all its keys.  M and l are
// known only when the whole row has been walked, so stage 1 (decode_stage1.cuh, with SCORES) leaves
// its scores behind, 4 bytes per (query row, key) against the 2 * head_dim + 8 bytes of the key's K
// and V, and accum_kernel turns them into weights.  Its reads mostly hit L2: the scores of a call
// were just written.  A thread owns four keys and sums the rows in a fixed order: no atomics, the
// same result every time.
#include "decode_stage1.cuh"

namespace kvq {

namespace {

constexpr int kAccumThreads = 256;
constexpr int kAccumKeys = 4 * kAccumThreads;  // keys per CTA

}  // namespace

__global__ void __launch_bounds__(kAccumThreads) accum_kernel(StepAccumArgs sa) {
  const DecodeArgs& a = sa.d;
  __shared__ float row_m[KVQ_VERIFY_MAX_ROWS], row_il[KVQ_VERIFY_MAX_ROWS];
  const int kvh = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hq = a.n_q_heads, G = Hq / a.n_kv_heads, nq = a.nq, R = G * nq;
  grid_dep_wait();
  const int raw = a.ctx_lens[b];
  const int cap = min(a.max_blocks_per_seq * KVQ_BLOCK_SIZE, a.max_ctx);
  const int ctx = max(0, min(raw, cap));
  const int t = static_cast<int>(blockIdx.x) * kAccumKeys + 4 * tid;
  if (static_cast<int>(blockIdx.x) * kAccumKeys >= ctx) return;
  const int n = min(a.n_split, (ctx + a.split_rows - 1) / a.split_rows);
  // each row's maximum and 1 / l over the splits' statistics
  for (int r = warp; r < R; r += kAccumThreads / 32) {
    const long long orow = (static_cast<long long>(b) * nq + r / G) * Hq + kvh * G + r % G;
    const float4* st = reinterpret_cast<const float4*>(a.part_stats) + orow * a.n_split;
    float m = -INFINITY;
    for (int s = lane; s < n; s += 32) m = fmaxf(m, st[s].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float mr = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int s = lane; s < n; s += 32) {
      const float4 v = st[s];
      if (v.x != -INFINITY) l += v.z * fast_exp2(v.x - mr);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane == 0) {
      row_m[r] = mr;
      row_il[r] = l == 0.f ? 0.f : __fdiv_rn(1.0f, l);  // a row with no key gives no weight
    }
  }
  __syncthreads();
  if (t >= ctx) return;
  // scores rows start on 16 bytes and hold whole groups of 16 keys
  const float* sc = a.scores + (static_cast<long long>(b) * a.n_kv_heads + kvh) * R * a.scores_stride + t;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int r = 0; r < R; ++r) {
    const float4 s4 = __ldcg(reinterpret_cast<const float4*>(sc + static_cast<long long>(r) * a.scores_stride));
    const float m = row_m[r], il = row_il[r];
    w[0] = fmaf(fast_exp2(s4.x - m), il, w[0]);
    w[1] = fmaf(fast_exp2(s4.y - m), il, w[1]);
    w[2] = fmaf(fast_exp2(s4.z - m), il, w[2]);
    w[3] = fmaf(fast_exp2(s4.w - m), il, w[3]);
  }
  // new tokens (when they were written) start from zero
  const bool wrote = a.k_new != nullptr && raw >= nq && raw <= cap;
  const int first_new = wrote ? ctx - nq : ctx;
  const long long at = (static_cast<long long>(b) * a.n_kv_heads + kvh) * sa.acc_stride + t;
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
  *launched = 3;
  const dim3 grid(a.d.n_split, a.d.n_kv_heads, a.d.batch);
  cudaError_t e = a.d.head_dim == 256 ? launch_stage1_scores<256>(a.d, grid, stream)
                                      : launch_stage1_scores<128>(a.d, grid, stream);
  if (e != cudaSuccess) return e;
  if ((e = launch_decode_merge(a.d, stream)) != cudaSuccess) return e;
  const dim3 ga((a.d.max_ctx + kAccumKeys - 1) / kAccumKeys, a.d.n_kv_heads, a.d.batch);
  return launch_pdl(accum_kernel, ga, dim3(kAccumThreads), 0, stream, a);
}

}  // namespace kvq
