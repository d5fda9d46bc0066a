// decode_merge.cuh — stage 2 of decode's split route: the splits' partials of a query row into its output.
// Shared by the merge launches of decode.cu and by the step that adds up attention weights, whose
// second launch also merges.
#pragma once

#include "kvq_dev.cuh"
#include "kvq_launch.h"

namespace kvq {

// Stage 2: log-sum-exp merge of the splits of one (sequence, query row, query head).
//   M_s = max m_s, M_z = max m_z;  l = sum l_s 2^{m_s - M_s};  o = sum acc_s 2^{m_z - M_z};
//   out = o 2^{M_z - M_s} / l.  The per-split weights are computed once into shared memory
// ("ROCm/RDNA4 (gfx1201) vLLM ...", "The reduce is not free": one cooperative pass, each
// exponential once per split).  One CTA per (query head, sequence, 64-dim column block), so that
// a small batch still spreads over many SMs; 256 threads = 16 split groups x 16 threads of 4
// dims; each thread keeps 8 independent loads in flight.
constexpr int kMergeThreads = 256;
constexpr int kMergeCols = 64;
constexpr size_t kMergeSmem = 40 * 1024;  // of splits' weights: with the merge's own arrays below the 48 KB of any kernel

// wts: [n_split] weights of the partial accumulators (shared memory).
template <int D>
__device__ __forceinline__ void decode_merge_block(const DecodeArgs& a, int h, int row, int col_block, float* wts) {
  constexpr int TPG = kMergeCols / 4;           // threads per split group (4 dims each)
  constexpr int NG = kMergeThreads / TPG;       // split groups
  constexpr int PRE = 8;                        // partials per thread loaded before the weights
  __shared__ float red[2][kMergeThreads / 32];
  __shared__ __align__(16) float4 part[NG][TPG];
  // row = b * nq + i: query row i of sequence b
  const int b = row / a.nq, Hq = a.n_q_heads, col0 = col_block * kMergeCols;
  const long long pu0 = (static_cast<long long>(row) * Hq + h) * a.n_split;
  const float* stats = a.part_stats + pu0 * 4;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int grp = tid / TPG, dq = tid % TPG;
  const float4* acc = reinterpret_cast<const float4*>(a.part_acc + pu0 * D + col0) + dq;
  grid_dep_wait();  // the partials come from stage 1
  // The first PRE partials of this thread and its split's statistics are loaded together with
  // ctx, before the number of live splits is known: the reads stay inside the grid's n_split
  // slots, and slots past the live ones are never used.
  float4 v[PRE];
#pragma unroll
  for (int u = 0; u < PRE; ++u)
    if (grp + u * NG < a.n_split) v[u] = acc[static_cast<long long>(grp + u * NG) * (D / 4)];
  float4 st0 = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
  if (tid < a.n_split) st0 = reinterpret_cast<const float4*>(stats)[tid];
  int ctx = a.ctx_lens[b];
  ctx = max(0, min(ctx, min(a.max_blocks_per_seq * KVQ_BLOCK_SIZE, a.max_ctx)));
  const int n = min(a.n_split, (ctx + a.split_rows - 1) / a.split_rows);

  float Ms = tid < n ? st0.x : -INFINITY, Mz = tid < n ? st0.y : -INFINITY;
  for (int s = tid + kMergeThreads; s < n; s += kMergeThreads) {
    Ms = fmaxf(Ms, stats[s * 4 + 0]);
    Mz = fmaxf(Mz, stats[s * 4 + 1]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    Ms = fmaxf(Ms, __shfl_xor_sync(0xffffffffu, Ms, off));
    Mz = fmaxf(Mz, __shfl_xor_sync(0xffffffffu, Mz, off));
  }
  if (lane == 0) {
    red[0][wid] = Ms;
    red[1][wid] = Mz;
  }
  __syncthreads();
  Ms = -INFINITY;
  Mz = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMergeThreads / 32; ++i) {
    Ms = fmaxf(Ms, red[0][i]);
    Mz = fmaxf(Mz, red[1][i]);
  }
  float lpart = 0.f;
  for (int s = tid; s < n; s += kMergeThreads) {
    const float4 st = s == tid ? st0 : reinterpret_cast<const float4*>(stats)[s];
    wts[s] = (Mz != -INFINITY && st.y != -INFINITY) ? fast_exp2(st.y - Mz) : 0.f;
    lpart += (Ms != -INFINITY && st.x != -INFINITY) ? st.z * fast_exp2(st.x - Ms) : 0.f;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) lpart += __shfl_xor_sync(0xffffffffu, lpart, off);
  __syncthreads();  // red[] and wts[] reuse
  if (lane == 0) red[0][wid] = lpart;
  __syncthreads();
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < kMergeThreads / 32; ++i) l += red[0][i];

  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int u = 0; u < PRE; ++u) {
    const int s = grp + u * NG;
    if (s < n) {
      const float wgt = wts[s];
      o.x = fmaf(v[u].x, wgt, o.x);
      o.y = fmaf(v[u].y, wgt, o.y);
      o.z = fmaf(v[u].z, wgt, o.z);
      o.w = fmaf(v[u].w, wgt, o.w);
    }
  }
  int s = grp + PRE * NG;
  for (; s + 7 * NG < n; s += 8 * NG) {
    float4 w8[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) w8[u] = acc[static_cast<long long>(s + u * NG) * (D / 4)];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float wgt = wts[s + u * NG];
      o.x = fmaf(w8[u].x, wgt, o.x);
      o.y = fmaf(w8[u].y, wgt, o.y);
      o.z = fmaf(w8[u].z, wgt, o.z);
      o.w = fmaf(w8[u].w, wgt, o.w);
    }
  }
  for (; s < n; s += NG) {
    const float4 w1 = acc[static_cast<long long>(s) * (D / 4)];
    const float wgt = wts[s];
    o.x = fmaf(w1.x, wgt, o.x);
    o.y = fmaf(w1.y, wgt, o.y);
    o.z = fmaf(w1.z, wgt, o.z);
    o.w = fmaf(w1.w, wgt, o.w);
  }
  part[grp][dq] = o;
  __syncthreads();
  if (grp == 0) {
    float4 t = part[0][dq];
#pragma unroll
    for (int g2 = 1; g2 < NG; ++g2) {
      const float4 u = part[g2][dq];
      t.x += u.x;
      t.y += u.y;
      t.z += u.z;
      t.w += u.w;
    }
    const float sc = (l > 0.f && Mz != -INFINITY) ? fast_exp2(Mz - Ms) / l : 0.f;
    reinterpret_cast<float4*>(a.out + (static_cast<long long>(row) * Hq + h) * D + col0)[dq] =
        make_float4(t.x * sc, t.y * sc, t.z * sc, t.w * sc);
  }
}

// Stage 2 for many (query row, head) units with few splits each (a large batch): one warp per
// unit, the splits' statistics in its lanes and their weights passed by shuffles, each lane
// combining D / 32 head dimensions of every split.  No shared memory and no block barrier, and
// a CTA of eight warps takes eight units, so the grid stays within a wave where the per-(unit,
// 64-dim block) CTAs of decode_merge_block would take several.  The same rule as that kernel.
constexpr int kMergeWarpMaxSplits = 32;

template <int D>
__device__ __forceinline__ void decode_merge_warps(const DecodeArgs& a, int block) {
  constexpr int PER = D / 32;  // dims per lane
  const int lane = threadIdx.x & 31;
  const int Hq = a.n_q_heads;
  const long long unit = static_cast<long long>(block) * 8 + (threadIdx.x >> 5);  // row * Hq + h
  grid_dep_wait();  // the partials come from stage 1
  if (unit >= static_cast<long long>(a.batch) * a.nq * Hq) return;  // warp-uniform
  const int row = static_cast<int>(unit / Hq), b = row / a.nq;
  int ctx = a.ctx_lens[b];
  ctx = max(0, min(ctx, min(a.max_blocks_per_seq * KVQ_BLOCK_SIZE, a.max_ctx)));
  const int n = min(a.n_split, (ctx + a.split_rows - 1) / a.split_rows);
  const long long pu0 = unit * a.n_split;
  float4 st = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
  if (lane < n) st = reinterpret_cast<const float4*>(a.part_stats)[pu0 + lane];
  float Ms = st.x, Mz = st.y;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    Ms = fmaxf(Ms, __shfl_xor_sync(0xffffffffu, Ms, off));
    Mz = fmaxf(Mz, __shfl_xor_sync(0xffffffffu, Mz, off));
  }
  float l = (Ms != -INFINITY && st.x != -INFINITY) ? st.z * fast_exp2(st.x - Ms) : 0.f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  const float wgt = (Mz != -INFINITY && st.y != -INFINITY) ? fast_exp2(st.y - Mz) : 0.f;  // split `lane`
  float o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.f;
  const float* acc = a.part_acc + pu0 * D + lane * PER;
  for (int s0 = 0; s0 < n; s0 += 8) {
    float4 v[8][PER / 4];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (s0 + u < n)
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) v[u][i] = *reinterpret_cast<const float4*>(acc + static_cast<long long>(s0 + u) * D + 4 * i);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float w = __shfl_sync(0xffffffffu, wgt, (s0 + u) & 31);
      if (s0 + u < n)
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
          o[4 * i + 0] = fmaf(v[u][i].x, w, o[4 * i + 0]);
          o[4 * i + 1] = fmaf(v[u][i].y, w, o[4 * i + 1]);
          o[4 * i + 2] = fmaf(v[u][i].z, w, o[4 * i + 2]);
          o[4 * i + 3] = fmaf(v[u][i].w, w, o[4 * i + 3]);
        }
    }
  }
  const float sc = (l > 0.f && Mz != -INFINITY) ? fast_exp2(Mz - Ms) / l : 0.f;
  float* dst = a.out + unit * D + lane * PER;
#pragma unroll
  for (int i = 0; i < PER / 4; ++i)
    *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(o[4 * i] * sc, o[4 * i + 1] * sc, o[4 * i + 2] * sc, o[4 * i + 3] * sc);
}

// Many (query row, head) units and few splits: a warp a unit.
inline bool decode_merge_by_warps(const DecodeArgs& a) {
  return a.n_split <= kMergeWarpMaxSplits && static_cast<long long>(a.batch) * a.nq * a.n_q_heads >= 512;
}

}  // namespace kvq
