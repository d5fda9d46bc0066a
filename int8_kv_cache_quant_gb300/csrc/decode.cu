// decode.cu — decode attention over the int8 paged K/V cache: one query per sequence, or nq
// query rows per sequence (speculative / MTP verify, causal among the nq newest tokens).
//
// Method: "gfx936 DCU上实现INT8 KV与INT8 MMAC Attention推理优化" §3.3 (locate the paged
// int8 K/V, QK on the int8 codes, scale restore and online softmax, PV, partition merge;
// no dequantised K/V tensor), §1.2 (decode is bound by the K/V read); "dot4-flash-attention"
// README route table (one CTA per head for short contexts; split-K stage 1 over 512-row
// splits emitting partial max / sum / acc, stage 2 merging them with the online-softmax
// rule); "ROCm/RDNA4 (gfx1201) vLLM ..." ("Don't re-read what a group shares": the GQA
// group is folded into the matrix dimension so each K/V page is read once per KV head).
//
// GB300 design.
// * Grid over (split, KV head, sequence).  Each of the CTA's eight warps takes whole pages
//   (warp w: pages w, w + 8, ...) and streams each (page, head) block of K and V (4 KB each
//   at head_dim 256, contiguous in the cache layout) and its two 64-byte scale runs into its
//   own DEPTH-stage shared-memory ring with 1-D bulk copies (TMA) completing on mbarriers;
//   it refills a slot as soon as it has read the page in it.  A warp does QK, the online
//   softmax and PV of a page over the whole head dimension: no exchange with another warp
//   and no softmax computed twice.  The warps' partial results are merged at the end of the
//   CTA.
// * QK and PV of a 16-token page run on the tensor cores (mma.sync m16n8k16, fp32
//   accumulate) with the int8 codes widened to integer-valued fp16 in registers (exact:
//   |code| <= 127).  S^T = K * Q^T puts the 16 tokens on M and the GQA group (<= 8 heads; a
//   larger group, up to 16, takes the rows path below with its heads as the rows)
//   on N; O^T = V^T * W puts 16 head dimensions on M.  This keeps the FP32 pipe free: at
//   GQA 6 x head_dim 256 a CUDA-core FMA decode needs ~11 us of FMA issue per 68 MB of
//   K/V on GB300, more than the ~10 us the bytes take at the measured HBM rate.
// * Q is bf16, scaled per head by a power of two into fp16 range (exact for bf16 values);
//   the softmax weight W = p * sV of each token is split into fp16 hi + lo parts, two MMAs,
//   so PV keeps ~22 bits.  log2(sV) is folded into a second running maximum so that W
//   stays in [0, 1] whatever the V scales are.
// * Split route: each CTA writes (m_s, m_z, l, acc[D]) per query head; stage 2 merges.
// * Verify rows ([DOT4] "Future Work": MTP verify at nq = 2-4; "ROCm/RDNA4 (gfx1201) vLLM
//   ..." row-shape routing: spec-verify with 2-6 rows): the nq query rows of a sequence
//   join the GQA group on the N side, rows = G * nq (row r = query i * G + head).  A warp
//   holds one 8-row n-tile of S^T and O^T; NT = ceil(rows / 8) warps form a team that shares
//   one page ring, so each K/V page is still read from HBM once for all nq rows ("Redundancy
//   is a currency": the byte-bound decode does not re-stream K per row tile).  A slot is
//   refilled once every warp of its team has arrived on the slot's empty barrier.
// * Fused decode step ("gfx936 ..." §4.2 measures decode together with the producer; §2.2
//   writes the new token's K/V in the producer): with k_new / v_new given, the nq newest
//   tokens of each sequence are quantised (quant_rule.cuh, the kvq_quant_write rule) and
//   written into their page, before its bulk copy, by the warp that will issue that copy (a
//   proxy fence orders the generic stores before the copy's reads).  Only that warp's team
//   reads the page, so no other CTA or launch has to wait for the write; the write sits in the
//   CTA's prologue, off the page loop.  One new token at head_dim 256: the owning warp stores the
//   codes without waiting for them and writes them into its landed shared-memory copy of the
//   page instead (see PATCH below).
#include "decode_stage1.cuh"

namespace kvq {

// The K/V stream of the stage-1 kernel alone (measurement entry point kvq_debug_stream_floor): the
// same grid, the same eight warps with their three-stage rings, the same bulk copies of the same
// pages in the same order, and no arithmetic.  Its duration is what streaming one launch's pages
// costs on this GPU by itself (launch, ramp-up and tail included), the floor of stage 1.
template <int D>
__global__ void __launch_bounds__(256, D == 128 ? 2 : 1) decode_stream_kernel(DecodeArgs a) {
  constexpr int NTEAM = 8, DEPTH = 3;
  using L = DecodeSmem<D, 1, NTEAM, DEPTH>;
  constexpr int KB = L::kKvBytes;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOffset);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.y, b = blockIdx.z;
  grid_dep_wait();
  const int t_begin = static_cast<int>(blockIdx.x) * a.split_rows;
  const int32_t* bt = a.block_table + static_cast<long long>(b) * a.max_blocks_per_seq + t_begin / KVQ_BLOCK_SIZE;
  int pg = -1;
  if (t_begin / KVQ_BLOCK_SIZE + warp + lane * NTEAM < a.max_blocks_per_seq) pg = __ldg(bt + warp + lane * NTEAM);
  const int ctx = max(0, min(a.ctx_lens[b], min(a.max_blocks_per_seq * KVQ_BLOCK_SIZE, a.max_ctx)));
  const int t_end = min(ctx, t_begin + a.split_rows);
  const int n_pages = (t_end > t_begin) ? (t_end - t_begin + KVQ_BLOCK_SIZE - 1) / KVQ_BLOCK_SIZE : 0;
  if (n_pages == 0) return;
  if (threadIdx.x == 0) {
    for (int st = 0; st < L::kStages; ++st) mbar_init(&full[st], 1);
    mbar_fence_init();
  }
  __syncthreads();
  const int npp = (warp < n_pages) ? (n_pages - warp + NTEAM - 1) / NTEAM : 0;
  uint64_t* pfull = full + warp * DEPTH;
  uint8_t* pring = smem + warp * DEPTH * L::kStageBytes;
  if (lane >= npp) pg = -1;
  int wb = 0, n_issued = 0;
  auto issue = [&](int k) {
    while (k >= wb + 32) {
      wb += 32;
      pg = (wb + lane < npp) ? __ldg(bt + warp + (wb + lane) * NTEAM) : -1;
    }
    const int page = __shfl_sync(0xffffffffu, pg, k - wb);
    ++n_issued;
    if (lane == 0) {
      const int st = k % DEPTH;
      if (page >= 0 && page < a.num_blocks) {
        uint8_t* dst = pring + st * L::kStageBytes;
        const long long ph = static_cast<long long>(page) * a.n_kv_heads + kvh;
        mbar_arrive_expect_tx(&pfull[st], 2 * KB + 128);
        bulk_g2s(dst, a.k + ph * KB, KB, &pfull[st]);
        bulk_g2s(dst + KB, a.v + ph * KB, KB, &pfull[st]);
        bulk_g2s(dst + 2 * KB, a.k_scale + ph * KVQ_BLOCK_SIZE, 64, &pfull[st]);
        bulk_g2s(dst + 2 * KB + 64, a.v_scale + ph * KVQ_BLOCK_SIZE, 64, &pfull[st]);
      } else {
        set_status(a.status, KVQ_DEV_BAD_BLOCK);
        mbar_arrive(&pfull[st]);
      }
    }
  };
  for (int k = 0; k < min(DEPTH, npp); ++k) issue(k);
  for (int k = 0; k < npp; ++k) {
    const bool got = mbar_wait(&pfull[k % DEPTH], (k / DEPTH) & 1, a.status, a.wait_budget);
    if (!__all_sync(0xffffffffu, got)) {
      // the copies issued past this page land before the CTA exits
      if (lane == 0)
        for (int kk = k; kk < n_issued; ++kk) mbar_wait(&pfull[kk % DEPTH], (kk / DEPTH) & 1, a.status, a.wait_budget);
      __syncwarp();
      break;
    }
    if (k + DEPTH < npp) issue(k + DEPTH);
  }
}

cudaError_t launch_stream_floor(const DecodeArgs& a, cudaStream_t stream) {
  dim3 grid(a.n_split, a.n_kv_heads, a.batch);
  if (a.head_dim == 256) {
    using L = DecodeSmem<256, 1, 8, 3>;
    cudaError_t e = cudaFuncSetAttribute(decode_stream_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
    if (e != cudaSuccess) return e;
    return launch_pdl(decode_stream_kernel<256>, grid, dim3(256), L::kTotal, stream, a);
  }
  using L = DecodeSmem<128, 1, 8, 3>;
  cudaError_t e = cudaFuncSetAttribute(decode_stream_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_stream_kernel<128>, grid, dim3(256), L::kTotal, stream, a);
}

// Stage 2: log-sum-exp merge of the splits of one (sequence, query row, query head).
//   M_s = max m_s, M_z = max m_z;  l = sum l_s 2^{m_s - M_s};  o = sum acc_s 2^{m_z - M_z};
//   out = o 2^{M_z - M_s} / l.  The per-split weights are computed once into shared memory
// ("ROCm/RDNA4 (gfx1201) vLLM ...", "The reduce is not free": one cooperative pass, each
// exponential once per split).  One CTA per (query head, sequence, 64-dim column block), so that
// a small batch still spreads over many SMs; 256 threads = 16 split groups x 16 threads of 4
// dims; each thread keeps 8 independent loads in flight.
constexpr int kMergeThreads = 256;
constexpr int kMergeCols = 64;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) decode_merge_kernel(DecodeArgs a) {
  constexpr int TPG = kMergeCols / 4;           // threads per split group (4 dims each)
  constexpr int NG = kMergeThreads / TPG;       // split groups
  constexpr int PRE = 8;                        // partials per thread loaded before the weights
  extern __shared__ float wts[];                // [n_split] weights of the partial accumulators
  __shared__ float red[2][kMergeThreads / 32];
  __shared__ __align__(16) float4 part[NG][TPG];
  // blockIdx.y = b * nq + i: query row i of sequence b
  const int h = blockIdx.x, row = blockIdx.y, b = row / a.nq, Hq = a.n_q_heads, col0 = blockIdx.z * kMergeCols;
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
// 64-dim block) CTAs of decode_merge_kernel would take several.  The same rule as that kernel.
constexpr int kMergeWarpMaxSplits = 32;

template <int D>
__global__ void __launch_bounds__(256) decode_merge_warp_kernel(DecodeArgs a) {
  constexpr int PER = D / 32;  // dims per lane
  const int lane = threadIdx.x & 31;
  const int Hq = a.n_q_heads;
  const long long unit = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);  // row * Hq + h
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

size_t decode_workspace_bytes(int batch, int n_q_heads, int max_ctx, int head_dim, int split_rows) {
  const long long n_split = (static_cast<long long>(max_ctx) + split_rows - 1) / split_rows;
  const long long units = static_cast<long long>(batch) * n_q_heads * n_split;
  const long long acc = units * head_dim * 4;
  const long long stats = units * 4 * 4;
  return static_cast<size_t>(((acc + 255) / 256) * 256 + stats);
}

template <int D, bool SPLIT>
static cudaError_t launch_stage1_rows(const DecodeArgs& a, dim3 grid, cudaStream_t stream) {
  if (a.nq == 1 && a.n_q_heads / a.n_kv_heads <= 8) {  // plain decode, or the fused one-token step
    if (a.k_new) return launch_stage1<D, 1, SPLIT, false, true>(a, grid, stream);
    return launch_stage1<D, 1, SPLIT, false, false>(a, grid, stream);
  }
  const int rows = (a.n_q_heads / a.n_kv_heads) * a.nq;
  switch ((rows + 7) / 8) {
    case 1: return launch_stage1<D, 1, SPLIT>(a, grid, stream);
    case 2: return launch_stage1<D, 2, SPLIT>(a, grid, stream);
    case 3: return launch_stage1<D, 3, SPLIT>(a, grid, stream);
    case 4: return launch_stage1<D, 4, SPLIT>(a, grid, stream);
    case 5: return launch_stage1<D, 5, SPLIT>(a, grid, stream);
    case 6: return launch_stage1<D, 6, SPLIT>(a, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_merge(const DecodeArgs& a, cudaStream_t stream) {
  cudaError_t e;
  const long long units = static_cast<long long>(a.batch) * a.nq * a.n_q_heads;
  if (a.n_split <= kMergeWarpMaxSplits && units >= 512) {
    // many units, few splits each: a warp per unit
    const dim3 gw(static_cast<unsigned>((units + 7) / 8));
    e = a.head_dim == 256 ? launch_pdl(decode_merge_warp_kernel<256>, gw, dim3(256), 0, stream, a)
                          : launch_pdl(decode_merge_warp_kernel<128>, gw, dim3(256), 0, stream, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
  }
  const size_t wbytes = static_cast<size_t>(a.n_split) * sizeof(float);
  dim3 g2(a.n_q_heads, a.batch * a.nq, a.head_dim / kMergeCols);
  if (a.head_dim == 256) {
    if (wbytes > 48 * 1024) {
      e = cudaFuncSetAttribute(decode_merge_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(wbytes));
      if (e != cudaSuccess) return e;
    }
    e = launch_pdl(decode_merge_kernel<256>, g2, dim3(kMergeThreads), wbytes, stream, a);
  } else {
    if (wbytes > 48 * 1024) {
      e = cudaFuncSetAttribute(decode_merge_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(wbytes));
      if (e != cudaSuccess) return e;
    }
    e = launch_pdl(decode_merge_kernel<128>, g2, dim3(kMergeThreads), wbytes, stream, a);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_decode(const DecodeArgs& a, DecodeRoute route, cudaStream_t stream, int* launched) {
  *launched = route == DecodeRoute::kSingle ? 1 : 2;
  if (route == DecodeRoute::kSingle) {
    dim3 grid(1, a.n_kv_heads, a.batch);
    if (a.head_dim == 256) return launch_stage1_rows<256, false>(a, grid, stream);
    return launch_stage1_rows<128, false>(a, grid, stream);
  }
  dim3 grid(a.n_split, a.n_kv_heads, a.batch);
  cudaError_t e;
  if (a.head_dim == 256)
    e = launch_stage1_rows<256, true>(a, grid, stream);
  else
    e = launch_stage1_rows<128, true>(a, grid, stream);
  if (e != cudaSuccess) return e;
  return launch_decode_merge(a, stream);
}

}  // namespace kvq
