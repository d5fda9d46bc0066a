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
#include "decode_merge.cuh"
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

template <int D>
__global__ void __launch_bounds__(kMergeThreads) decode_merge_kernel(DecodeArgs a) {
  extern __shared__ float wts[];
  decode_merge_block<D>(a, blockIdx.x, blockIdx.y, blockIdx.z, wts);
}

template <int D>
__global__ void __launch_bounds__(256) decode_merge_warp_kernel(DecodeArgs a) {
  decode_merge_warps<D>(a, blockIdx.x);
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

// Past kMergeSmem bytes of splits' weights the merge has to ask for its shared memory (48 KB less its own arrays are
// free); it does so before stage 1, which may write the cache.
template <int D>
static cudaError_t prepare_merge(const DecodeArgs& a) {
  static std::atomic<uint64_t> done{0};
  if (decode_merge_by_warps(a) || a.n_split * sizeof(float) <= kMergeSmem) return cudaSuccess;
  return allow_smem(reinterpret_cast<const void*>(decode_merge_kernel<D>), kMaxSplits * sizeof(float), done);
}

template <int D>
static cudaError_t launch_decode_merge(const DecodeArgs& a, cudaStream_t stream) {
  const long long units = static_cast<long long>(a.batch) * a.nq * a.n_q_heads;
  cudaError_t e;
  if (decode_merge_by_warps(a)) {
    e = launch_pdl(decode_merge_warp_kernel<D>, dim3(static_cast<unsigned>((units + 7) / 8)), dim3(256), 0, stream, a);
  } else {
    const dim3 g2(a.n_q_heads, a.batch * a.nq, D / kMergeCols);
    e = launch_pdl(decode_merge_kernel<D>, g2, dim3(kMergeThreads), a.n_split * sizeof(float), stream, a);
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
  cudaError_t e = a.head_dim == 256 ? prepare_merge<256>(a) : prepare_merge<128>(a);
  if (e != cudaSuccess) return e;
  e = a.head_dim == 256 ? launch_stage1_rows<256, true>(a, grid, stream) : launch_stage1_rows<128, true>(a, grid, stream);
  if (e != cudaSuccess) return e;
  return a.head_dim == 256 ? launch_decode_merge<256>(a, stream) : launch_decode_merge<128>(a, stream);
}

}  // namespace kvq
