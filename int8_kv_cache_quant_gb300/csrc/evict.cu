// evict.cu — eviction from the paged int8 cache by accumulated attention weight.
//
// Per (sequence, KV head) the cache holds ctx tokens in logical slots 0 .. ctx - 1, each with the
// attention weight that its queries have given it so far (acc) and its position (slot_pos).  Kept are
// `keep` of them: the protected ones (position below n_sink, or among the n_recent newest), then
// those of the largest weight, ties to the lowest slot.  A softmax does not depend on the order of
// its keys, so nothing is compacted in order: the kept tokens that lie in slots at or past `keep`
// (the movers, ascending) go one by one into the slots below it that are given up (the holes,
// ascending).  Sources and destinations never overlap, so all moves run at once and in place, and
// only what has to move is moved.
//
// Two kernels.
// * evict_select_kernel: a cluster of CTAs per (sequence, KV head), each CTA a contiguous range of
//   slots with its order keys in shared memory.  The keep-th largest key is found by a radix select
//   (digits of 11, 11 and 10 bits: a histogram per CTA in shared memory, summed over the cluster
//   through distributed shared memory); then each warp walks its own run of slots with ballots, which
//   gives ties, holes and movers their ranks without a barrier a step.  The weight and position of
//   every slot are read once.
// * evict_move_kernel: a CTA per (page below the budget, KV head, sequence) fills that page's holes.
//   The cache stores V as [dim][16 slots], so a token's V is one byte of every 16: a whole page's
//   rows are rebuilt in registers and stored as 16-byte words.
#include <algorithm>

#include <cooperative_groups.h>

#include "kvq_dev.cuh"
#include "kvq_launch.h"

namespace kvq {

namespace cg = cooperative_groups;

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
// Order keys a CTA keeps in shared memory (64 KB); slots of its range past them are read again.
constexpr int kKeyCap = 16384;

// Order-preserving image of a weight: NaN lowest, then -inf .. +inf (-0 as +0); protected slots are
// 0xFFFFFFFF, above +inf.
__device__ __forceinline__ uint32_t order_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelShared {
  uint32_t hist[2][kBins];
  uint32_t warp_a[kSelWarps], warp_b[kSelWarps];  // per-warp counts
  uint32_t cta_a, cta_b;                          // this CTA's totals, read by the cluster
  int cta_max;
  uint32_t pick_digit, pick_above;
};

// Exclusive prefix of the CTA's warp counts; returns the CTA's total.
__device__ __forceinline__ uint32_t warp_prefix(const uint32_t* counts, int warp, uint32_t& before) {
  uint32_t b = 0, t = 0;
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) {
    const uint32_t v = counts[i];
    if (i < warp) b += v;
    t += v;
  }
  before = b;
  return t;
}

}  // namespace

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), n_cta = static_cast<int>(cluster.num_blocks());
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ SelShared sh;
  extern __shared__ uint32_t keys[];  // [min(range, kKeyCap)]
  grid_dep_wait();
  int ctx = a.ctx_lens[b];
  const int cap = min(a.max_blocks_per_seq > 0x7FFFFFF ? 0x7FFFFFF0 : a.max_blocks_per_seq * KVQ_BLOCK_SIZE, a.max_ctx);
  if (ctx > cap) {
    if (tid == 0 && rank == 0) set_status(a.status, KVQ_DEV_BAD_POS);
    ctx = cap;
  }
  if (ctx < 0) ctx = 0;
  const int keep = a.keep, new_len = min(ctx, keep);
  const long long unit = static_cast<long long>(b) * a.n_kv_heads + kvh;
  const float* acc = a.acc + unit * a.acc_stride;
  const int32_t* pos = a.slot_pos + unit * a.acc_stride;
  float* acc_out = a.acc_out + unit * a.out_stride;
  int32_t* pos_out = a.slot_pos_out + unit * a.out_stride;
  const bool in_place = a.acc_out == a.acc;
  if (kvh == 0 && rank == 0 && tid == 0) a.new_lens[b] = new_len;
  if (ctx <= keep) {  // nothing goes (the same in every CTA of the cluster)
    if (rank == 0 && tid == 0) a.n_moves[unit] = 0;
    if (!in_place)
      for (int t = rank * kSelThreads + tid; t < ctx; t += n_cta * kSelThreads) {
        acc_out[t] = acc[t];
        pos_out[t] = pos[t];
      }
    return;
  }
  // This CTA's slots [t0, t1), and each warp's run of them (whole ballots of 32, whole pages).
  const int range = ((ctx + n_cta - 1) / n_cta + 31) / 32 * 32;
  const int t0 = min(ctx, rank * range), t1 = min(ctx, t0 + range);
  const int run = ((range + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(t1, t0 + warp * run), w1 = min(t1, w0 + run);

  // ---- the newest position, then the order keys
  int pmax = INT32_MIN;
  for (int t = t0 + tid; t < t1; t += kSelThreads) pmax = max(pmax, pos[t]);
  pmax = __reduce_max_sync(0xffffffffu, pmax);
  if (tid == 0) sh.cta_max = INT32_MIN;
  for (int i = tid; i < 2 * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0u;
  __syncthreads();
  if (lane == 0) atomicMax(&sh.cta_max, pmax);
  cluster.sync();
  for (int r = 0; r < n_cta; ++r) pmax = max(pmax, *cluster.map_shared_rank(&sh.cta_max, r));
  const long long recent_from = static_cast<long long>(pmax) - a.n_recent;  // protected above it
  auto make_key = [&](int t) {
    const int p = pos[t];
    return (p < a.n_sink || p > recent_from) ? 0xFFFFFFFFu : order_key(acc[t]);
  };
  for (int t = t0 + tid; t < t1; t += kSelThreads) {
    const uint32_t k = make_key(t);
    if (t - t0 < kKeyCap) keys[t - t0] = k;
    atomicAdd(&sh.hist[0][k >> 21], 1u);
  }
  auto key_of = [&](int t) { return t - t0 < kKeyCap ? keys[t - t0] : make_key(t); };

  // ---- radix select: the prefix of the keep-th largest key, digit by digit
  uint32_t prefix = 0, need = static_cast<uint32_t>(keep);  // still wanted among keys that start with prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    uint32_t* hist = sh.hist[pass & 1];
    cluster.sync();  // every CTA's histogram of this digit is complete
    // bins 4 tid .. 4 tid + 3, from the top: sums over the cluster, suffix sums over the CTA
    uint32_t bin[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = kBins - 1 - (4 * tid + i);
      uint32_t v = 0;
      for (int r = 0; r < n_cta; ++r) v += cluster.map_shared_rank(hist, r)[d];
      bin[i] = v;
      sum += v;
    }
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) sh.warp_a[warp] = incl;
    __syncthreads();
    uint32_t before;
    warp_prefix(sh.warp_a, warp, before);
    uint32_t above = before + incl - sum;  // keys in higher bins than this thread's first
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (above < need && need <= above + bin[i]) {
        sh.pick_digit = kBins - 1 - (4 * tid + i);
        sh.pick_above = above;
      }
      above += bin[i];
    }
    __syncthreads();
    const uint32_t digit = sh.pick_digit;
    need -= sh.pick_above;
    prefix |= digit << shift;
    if (pass == 2) break;
    // the next digit's histogram, of the keys that share the prefix
    uint32_t* next = sh.hist[(pass + 1) & 1];
    if (pass == 1) {  // its buffer held the first digit, which every CTA read before the last cluster barrier
      for (int i = tid; i < kBins; i += kSelThreads) next[i] = 0u;
      __syncthreads();
    }
    for (int t = t0 + tid; t < t1; t += kSelThreads) {
      const uint32_t k = key_of(t);
      if ((k >> shift) == (prefix >> shift)) atomicAdd(&next[pass == 0 ? (k >> 10) & 2047u : k & 1023u], 1u);
    }
  }
  const uint32_t thr = prefix;  // kept: keys above thr, and the first `need` that equal it

  // ---- ranks of the ties, in slot order: over the warp's run, the CTA, the cluster
  uint32_t ties = 0;
  for (int t = w0 + lane; t - lane < w1; t += 32)
    ties += __popc(__ballot_sync(0xffffffffu, t < w1 && key_of(t) == thr));
  if (lane == 0) sh.warp_b[warp] = ties;
  __syncthreads();
  uint32_t tie_before;
  const uint32_t cta_ties = warp_prefix(sh.warp_b, warp, tie_before);
  if (tid == 0) sh.cta_a = cta_ties;
  cluster.sync();
  for (int r = 0; r < rank; ++r) tie_before += *cluster.map_shared_rank(&sh.cta_a, r);

  // ---- kept or not, and the counts of holes (below keep) and movers (at or past it) of the run
  const uint32_t lt = (1u << lane) - 1u;
  auto walk = [&](auto&& visit) {
    uint32_t tb = tie_before;
    for (int t = w0 + lane; t - lane < w1; t += 32) {
      const bool live = t < w1;
      const uint32_t k = live ? key_of(t) : 0u;
      const bool tie = live && k == thr;
      const uint32_t tm = __ballot_sync(0xffffffffu, tie);
      const bool kept = live && (k > thr || (tie && tb + __popc(tm & lt) < need));
      tb += __popc(tm);
      visit(t, live, kept);
    }
  };
  uint32_t holes = 0, movers = 0;
  walk([&](int t, bool live, bool kept) {
    holes += __popc(__ballot_sync(0xffffffffu, live && !kept && t < keep));
    movers += __popc(__ballot_sync(0xffffffffu, kept && t >= keep));
  });
  __syncthreads();  // warp_a, warp_b are free again
  if (lane == 0) {
    sh.warp_a[warp] = holes;
    sh.warp_b[warp] = movers;
  }
  __syncthreads();
  uint32_t hole_at, mover_at;
  const uint32_t cta_holes = warp_prefix(sh.warp_a, warp, hole_at), cta_movers = warp_prefix(sh.warp_b, warp, mover_at);
  cluster.sync();  // every CTA has read the tie counts
  if (tid == 0) {
    sh.cta_a = cta_holes;
    sh.cta_b = cta_movers;
  }
  cluster.sync();
  uint32_t total = 0;
  for (int r = 0; r < n_cta; ++r) {
    const uint32_t h = *cluster.map_shared_rank(&sh.cta_a, r);
    if (r < rank) {
      hole_at += h;
      mover_at += *cluster.map_shared_rank(&sh.cta_b, r);
    }
    total += h;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory

  // ---- the lists, the first hole of every page, and what stays where it is
  int32_t* src = a.move_src + unit * a.max_moves;
  int32_t* dst = a.move_dst + unit * a.max_moves;
  int32_t* first = a.page_first + unit * a.n_pages;
  if (rank == 0 && tid == 0) a.n_moves[unit] = static_cast<int32_t>(total);
  walk([&](int t, bool live, bool kept) {
    const bool hole = live && !kept && t < keep, mover = kept && t >= keep;
    const uint32_t hm = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
    if (hole) dst[hole_at + __popc(hm & lt)] = t;
    if (mover) src[mover_at + __popc(mm & lt)] = t;
    if (live && t < keep && t % KVQ_BLOCK_SIZE == 0) first[t / KVQ_BLOCK_SIZE] = static_cast<int32_t>(hole_at + __popc(hm & lt));
    if (kept && t < keep && !in_place) {
      acc_out[t] = acc[t];
      pos_out[t] = pos[t];
    }
    hole_at += __popc(hm);
    mover_at += __popc(mm);
  });
}

// The moves into one page below the budget.  Holes of the page are entries page_first[p] .. up to the
// next page's first; their movers are the same entries of move_src.
template <int D>
__global__ void __launch_bounds__(D) evict_move_kernel(EvictArgs a) {
  const int p = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  __shared__ long long src_ph[KVQ_BLOCK_SIZE];  // source page * n_kv_heads + kvh, -1: none
  __shared__ int src_slot[KVQ_BLOCK_SIZE];      // by destination slot
  grid_dep_wait();
  const long long unit = static_cast<long long>(b) * a.n_kv_heads + kvh;
  const int total = a.n_moves[unit];
  if (total == 0) return;
  const int32_t* first = a.page_first + unit * a.n_pages;
  const int j0 = first[p], j1 = p + 1 < a.n_pages ? first[p + 1] : total;
  if (j0 == j1) return;
  const int32_t* bt = a.block_table + static_cast<long long>(b) * a.max_blocks_per_seq;
  const int dpage = bt[p];
  const bool dst_ok = dpage >= 0 && dpage < a.num_blocks;
  const long long dph = static_cast<long long>(dpage) * a.n_kv_heads + kvh;
  if (tid < KVQ_BLOCK_SIZE) src_ph[tid] = -1;
  __syncthreads();
  if (tid < j1 - j0) {
    const int s = a.move_src[unit * a.max_moves + j0 + tid], t = a.move_dst[unit * a.max_moves + j0 + tid];
    const int page = bt[s / KVQ_BLOCK_SIZE];
    const bool ok = dst_ok && page >= 0 && page < a.num_blocks;
    if (!ok) set_status(a.status, KVQ_DEV_BAD_BLOCK);
    const long long ph = static_cast<long long>(page) * a.n_kv_heads + kvh;
    src_ph[t % KVQ_BLOCK_SIZE] = ok ? ph : -1;
    src_slot[t % KVQ_BLOCK_SIZE] = s % KVQ_BLOCK_SIZE;
    if (ok) {
      const int so = s % KVQ_BLOCK_SIZE, dz = t % KVQ_BLOCK_SIZE;
      a.k_scale[dph * KVQ_BLOCK_SIZE + dz] = a.k_scale[ph * KVQ_BLOCK_SIZE + so];
      a.v_scale[dph * KVQ_BLOCK_SIZE + dz] = a.v_scale[ph * KVQ_BLOCK_SIZE + so];
    }
    a.acc_out[unit * a.out_stride + t] = a.acc[unit * a.acc_stride + s];
    a.slot_pos_out[unit * a.out_stride + t] = a.slot_pos[unit * a.acc_stride + s];
  }
  __syncthreads();
  if (!dst_ok) return;
  // K: a token's chunk of 16 dims is one 16-byte word
  for (int i = tid; i < KVQ_BLOCK_SIZE * (D / 16); i += D) {
    const int slot = i % KVQ_BLOCK_SIZE, ch = i / KVQ_BLOCK_SIZE;
    const long long ph = src_ph[slot];
    if (ph >= 0)
      *reinterpret_cast<uint4*>(a.k + ((dph * (D / 16) + ch) * KVQ_BLOCK_SIZE + slot) * 16) =
          *reinterpret_cast<const uint4*>(a.k + ((ph * (D / 16) + ch) * KVQ_BLOCK_SIZE + src_slot[slot]) * 16);
  }
  // V: thread = dim; its 16 slots are one 16-byte word, into which the movers' bytes go
  uint4* row = reinterpret_cast<uint4*>(a.v + (dph * D + tid) * KVQ_BLOCK_SIZE);
  uint4 w = *row;
  uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int slot = 0; slot < KVQ_BLOCK_SIZE; ++slot) {
    const long long ph = src_ph[slot];
    if (ph >= 0) {
      const uint32_t byte = static_cast<uint8_t>(a.v[(ph * D + tid) * KVQ_BLOCK_SIZE + src_slot[slot]]);
      const uint32_t sh = 8u * (slot % 4);
      word[slot / 4] = (word[slot / 4] & ~(0xFFu << sh)) | (byte << sh);
    }
  }
  *row = make_uint4(word[0], word[1], word[2], word[3]);
}

// CTAs of a select cluster: as many (1, 2, 4 or 8) as keep at least 1024 slots each and all clusters
// in one wave of the SMs.
static int select_cluster(const EvictArgs& a, int n_sms) {
  const long long units = static_cast<long long>(a.batch) * a.n_kv_heads;
  int c = 1;
  while (c < kMaxCluster && units * (2 * c) <= n_sms && a.max_ctx / (2 * c) >= 1024) c *= 2;
  return c;
}

EvictWorkspace evict_workspace(int batch, int n_kv_heads, int max_ctx, int keep) {
  EvictWorkspace w{};
  const long long units = static_cast<long long>(batch) * n_kv_heads;
  w.max_moves = max_ctx > keep ? std::min(keep, max_ctx - keep) : 0;
  w.n_pages = max_ctx > keep ? (keep + KVQ_BLOCK_SIZE - 1) / KVQ_BLOCK_SIZE : 0;
  w.off_dst = (units * w.max_moves * 4 + 255) / 256 * 256;
  w.off_first = 2 * w.off_dst;
  w.off_count = w.off_first + (units * w.n_pages * 4 + 255) / 256 * 256;
  w.bytes = w.off_count + units * 4;
  return w;
}

cudaError_t launch_evict(const EvictArgs& a, int n_sms, cudaStream_t stream) {
  const int c = select_cluster(a, n_sms);
  const int range = ((a.max_ctx + c - 1) / c + 31) / 32 * 32;
  const size_t smem = static_cast<size_t>(std::min(range, kKeyCap)) * 4;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyCap * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c, a.n_kv_heads, a.batch);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if ((e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a)) != cudaSuccess) return e;
  if (a.max_moves == 0) return cudaSuccess;
  const dim3 grid(a.n_pages, a.n_kv_heads, a.batch);
  return a.head_dim == 256 ? launch_pdl(evict_move_kernel<256>, grid, dim3(256), 0, stream, a)
                           : launch_pdl(evict_move_kernel<128>, grid, dim3(128), 0, stream, a);
}

}  // namespace kvq
