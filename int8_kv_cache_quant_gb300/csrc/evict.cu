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
//   (digits of 8 bits): a histogram per CTA in shared memory, the bins that are not zero pushed into
//   every other CTA's total, and each warp finding the digit by itself, so that a digit costs one
//   barrier.  Once 256 keys or fewer start with the prefix (two digits of most real weights), every CTA
//   gets them all and finds the last that stays by comparing them with each other, ties included.
//   Then each warp walks its run of slots with ballots and leaves which are kept, as bits, with the
//   holes or movers before each 32; after that any thread can take any slot, and the dependent loads of
//   the moves overlap.  The kernel also moves weights and positions, and leaves for every slot below
//   the budget the physical slot that moves into it, if any.
// * evict_move_kernel: a CTA per (page below the budget, KV head, sequence) fills that page's holes.
//   The cache stores V as [dim][16 slots], so a token's V is one byte of every 16: a whole page's
//   rows are rebuilt in registers and stored as 16-byte words.
// When few tokens can move (a serving batch that evicts a token a step, or some hundreds every now and
// then), the select kernel's warps move the codes too (FEW), and the second launch falls away.
//
// Bound.  One sequence: the chain of barriers and dependent loads (32768 to 4096 in 4 heads: 30 us, the select
// kernel 19 on 32 SMs; 1025 to 1024 in 8 x 8: 6.6 us with a max_ctx of at most 1152, 12.5 from 2048 on, where the
// host's bound leaves room for many moves).  A large batch: select about half its issue slots, move the
// sectors of the layout, in which a token's V is a byte of every 16: 64 x 8 of up to 16384 to 2048 moves 1.12 GB
// of sectors for 0.41 GB of tokens, about 175 us at 6.4 TB/s, select 71 us.
#include <algorithm>
#include <type_traits>
#include <utility>

#include <cooperative_groups.h>

#include "kvq_dev.cuh"
#include "kvq_launch.h"

namespace kvq {

namespace cg = cooperative_groups;

namespace {

// 256 | 512 | 1024 threads: 330 | 285 | 299 us at 64 x 8 of up to 16384, 43 | 36 | 39 at 1 x 4 of 32768.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kDigits = 4;
constexpr int kMaxCluster = 8;
// Order keys a CTA keeps in shared memory (64 KB); slots of its range past them are read again.
constexpr int kKeyCap = 16384;
constexpr int kPosRegs = 8;  // positions a thread keeps in registers between their maximum and the keys
// Tokens of a (sequence, KV head) that the select kernel moves itself at most, for a batch of fewer units than
// SMs and for a larger one.  A warp's move of a token costs little but its sectors; the page kernel
// reads and writes every page below the budget, but uses all SMs and whole words.  Measured (select kernel |
// page kernel, us): 8 sequences x 8 heads of 1024 tokens, 64 moves 10.9 | 13.8, 128 15.7 | 16.7, 256 20.4 | 17.2; 1 x 4 of
// 4096: 64 12.7 | 13.7, 128 14.6 | 14.4, 256 18.9 | 15.6; 64 x 8 of 2048: 16 25 | 57, 256 87 | 126, 512 125 | 140,
// 1024 176 | 149.
constexpr int kFewMoves = 128, kFewMovesLarge = 512;
constexpr int kBatch = 4;  // slots a thread has in flight
constexpr int kCands = 256;  // keys that are compared with each other
// What the move kernel finds for a slot below the budget: the physical slot (page * 16 + slot) that
// moves into it, or one of these.
constexpr int32_t kStays = -1, kBadMove = -2;

// Order-preserving image of a weight: NaN lowest, then -inf .. +inf (-0 as +0); protected slots are
// 0xFFFFFFFF, above +inf.
__device__ __forceinline__ uint32_t order_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <bool FEW>
struct SelShared {
  uint32_t own[kDigits][256];    // this CTA's histograms
  uint32_t total[kDigits][256];  // the cluster's
  uint32_t warp_a[kSelWarps], warp_b[kSelWarps];
  uint32_t ties[kMaxCluster], holes[kMaxCluster], movers[kMaxCluster];  // by rank, pushed by each CTA
  int newest[kMaxCluster];                     // by rank
  int n_cand, cand_base, thr_slot;
  uint32_t n_cands, thr_key;
  unsigned long long own_cand[kCands], cand[kCands];  // this CTA's, the cluster's: the keys that the last selection is among, with ~slot below
  int n_few;
  int2 few[FEW ? kFewMovesLarge : 1];  // FEW: this CTA's moves, from and to
};
static_assert(2 * (kKeyCap / 32) <= kDigits * 256, "a CTA's kept bits and ranks fit in place of its histograms");

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

// hist[digit] += 1 for every lane with `in`, N digits a lane (all in flight together).  Lanes with the first
// one's digit add once: equal weights are common, and 32 additions to one bin would run one after another.
template <int N>
__device__ __forceinline__ void count_digits(uint32_t* hist, const uint32_t (&digit)[N], const bool (&in)[N], int lane) {
  int leader[N];
  uint32_t first[N], same[N];
#pragma unroll
  for (int i = 0; i < N; ++i) leader[i] = __ffs(__ballot_sync(0xffffffffu, in[i])) - 1;
#pragma unroll
  for (int i = 0; i < N; ++i) first[i] = __shfl_sync(0xffffffffu, digit[i], leader[i] & 31);
#pragma unroll
  for (int i = 0; i < N; ++i) same[i] = __ballot_sync(0xffffffffu, in[i] && digit[i] == first[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool leads = lane == leader[i];
    if (leads || (in[i] && digit[i] != first[i])) atomicAdd(hist + digit[i], leads ? __popc(same[i]) : 1);
  }
}

// One token's codes and scales, slot s to slot t of the sequence (a warp).
__device__ __forceinline__ void move_token(const EvictArgs& a, const int32_t* bt, int kvh, int s, int t, int lane) {
  const int sp = bt[s / KVQ_BLOCK_SIZE], dp = bt[t / KVQ_BLOCK_SIZE];
  if (sp < 0 || sp >= a.num_blocks || dp < 0 || dp >= a.num_blocks) {
    if (lane == 0) set_status(a.status, KVQ_DEV_BAD_BLOCK);
    return;
  }
  const int D = a.head_dim, so = s % KVQ_BLOCK_SIZE, to = t % KVQ_BLOCK_SIZE;
  const long long sph = static_cast<long long>(sp) * a.n_kv_heads + kvh, dph = static_cast<long long>(dp) * a.n_kv_heads + kvh;
  // every load before the first store: K 16 dims a lane, V bytes of dims lane, lane + 32, ..
  uint4 kc = make_uint4(0, 0, 0, 0);
  if (lane < D / 16) kc = *reinterpret_cast<const uint4*>(a.k + ((sph * (D / 16) + lane) * KVQ_BLOCK_SIZE + so) * 16);
  int8_t vb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < D / 32) vb[i] = a.v[(sph * D + lane + 32 * i) * KVQ_BLOCK_SIZE + so];
  float sc = 0.f;
  if (lane < 2) sc = (lane ? a.v_scale : a.k_scale)[sph * KVQ_BLOCK_SIZE + so];
  if (lane < D / 16) *reinterpret_cast<uint4*>(a.k + ((dph * (D / 16) + lane) * KVQ_BLOCK_SIZE + to) * 16) = kc;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < D / 32) a.v[(dph * D + lane + 32 * i) * KVQ_BLOCK_SIZE + to] = vb[i];
  if (lane < 2) (lane ? a.v_scale : a.k_scale)[dph * KVQ_BLOCK_SIZE + to] = sc;
}

}  // namespace

// FEW: few tokens can move (kFewMovesLarge at most); the codes are moved here.
template <bool FEW>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(EvictArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), n_cta = static_cast<int>(cluster.num_blocks());
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ SelShared<FEW> sh;
  extern __shared__ __align__(16) uint32_t keys[];  // [min(range, kKeyCap)]
  auto barrier = [&] {  // of the cluster
    if (n_cta > 1) cluster.sync();
    else __syncthreads();
  };
  auto peer = [&](auto* p, int r) { return cluster.map_shared_rank(p, r); };
  grid_dep_wait();
  grid_dep_trigger();
  int ctx = a.ctx_lens[b];
  const int cap = static_cast<int>(min(static_cast<long long>(a.max_blocks_per_seq) * KVQ_BLOCK_SIZE, static_cast<long long>(a.max_ctx)));
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
  const int32_t* bt = a.block_table + static_cast<long long>(b) * a.max_blocks_per_seq;
  const bool in_place = a.acc_out == a.acc;
  if (kvh == 0 && rank == 0 && tid == 0) a.new_lens[b] = new_len;
  if (rank == 0 && tid == 0) a.n_moves[unit] = ctx > keep;  // read by the move kernel: anything to do
  if (ctx <= keep) {  // nothing goes (the same in every CTA of the cluster)
    if (!in_place)
      for (int t = rank * kSelThreads + tid; t < ctx; t += n_cta * kSelThreads) {
        acc_out[t] = acc[t];
        pos_out[t] = pos[t];
      }
    return;
  }
  cg::cluster_group::arrival_token started{};
  if (n_cta > 1) started = cluster.barrier_arrive();
  // This CTA's slots [t0, t1), and each warp's run of them (whole ballots of 32, whole pages).
  const int range = ((ctx + n_cta - 1) / n_cta + 31) / 32 * 32;
  const int t0 = min(ctx, rank * range), t1 = min(ctx, t0 + range);
  const int run = ((range + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(t1, t0 + warp * run), w1 = min(t1, w0 + run);

  // ---- positions and weights, the newest position
  const bool in_regs = range <= kPosRegs * kSelThreads;  // the same in every CTA
  int32_t p_reg[kPosRegs];
  float w_reg[kPosRegs];
  int pmax = INT32_MIN;
  auto load = [&](int from) {  // kPosRegs of the thread's slots, from `from` on, all in flight at once
#pragma unroll
    for (int i = 0; i < kPosRegs; ++i) {
      const int t = from + tid + i * kSelThreads;
      if (t < t1) {
        p_reg[i] = pos[t];
        w_reg[i] = acc[t];
      }
    }
  };
  if (in_regs) {
    load(t0);
#pragma unroll
    for (int i = 0; i < kPosRegs; ++i)
      if (t0 + tid + i * kSelThreads < t1) pmax = max(pmax, p_reg[i]);
  } else {
#pragma unroll 8
    for (int t = t0 + tid; t < t1; t += kSelThreads) pmax = max(pmax, pos[t]);
  }
  pmax = __reduce_max_sync(0xffffffffu, pmax);
  if (lane == 0) sh.warp_a[warp] = static_cast<uint32_t>(pmax);
  if (tid == 0) sh.n_few = sh.n_cand = 0, sh.n_cands = 0;
  for (int i = tid; i < 2 * kDigits * 256; i += kSelThreads) (&sh.own[0][0])[i] = 0u;
  __syncthreads();
  int newest = INT32_MIN;
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) newest = max(newest, static_cast<int>(sh.warp_a[i]));
  if (n_cta > 1) {
    cluster.barrier_wait(std::move(started));  // every CTA of the cluster runs
    if (tid < n_cta) *peer(&sh.newest[rank], tid) = newest;
    cluster.sync();
    for (int r = 0; r < n_cta; ++r) newest = max(newest, sh.newest[r]);
  }
  const long long recent_from = static_cast<long long>(newest) - a.n_recent;  // protected above it
  auto key_from = [&](int p, float w) { return (p < a.n_sink || p > recent_from) ? 0xFFFFFFFFu : order_key(w); };
  const bool in_smem = range <= kKeyCap;
  auto key_of = [&](int t) { return t - t0 < kKeyCap ? keys[t - t0] : key_from(pos[t], acc[t]); };

  // ---- order keys, and the first digit's histogram
  for (int from = t0; from < t1; from += kPosRegs * kSelThreads) {
    if (!in_regs) load(from);
#pragma unroll
    for (int i0 = 0; i0 < kPosRegs; i0 += 4) {
      if (from + warp * 32 + i0 * kSelThreads >= t1) break;  // the same for a warp's lanes
      uint32_t digit[4];
      bool in[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = from + tid + (i0 + i) * kSelThreads;
        in[i] = t < t1;
        const uint32_t k = in[i] ? key_from(p_reg[i0 + i], w_reg[i0 + i]) : 0u;
        if (in[i] && t - t0 < kKeyCap) keys[t - t0] = k;
        digit[i] = k >> 24;
      }
      count_digits(sh.own[0], digit, in, lane);
    }
  }

  // ---- radix select: the prefix of the keep-th largest key, digit by digit
  uint32_t prefix = 0, need = static_cast<uint32_t>(keep);  // still wanted among keys that start with prefix
  uint32_t equal = 0;                                       // keys that do
  bool chosen = false;                                      // the last key kept is known, with its slot
#pragma unroll 1
  for (int d = 0; d < kDigits; ++d) {
    const uint32_t* hist = sh.own[d];
    __syncthreads();
    if (n_cta > 1) {
      for (int i = tid; i < 256 * n_cta; i += kSelThreads) {
        const uint32_t v = sh.own[d][i & 255];
        if (v) atomicAdd(peer(&sh.total[d][i & 255], i >> 8), v);
      }
      cluster.sync();
      hist = sh.total[d];
    }
    // every warp: lane l has bins 255 - 8 l down to 248 - 8 l
    uint32_t bin[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bin[i] = hist[255 - 8 * lane - i];
      sum += bin[i];
    }
    uint32_t above = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, above, off);
      if (lane >= off) above += o;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, above >= need);
    above -= sum;  // keys in the bins above this lane's
    const int l = __ffs(here) - 1;  // the lane whose bins hold the keep-th key
    uint32_t digit = 0, left = need, count = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!found && need <= above + bin[i]) {
        found = true;
        digit = 255 - 8 * lane - i;
        left = need - above;
        count = bin[i];
      }
      above += bin[i];
    }
    digit = __shfl_sync(0xffffffffu, digit, l);
    need = __shfl_sync(0xffffffffu, left, l);
    equal = __shfl_sync(0xffffffffu, count, l);
    const int shift = 24 - 8 * d;
    prefix |= digit << shift;
    if (d + 1 == kDigits || equal == need) break;
    auto starts = [&](uint32_t k) { return (k >> shift) == (prefix >> shift); };
    chosen = equal <= kCands;  // few keys left: they are compared with each other
    auto scan = [&](auto&& visit) {  // visit(keys, first slot, is it one of them) for four keys a lane
      if (in_smem) {
        for (int i0 = 128 * warp; i0 < t1 - t0; i0 += 4 * kSelThreads) {
          const int i = i0 + 4 * lane, n = t1 - t0 - i;
          const uint4 q = n > 0 ? *reinterpret_cast<const uint4*>(keys + i) : make_uint4(0, 0, 0, 0);
          const uint32_t k[4] = {q.x, q.y, q.z, q.w};
          const bool in[4] = {n > 0 && starts(q.x), n > 1 && starts(q.y), n > 2 && starts(q.z), n > 3 && starts(q.w)};
          if (__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) visit(k, t0 + i, in);
        }
      } else {
        for (int i0 = 128 * warp; i0 < t1 - t0; i0 += 4 * kSelThreads) {
          const int t = t0 + i0 + 4 * lane;
          uint32_t k[4];
          bool in[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            k[i] = t + i < t1 ? key_of(t + i) : 0u;
            in[i] = t + i < t1 && starts(k[i]);
          }
          visit(k, t, in);
        }
      }
    };
    if (chosen) {
      scan([&](const uint32_t (&k)[4], int t, const bool (&in)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (in[i]) sh.own_cand[atomicAdd(&sh.n_cand, 1)] = static_cast<unsigned long long>(k[i]) << 32 | ~static_cast<uint32_t>(t + i);
      });
      break;
    }
    scan([&](const uint32_t (&k)[4], int, const bool (&in)[4]) {
      uint32_t digit[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) digit[i] = (k[i] >> (shift - 8)) & 255u;
      count_digits(sh.own[d + 1], digit, in, lane);
    });
  }
  // Kept: keys above thr, and those that are thr up to slot thr_slot (chosen), or the first `need` of the
  // `equal` that are thr.
  uint32_t thr = prefix;
  int thr_slot = INT32_MAX;
  if (chosen) {
    // Every CTA gets all of them (key, and ~slot so that the lower of equal keys is the larger), in no
    // particular order: the one with need - 1 above it is the last that stays.
    __syncthreads();
    const int mine = sh.n_cand;
    if (n_cta > 1) {
      if (tid == 0 && mine) sh.cand_base = static_cast<int>(atomicAdd(peer(&sh.n_cands, 0), static_cast<uint32_t>(mine)));
      __syncthreads();
      for (int i = tid; i < mine * n_cta; i += kSelThreads) *peer(&sh.cand[sh.cand_base + i / n_cta], i % n_cta) = sh.own_cand[i / n_cta];
      cluster.sync();
    }
    const unsigned long long* cand = n_cta > 1 ? sh.cand : sh.own_cand;
    if (tid < static_cast<int>(equal)) {
      const unsigned long long c = cand[tid];
      uint32_t above = 0;
#pragma unroll 8
      for (uint32_t i = 0; i < equal; ++i) above += cand[i] > c;
      if (above == need - 1) {
        sh.thr_key = static_cast<uint32_t>(c >> 32);
        sh.thr_slot = static_cast<int>(~static_cast<uint32_t>(c));
      }
    }
    __syncthreads();
    thr = sh.thr_key;
    thr_slot = sh.thr_slot;
  }

  // ---- ranks of the ties, in slot order: over the warp's run, the CTA, the cluster (when some of them go)
  uint32_t tie_before = 0;
  const bool count_ties = equal != need && !chosen;
  if (count_ties) {
    uint32_t ties = 0;
    for (int t = w0 + lane; t - lane < w1; t += 32)
      ties += __popc(__ballot_sync(0xffffffffu, t < w1 && key_of(t) == thr));
    if (lane == 0) sh.warp_a[warp] = ties;
    __syncthreads();
    const uint32_t cta_ties = warp_prefix(sh.warp_a, warp, tie_before);
    if (n_cta > 1) {
      if (tid < n_cta) *peer(&sh.ties[rank], tid) = cta_ties;
      cluster.sync();
      for (int r = 0; r < rank; ++r) tie_before += sh.ties[r];
    } else {
      __syncthreads();  // warp_a is free again
    }
  }

  // ---- kept or not, as bits, with the holes (below keep) or movers (at or past it) before each word of 32
  // slots: first in the warp's run, then in the sequence
  uint32_t* kept_bits = n_cta > 1 ? &sh.own[0][0] : &sh.total[0][0];  // histograms that are not read any more
  uint32_t* ranks = kept_bits + kKeyCap / 32;
  if (!in_smem) {
    kept_bits = a.words + (unit * a.n_words + t0 / 32) * 2;
    ranks = kept_bits + (t1 - t0 + 31) / 32;
  }
  const uint32_t lt = (1u << lane) - 1u;
  uint32_t holes = 0, movers = 0;
  auto mark = [&](auto keys_near, auto some_ties_go) {
#pragma unroll 4
    for (int t = w0 + lane; t - lane < w1; t += 32) {
      const bool live = t < w1;
      const uint32_t k = !live ? 0u : keys_near.value ? keys[t - t0] : key_of(t);
      bool keeps = live && (k > thr || (k == thr && t <= thr_slot));
      if (some_ties_go.value) {
        const uint32_t tm = __ballot_sync(0xffffffffu, live && k == thr);
        keeps = keeps && (k > thr || tie_before + __popc(tm & lt) < need);
        tie_before += __popc(tm);
      }
      const uint32_t kept = __ballot_sync(0xffffffffu, keeps);
      if (lane == 0) {
        kept_bits[(t - t0) / 32] = kept;
        ranks[(t - t0) / 32] = t < keep ? holes : movers;
      }
      const int below = min(32, max(0, keep - (t - lane)));  // slots of the word below keep
      const uint32_t bm = below == 32 ? 0xffffffffu : (1u << below) - 1u;
      holes += below - __popc(kept & bm);  // ctx > keep: slots below keep all live
      movers += __popc(kept & ~bm);
    }
  };
  using std::false_type;
  using std::true_type;
  if (in_smem && !count_ties) mark(true_type{}, false_type{});
  else if (in_smem) mark(true_type{}, true_type{});
  else if (!count_ties) mark(false_type{}, false_type{});
  else mark(false_type{}, true_type{});
  if (lane == 0) {
    sh.warp_a[warp] = holes;
    sh.warp_b[warp] = movers;
  }
  __syncthreads();
  uint32_t hole_at, mover_at;
  const uint32_t cta_holes = warp_prefix(sh.warp_a, warp, hole_at), cta_movers = warp_prefix(sh.warp_b, warp, mover_at);
  if (n_cta > 1) {
    if (tid < n_cta) {
      *peer(&sh.holes[rank], tid) = cta_holes;
      *peer(&sh.movers[rank], tid) = cta_movers;
    }
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
      hole_at += sh.holes[r];
      mover_at += sh.movers[r];
    }
  }
  for (int t = w0 + 32 * lane; t < w1; t += 32 * 32) ranks[(t - t0) / 32] += t < keep ? hole_at : mover_at;
  __syncthreads();

  // ---- the movers, by rank; then each hole takes the mover of its rank.  Any thread can take any slot now.
  int32_t* src = a.move_src + unit * a.max_moves;
  int32_t* map = a.slot_map + unit * a.n_pages * KVQ_BLOCK_SIZE;
#pragma unroll 4
  for (int t = max(t0, keep / 32 * 32) + tid; t < t1; t += kSelThreads) {
    const int w = (t - t0) / 32, base = t / 32 * 32;
    const uint32_t bits = kept_bits[w];
    const uint32_t past = base < keep ? ~((1u << (keep - base)) - 1u) : 0xffffffffu;  // of a word across keep
    if (t >= keep && ((bits >> lane) & 1u)) src[(base < keep ? 0u : ranks[w]) + __popc(bits & past & lt)] = t;
  }
  barrier();  // no CTA touches another's shared memory after this one
  const int h1 = min(t1, keep);
  for (int tb = t0 + tid; tb < h1; tb += kBatch * kSelThreads) {
    int s[kBatch], page[kBatch], p[kBatch];  // s: the slot that comes here (the slot itself: it stays)
    float w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = tb + i * kSelThreads;
      s[i] = t;
      if (t < h1) {
        const uint32_t bits = kept_bits[(t - t0) / 32];
        if (!((bits >> lane) & 1u)) s[i] = src[ranks[(t - t0) / 32] + __popc(~bits & lt)];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = tb + i * kSelThreads;
      if (t < h1 && (s[i] != t || !in_place)) {
        page[i] = !FEW && s[i] != t ? bt[s[i] / KVQ_BLOCK_SIZE] : 0;
        w[i] = acc[s[i]];
        p[i] = pos[s[i]];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = tb + i * kSelThreads;
      if (t >= h1) break;
      if (s[i] != t || !in_place) {
        acc_out[t] = w[i];
        pos_out[t] = p[i];
      }
      if (FEW) {
        if (s[i] != t) {
          sh.few[atomicAdd(&sh.n_few, 1)] = make_int2(s[i], t);
        }
      } else {
        int32_t m = kStays;
        if (s[i] != t) {
          const bool ok = page[i] >= 0 && page[i] < a.num_blocks;  // page * 16 + 15 < 2^31: a pool is far smaller
          if (!ok) set_status(a.status, KVQ_DEV_BAD_BLOCK);
          m = ok ? page[i] * KVQ_BLOCK_SIZE + s[i] % KVQ_BLOCK_SIZE : kBadMove;
        }
        map[t] = m;
      }
    }
  }
  if (FEW) {  // the codes, a warp a token; no two moves touch the same slot
    __syncthreads();
    for (int i = warp; i < sh.n_few; i += kSelWarps) move_token(a, bt, kvh, sh.few[i].x, sh.few[i].y, lane);
  }
}

// The moves into one page below the budget: every load before the first store, and eight CTAs of 256 threads an
// SM (sixteen of 128).  64 x 8 of up to 16384: 244 us the call, 273 without the bound on registers, 260 with K's stores
// before V's words.
template <int D>
__global__ void __launch_bounds__(D, 2048 / D) evict_move_kernel(EvictArgs a) {
  const int p = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  __shared__ int32_t from[KVQ_BLOCK_SIZE];  // by destination slot: physical slot, or negative
  __shared__ int any;
  const long long unit = static_cast<long long>(b) * a.n_kv_heads + kvh;
  grid_dep_wait();
  const int moves = a.n_moves[unit];
  const int dpage = a.block_table[static_cast<long long>(b) * a.max_blocks_per_seq + p];
  if (tid < 32) {
    int32_t f = kStays;
    const int t = p * KVQ_BLOCK_SIZE + tid;
    if (tid < KVQ_BLOCK_SIZE && t < a.keep && moves) f = a.slot_map[unit * a.n_pages * KVQ_BLOCK_SIZE + t];
    const bool moving = f != kStays;
    const bool dst_ok = dpage >= 0 && dpage < a.num_blocks;
    if (moving && !dst_ok) set_status(a.status, KVQ_DEV_BAD_BLOCK);
    if (tid < KVQ_BLOCK_SIZE) from[tid] = f;
    const uint32_t m = __ballot_sync(0xffffffffu, f >= 0 && dst_ok);
    if (tid == 0) any = m != 0;
  }
  __syncthreads();
  if (!any) return;
  const long long dph = static_cast<long long>(dpage) * a.n_kv_heads + kvh;
  auto ph_of = [&](int f) { return static_cast<long long>(f / KVQ_BLOCK_SIZE) * a.n_kv_heads + kvh; };
  // V: thread = dim; its 16 slots are one 16-byte word, into which the movers' bytes go
  uint4* row = reinterpret_cast<uint4*>(a.v + (dph * D + tid) * KVQ_BLOCK_SIZE);
  const uint4 w = *row;
  uint32_t byte[KVQ_BLOCK_SIZE];
#pragma unroll
  for (int slot = 0; slot < KVQ_BLOCK_SIZE; ++slot) {
    const int f = from[slot];
    if (f >= 0) byte[slot] = static_cast<uint8_t>(a.v[(ph_of(f) * D + tid) * KVQ_BLOCK_SIZE + f % KVQ_BLOCK_SIZE]);
  }
  // K: a token's chunk of 16 dims is one 16-byte word; thread = (chunk tid / 16, slot tid % 16)
  const int slot = tid % KVQ_BLOCK_SIZE, ch = tid / KVQ_BLOCK_SIZE;
  const int f = from[slot];
  uint4 kc = make_uint4(0, 0, 0, 0);
  float sc = 0.f;
  if (f >= 0) {
    const long long ph = ph_of(f);
    kc = *reinterpret_cast<const uint4*>(a.k + ((ph * (D / 16) + ch) * KVQ_BLOCK_SIZE + f % KVQ_BLOCK_SIZE) * 16);
    if (ch < 2) sc = (ch ? a.v_scale : a.k_scale)[ph * KVQ_BLOCK_SIZE + f % KVQ_BLOCK_SIZE];
  }
  uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int s = 0; s < KVQ_BLOCK_SIZE; ++s) {
    if (from[s] >= 0) {
      const uint32_t sh = 8u * (s % 4);
      word[s / 4] = (word[s / 4] & ~(0xFFu << sh)) | (byte[s] << sh);
    }
  }
  *row = make_uint4(word[0], word[1], word[2], word[3]);
  if (f >= 0) {
    *reinterpret_cast<uint4*>(a.k + ((dph * (D / 16) + ch) * KVQ_BLOCK_SIZE + slot) * 16) = kc;
    if (ch < 2) (ch ? a.v_scale : a.k_scale)[dph * KVQ_BLOCK_SIZE + slot] = sc;
  }
}

// CTAs of a select cluster: as many (1, 2, 4 or 8) as keep at least 1024 slots each and all clusters
// in one wave of the SMs.  (64 x 8 of up to 16384, where that is 1: 285 us, and 352 with two, 469 with four.)
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
  w.off_map = (units * w.max_moves * 4 + 255) / 256 * 256;
  w.off_count = w.off_map + units * w.n_pages * KVQ_BLOCK_SIZE * 4;
  w.n_words = max_ctx > keep && max_ctx > kKeyCap ? (max_ctx + 31) / 32 : 0;
  w.off_words = w.off_count + units * 4;
  w.bytes = w.off_words + units * w.n_words * 8;
  return w;
}

cudaError_t launch_evict(const EvictArgs& a, int n_sms, cudaStream_t stream) {
  const int c = select_cluster(a, n_sms);
  const int range = ((a.max_ctx + c - 1) / c + 31) / 32 * 32;
  const size_t smem = static_cast<size_t>(std::min(range, kKeyCap)) * 4;
  const bool few = a.max_moves <= (static_cast<long long>(a.batch) * a.n_kv_heads < n_sms ? kFewMoves : kFewMovesLarge);
  auto kern = few ? evict_select_kernel<true> : evict_select_kernel<false>;
  cudaError_t e;
  static std::atomic<uint64_t> done[2];
  if ((e = allow_smem(reinterpret_cast<const void*>(kern), kKeyCap * 4, done[few])) != cudaSuccess) return e;
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
  if ((e = cudaLaunchKernelEx(&cfg, kern, a)) != cudaSuccess) return e;
  if (few) return cudaSuccess;
  // (a budget past the block table's pages never evicts)
  const dim3 grid(std::min(a.n_pages, a.max_blocks_per_seq), a.n_kv_heads, a.batch);
  return a.head_dim == 256 ? launch_pdl(evict_move_kernel<256>, grid, dim3(256), 0, stream, a)
                           : launch_pdl(evict_move_kernel<128>, grid, dim3(128), 0, stream, a);
}

}  // namespace kvq
