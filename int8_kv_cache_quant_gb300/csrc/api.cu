// api.cu — the C ABI of libkvq (include/kvq.h): host-side validation, routing and launch.
// Every entry point checks its arguments before launching anything, allocates nothing and
// never synchronises (except kvq_device_status).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "kvq.h"
#include "kvq_dev.cuh"
#include "kvq_launch.h"

namespace {

// Device status word (KVQ_DEV_* bits), one per device that loads the library.
__device__ unsigned int g_kvq_status = 0;

constexpr int kMaxDevices = 64;
unsigned int* g_status_ptr[kMaxDevices] = {};
std::mutex g_status_mu;

// Device address of the status word on the current device, looked up once per device.
unsigned int* status_ptr() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_status_mu);
  if (!g_status_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_kvq_status) != cudaSuccess) return nullptr;
    g_status_ptr[dev] = static_cast<unsigned int*>(p);
  }
  return g_status_ptr[dev];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_cache(const kvq_cache* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return KVQ_ERR_INVALID_ARG;
  if (c->num_blocks <= 0 || c->n_kv_heads <= 0) return KVQ_ERR_INVALID_ARG;
  if (c->block_size != KVQ_BLOCK_SIZE) return KVQ_ERR_UNSUPPORTED;
  if (c->head_dim != 128 && c->head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
    return KVQ_ERR_MISALIGNED;
  return KVQ_OK;
}

// The decode kernels count the keys of a block-table row in 32 bits.  (Counted in 64 the step of 64 sequences was 2 us
// slower, 244 against 242, for rows that no memory fills.)
bool decode_row_ok(int max_blocks_per_seq) { return max_blocks_per_seq < (1 << 27); }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

kvq_decode_opts decode_defaults(const kvq_decode_opts* o) {
  kvq_decode_opts r = {0, 0, 0, nullptr, nullptr, nullptr};  // split_rows 0: sized to the GPU; route 0: automatic
  if (o) {
    if (o->split_rows > 0) r.split_rows = o->split_rows;
    if (o->route_threshold > 0) r.route_threshold = o->route_threshold;
    r.force_route = o->force_route;
    r.stage1_event_begin = o->stage1_event_begin;
    r.stage1_event_end = o->stage1_event_end;
    r.launches = o->launches;
  }
  return r;
}

// Test-only fault injection (kvq_debug_fault_inject): the mode and the wait budget that the
// kernels launched from now on receive.
std::atomic<int> g_fault_mode{0};
std::atomic<long long> g_wait_budget{kvq::kWaitBudgetCycles};

}  // namespace

namespace kvq {
int debug_fault_mode() { return g_fault_mode.load(std::memory_order_relaxed); }
long long debug_wait_budget() { return g_wait_budget.load(std::memory_order_relaxed); }
}  // namespace kvq

extern "C" {

int kvq_version(void) { return KVQ_ABI_VERSION; }

const char* kvq_status_string(int s) {
  switch (s) {
    case KVQ_OK: return "ok";
    case KVQ_ERR_INVALID_ARG: return "invalid argument";
    case KVQ_ERR_UNSUPPORTED: return "unsupported shape or option";
    case KVQ_ERR_MISALIGNED: return "device pointer not 16-byte aligned";
    case KVQ_ERR_WORKSPACE: return "workspace missing or too small";
    case KVQ_ERR_CUDA: return "CUDA launch or runtime error";
    default: return "unknown status";
  }
}

int kvq_debug_fault_inject(int32_t mode, int64_t wait_budget_cycles) {
  if (mode < 0 || mode > 5) return KVQ_ERR_INVALID_ARG;
  g_wait_budget.store(wait_budget_cycles > 0 ? static_cast<long long>(wait_budget_cycles) : kvq::kWaitBudgetCycles);
  g_fault_mode.store(mode);
  return KVQ_OK;
}

int kvq_device_status(uint32_t* flags_out, void* stream) {
  if (!flags_out) return KVQ_ERR_INVALID_ARG;
  *flags_out = 0;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return KVQ_ERR_CUDA;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kvq_status, sizeof v) != cudaSuccess) return KVQ_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_kvq_status, &zero, sizeof zero) != cudaSuccess) return KVQ_ERR_CUDA;
  *flags_out = v;
  return KVQ_OK;
}

int kvq_quant_write(const kvq_cache* cache, const void* k_new, const void* v_new, int32_t n_tokens,
                    const int32_t* seq_idx, const int32_t* pos, const int32_t* block_table,
                    int32_t num_seqs, int32_t max_blocks_per_seq, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (n_tokens < 0 || num_seqs <= 0 || max_blocks_per_seq <= 0) return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return KVQ_OK;
  if (!k_new || !v_new || !seq_idx || !pos || !block_table) return KVQ_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new)) return KVQ_ERR_MISALIGNED;
  if (!aligned4(seq_idx) || !aligned4(pos) || !aligned4(block_table)) return KVQ_ERR_MISALIGNED;
  kvq::QuantWriteArgs a{};
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks;
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.k_new = k_new;
  a.v_new = v_new;
  a.n_tokens = n_tokens;
  a.seq_idx = seq_idx;
  a.pos = pos;
  a.block_table = block_table;
  a.num_seqs = num_seqs;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.status = status_ptr();
  return cuda_status(kvq::launch_quant_write(a, static_cast<cudaStream_t>(stream)));
}

int kvq_rope_quant_write(const kvq_cache* cache, const void* q, int32_t n_q_heads, const void* k_new,
                         const void* v_new, int32_t n_tokens, const int32_t* seq_idx, const int32_t* pos,
                         const int32_t* block_table, int32_t num_seqs, int32_t max_blocks_per_seq,
                         const float* cos_sin, int32_t max_pos, int32_t rotary_dim, int8_t* q_codes,
                         float* q_scales, void* q_rot, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (n_tokens < 0 || num_seqs <= 0 || max_blocks_per_seq <= 0 || max_pos <= 0) return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return KVQ_OK;
  if (!k_new || !v_new || !seq_idx || !pos || !block_table || !cos_sin) return KVQ_ERR_INVALID_ARG;
  if (q && n_q_heads <= 0) return KVQ_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  if (rotary_dim <= 0 || rotary_dim > D || rotary_dim % 2 != 0 || (rotary_dim / 2) % (D / 32) != 0)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(cos_sin)) return KVQ_ERR_MISALIGNED;
  if ((q && !aligned16(q)) || (q_rot && !aligned16(q_rot))) return KVQ_ERR_MISALIGNED;
  if (q_codes && reinterpret_cast<uintptr_t>(q_codes) % 8 != 0) return KVQ_ERR_MISALIGNED;
  if ((q_scales && !aligned4(q_scales)) || !aligned4(seq_idx) || !aligned4(pos) || !aligned4(block_table))
    return KVQ_ERR_MISALIGNED;
  kvq::RopeQuantArgs r{};
  r.kv.k = cache->k;
  r.kv.v = cache->v;
  r.kv.k_scale = cache->k_scale;
  r.kv.v_scale = cache->v_scale;
  r.kv.num_blocks = cache->num_blocks;
  r.kv.n_kv_heads = cache->n_kv_heads;
  r.kv.head_dim = D;
  r.kv.k_new = k_new;
  r.kv.v_new = v_new;
  r.kv.n_tokens = n_tokens;
  r.kv.seq_idx = seq_idx;
  r.kv.pos = pos;
  r.kv.block_table = block_table;
  r.kv.num_seqs = num_seqs;
  r.kv.max_blocks_per_seq = max_blocks_per_seq;
  r.kv.status = status_ptr();
  r.q = q;
  r.n_q_heads = q ? n_q_heads : 0;
  r.cos_sin = cos_sin;
  r.max_pos = max_pos;
  r.rotary_dim = rotary_dim;
  r.q_codes = q_codes;
  r.q_scales = q_scales;
  r.q_rot = static_cast<uint16_t*>(q_rot);
  return cuda_status(kvq::launch_rope_quant_write(r, static_cast<cudaStream_t>(stream)));
}

// Smallest split the automatic rule chooses: the workspace bound when split_rows is 0.
constexpr int kAutoSplitMinRows = 4 * KVQ_BLOCK_SIZE;

// Whether the split route may be taken, from host arguments alone (sizes the workspace).  The
// automatic route splits only when the split size leaves more than one split, and the automatic
// split size is never below kAutoSplitMinRows keys.
static bool decode_split_route(const kvq_decode_opts& o, int32_t max_ctx) {
  if (o.force_route == 1) return false;
  if (o.force_route == 2) return true;
  if (o.route_threshold > 0) return max_ctx > o.route_threshold;
  const int rows = o.split_rows > 0 ? o.split_rows : kAutoSplitMinRows;
  return max_ctx > rows;
}

int32_t kvq_decode_auto_split_rows(int32_t batch, int32_t n_kv_heads, int32_t head_dim, int32_t max_ctx,
                                   int32_t n_sms) {
  if (batch <= 0 || n_kv_heads <= 0 || max_ctx <= 0 || n_sms <= 0) return 0;
  if (head_dim != 128 && head_dim != 256) return 0;
  const long long slots = static_cast<long long>(n_sms) * (head_dim == 256 ? 1 : 2);  // resident stage-1 CTAs
  const long long units = static_cast<long long>(batch) * n_kv_heads;
  const long long pages = (static_cast<long long>(max_ctx) + KVQ_BLOCK_SIZE - 1) / KVQ_BLOCK_SIZE;
  long long split_pages;
  if (units * ((pages + 31) / 32) > 2 * slots) {
    split_pages = std::min(128LL, std::max(32LL, units * pages / (4 * slots)));
  } else {
    const long long per_unit = std::max(1LL, slots / units);
    split_pages = std::max(4LL, (pages + per_unit - 1) / per_unit);
  }
  return static_cast<int32_t>(split_pages * KVQ_BLOCK_SIZE);
}

static int device_sm_count() {
  static std::mutex mu;
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!cached[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev] = n;
  }
  return cached[dev];
}

size_t kvq_decode_workspace_bytes(int32_t batch, int32_t n_q_heads, int32_t max_ctx,
                                  int32_t head_dim, const kvq_decode_opts* opts) {
  const kvq_decode_opts o = decode_defaults(opts);
  if (batch <= 0 || n_q_heads <= 0 || max_ctx <= 0 || head_dim <= 0 || o.split_rows < 0) return 0;
  if (!decode_split_route(o, max_ctx)) return 0;
  const int rows = o.split_rows > 0 ? o.split_rows : kAutoSplitMinRows;
  return kvq::decode_workspace_bytes(batch, n_q_heads, max_ctx, head_dim, rows);
}

size_t kvq_verify_workspace_bytes(int32_t batch, int32_t n_rows, int32_t n_q_heads, int32_t max_ctx,
                                  int32_t head_dim, const kvq_decode_opts* opts) {
  if (batch <= 0 || n_rows <= 0 || static_cast<long long>(batch) * n_rows > INT32_MAX) return 0;
  return kvq_decode_workspace_bytes(batch * n_rows, n_q_heads, max_ctx, head_dim, opts);
}

}  // extern "C"

namespace kvq {
int decode_plan(const kvq_cache* cache, int32_t batch, int32_t nq, int32_t n_q_heads, int32_t max_ctx,
                const kvq_decode_opts* opts, DecodePlan* plan) {
  if (!cache || batch <= 0 || nq <= 0 || n_q_heads <= 0 || cache->n_kv_heads <= 0) return KVQ_ERR_INVALID_ARG;
  if (cache->head_dim != 128 && cache->head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  kvq_decode_opts o = decode_defaults(opts);
  if (o.split_rows % KVQ_BLOCK_SIZE != 0 || o.force_route < 0 || o.force_route > 2) return KVQ_ERR_INVALID_ARG;
  const int mc = max_ctx > 0 ? max_ctx : 1;
  bool split = decode_split_route(o, mc);
  if (split && o.split_rows == 0) {
    const int sms = device_sm_count();
    if (sms <= 0) return KVQ_ERR_CUDA;
    o.split_rows = kvq_decode_auto_split_rows(batch, cache->n_kv_heads, cache->head_dim, mc, sms);
  }
  // automatic route: one split would be the single-CTA route plus a merge
  if (split && o.force_route == 0 && o.route_threshold == 0 && mc <= o.split_rows) split = false;
  plan->split = split;
  plan->split_rows = o.split_rows;
  plan->n_split = 1;
  plan->bytes = 0;
  if (split) {
    const long long n_split = (static_cast<long long>(mc) + o.split_rows - 1) / o.split_rows;
    if (n_split > kvq::kMaxSplits) return KVQ_ERR_UNSUPPORTED;
    plan->n_split = static_cast<int>(n_split);
    plan->bytes = decode_workspace_bytes(batch * nq, n_q_heads, mc, cache->head_dim, o.split_rows);
  }
  return KVQ_OK;
}
}  // namespace kvq

extern "C" {

// What every decode call checks before it plans: pointers, sizes, GQA groups, alignment.
static int check_decode(const kvq_cache* cache, const void* k_new, const void* v_new, const void* q, int32_t batch,
                        int32_t nq, int32_t n_q_heads, const int32_t* block_table, int32_t max_blocks_per_seq,
                        const int32_t* ctx_lens, int32_t max_ctx, const float* out) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!q || !block_table || !ctx_lens || !out) return KVQ_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return KVQ_ERR_INVALID_ARG;
  if (k_new && (!aligned16(k_new) || !aligned16(v_new))) return KVQ_ERR_MISALIGNED;
  if (batch <= 0 || nq <= 0 || n_q_heads <= 0 || max_blocks_per_seq <= 0 || max_ctx < 0) return KVQ_ERR_INVALID_ARG;
  // stage 1 puts the sequences on grid z, the merge puts (sequence, row) on grid y
  if (static_cast<long long>(batch) * nq > 65535) return KVQ_ERR_UNSUPPORTED;
  if (n_q_heads % cache->n_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  const int G = n_q_heads / cache->n_kv_heads;
  if (G > 16 || static_cast<long long>(G) * nq > KVQ_VERIFY_MAX_ROWS) return KVQ_ERR_UNSUPPORTED;
  if (!decode_row_ok(max_blocks_per_seq)) return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(out)) return KVQ_ERR_MISALIGNED;
  if (!aligned4(block_table) || !aligned4(ctx_lens)) return KVQ_ERR_MISALIGNED;
  return KVQ_OK;
}

// The kernels' arguments, but for the workspace.
static kvq::DecodeArgs decode_args(const kvq_cache* cache, const void* k_new, const void* v_new, const void* q,
                                   int32_t batch, int32_t nq, int32_t n_q_heads, const int32_t* block_table,
                                   int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t mc,
                                   float softmax_scale, float* out, const kvq_decode_opts& o,
                                   const kvq::DecodePlan& plan) {
  kvq::DecodeArgs a{};
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks;
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.q = q;
  a.batch = batch;
  a.nq = nq;
  a.n_q_heads = n_q_heads;
  a.block_table = block_table;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.ctx_lens = ctx_lens;
  a.max_ctx = mc;
  a.softmax_scale = softmax_scale;
  a.k_new = k_new;
  a.v_new = v_new;
  a.out = out;
  a.split_rows = plan.split_rows;
  a.n_split = plan.n_split;
  a.status = status_ptr();
  a.ev_begin = static_cast<cudaEvent_t>(o.stage1_event_begin);
  a.ev_end = static_cast<cudaEvent_t>(o.stage1_event_end);
  a.wait_budget = kvq::debug_wait_budget();
  a.fault = kvq::debug_fault_mode();
  return a;
}

// The split route's partials in the workspace: accumulators, then statistics on a 256-byte boundary.
static void place_partials(kvq::DecodeArgs* a, void* workspace) {
  const long long units = static_cast<long long>(a->batch) * a->nq * a->n_q_heads * a->n_split;
  const long long acc_bytes = ((units * a->head_dim * 4 + 255) / 256) * 256;
  a->part_acc = static_cast<float*>(workspace);
  a->part_stats = reinterpret_cast<float*>(static_cast<char*>(workspace) + acc_bytes);
}

// Decode with nq query rows per sequence (nq = 1: plain decode); with k_new / v_new, the fused
// step that first writes each sequence's nq newest tokens into the cache.
static int decode_rows(const kvq_cache* cache, const void* k_new, const void* v_new, const void* q, int32_t batch,
                       int32_t nq, int32_t n_q_heads, const int32_t* block_table, int32_t max_blocks_per_seq,
                       const int32_t* ctx_lens, int32_t max_ctx, float softmax_scale, float* out, void* workspace,
                       size_t workspace_bytes, const kvq_decode_opts* opts, void* stream) {
  int st = check_decode(cache, k_new, v_new, q, batch, nq, n_q_heads, block_table, max_blocks_per_seq, ctx_lens,
                        max_ctx, out);
  if (st != KVQ_OK) return st;
  const int mc = max_ctx > 0 ? max_ctx : 1;
  const kvq_decode_opts o = decode_defaults(opts);
  if (o.split_rows % KVQ_BLOCK_SIZE != 0 || o.force_route < 0 || o.force_route > 2) return KVQ_ERR_INVALID_ARG;
  // the workspace rule is pure host arithmetic (kvq_decode_workspace_bytes), checked before the GPU is asked
  if (decode_split_route(o, mc) && !workspace) return KVQ_ERR_WORKSPACE;
  kvq::DecodePlan plan;
  st = kvq::decode_plan(cache, batch, nq, n_q_heads, mc, opts, &plan);
  if (st != KVQ_OK) return st;
  if (plan.split) {
    if (!workspace || workspace_bytes < plan.bytes) return KVQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  }
  kvq::DecodeArgs a = decode_args(cache, k_new, v_new, q, batch, nq, n_q_heads, block_table, max_blocks_per_seq,
                                  ctx_lens, mc, softmax_scale, out, o, plan);
  if (plan.split) place_partials(&a, workspace);
  int launched = 0;
  const int rc = cuda_status(kvq::launch_decode(a, plan.split ? kvq::DecodeRoute::kSplit : kvq::DecodeRoute::kSingle,
                                                static_cast<cudaStream_t>(stream), &launched));
  if (o.launches) *o.launches = launched;
  return rc;
}

int kvq_attn_decode_int8kv(const kvq_cache* cache, const void* q, int32_t batch, int32_t n_q_heads,
                           const int32_t* block_table, int32_t max_blocks_per_seq,
                           const int32_t* ctx_lens, int32_t max_ctx, float softmax_scale, float* out,
                           void* workspace, size_t workspace_bytes, const kvq_decode_opts* opts,
                           void* stream) {
  return decode_rows(cache, nullptr, nullptr, q, batch, 1, n_q_heads, block_table, max_blocks_per_seq, ctx_lens,
                     max_ctx, softmax_scale, out, workspace, workspace_bytes, opts, stream);
}

int kvq_attn_verify_int8kv(const kvq_cache* cache, const void* q, int32_t batch, int32_t n_rows,
                           int32_t n_q_heads, const int32_t* block_table, int32_t max_blocks_per_seq,
                           const int32_t* ctx_lens, int32_t max_ctx, float softmax_scale, float* out,
                           void* workspace, size_t workspace_bytes, const kvq_decode_opts* opts,
                           void* stream) {
  return decode_rows(cache, nullptr, nullptr, q, batch, n_rows, n_q_heads, block_table, max_blocks_per_seq,
                     ctx_lens, max_ctx, softmax_scale, out, workspace, workspace_bytes, opts, stream);
}

int kvq_decode_step_int8kv(const kvq_cache* cache, const void* k_new, const void* v_new, const void* q,
                           int32_t batch, int32_t n_new, int32_t n_q_heads, const int32_t* block_table,
                           int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t max_ctx,
                           float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                           const kvq_decode_opts* opts, void* stream) {
  if (!k_new || !v_new) return KVQ_ERR_INVALID_ARG;
  return decode_rows(cache, k_new, v_new, q, batch, n_new, n_q_heads, block_table, max_blocks_per_seq, ctx_lens,
                     max_ctx, softmax_scale, out, workspace, workspace_bytes, opts, stream);
}

// The split route always: the weights are made from the scores of a finished stage 1.
static kvq_decode_opts accum_opts(const kvq_decode_opts* opts) {
  kvq_decode_opts o = decode_defaults(opts);
  o.force_route = 2;
  return o;
}

static long long accum_scores_bytes(int32_t batch, int32_t nq, int32_t n_q_heads, int32_t max_ctx) {
  const long long stride = (static_cast<long long>(max_ctx) + KVQ_BLOCK_SIZE - 1) / KVQ_BLOCK_SIZE * KVQ_BLOCK_SIZE;
  return static_cast<long long>(batch) * nq * n_q_heads * stride * 4;
}

size_t kvq_step_accum_workspace_bytes(int32_t batch, int32_t n_new, int32_t n_q_heads, int32_t max_ctx,
                                      int32_t head_dim, const kvq_decode_opts* opts) {
  const kvq_decode_opts o = accum_opts(opts);
  const size_t part = kvq_verify_workspace_bytes(batch, n_new, n_q_heads, max_ctx, head_dim, &o);
  if (part == 0) return 0;
  return (part + 255) / 256 * 256 + static_cast<size_t>(accum_scores_bytes(batch, n_new, n_q_heads, max_ctx));
}

int kvq_decode_step_accum_int8kv(const kvq_cache* cache, const void* k_new, const void* v_new, const void* q,
                                 int32_t batch, int32_t n_new, int32_t n_q_heads, const int32_t* block_table,
                                 int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t max_ctx,
                                 float softmax_scale, float* out, float* acc, int64_t acc_stride, int32_t* slot_pos,
                                 const int32_t* pos, void* workspace, size_t workspace_bytes,
                                 const kvq_decode_opts* opts, void* stream) {
  int st = check_decode(cache, k_new, v_new, q, batch, n_new, n_q_heads, block_table, max_blocks_per_seq, ctx_lens,
                        max_ctx, out);
  if (st != KVQ_OK) return st;
  if (!acc || max_ctx <= 0 || acc_stride < max_ctx) return KVQ_ERR_INVALID_ARG;
  if (max_ctx > 1 << 30) return KVQ_ERR_UNSUPPORTED;  // slots are counted in 32 bits, a block of them ahead
  if ((slot_pos == nullptr) != (pos == nullptr) || (slot_pos && !k_new)) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(acc) || !aligned4(slot_pos) || !aligned4(pos)) return KVQ_ERR_MISALIGNED;
  if (opts && opts->force_route == 1) return KVQ_ERR_UNSUPPORTED;
  const kvq_decode_opts o = accum_opts(opts);
  if (o.split_rows % KVQ_BLOCK_SIZE != 0 || (opts && (opts->force_route < 0 || opts->force_route > 2)))
    return KVQ_ERR_INVALID_ARG;
  if (!workspace) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  kvq::DecodePlan plan;
  st = kvq::decode_plan(cache, batch, n_new, n_q_heads, max_ctx, &o, &plan);
  if (st != KVQ_OK) return st;
  const size_t part = (plan.bytes + 255) / 256 * 256;
  if (workspace_bytes < part + static_cast<size_t>(accum_scores_bytes(batch, n_new, n_q_heads, max_ctx)))
    return KVQ_ERR_WORKSPACE;
  kvq::StepAccumArgs a{};
  a.d = decode_args(cache, k_new, v_new, q, batch, n_new, n_q_heads, block_table, max_blocks_per_seq, ctx_lens,
                    max_ctx, softmax_scale, out, o, plan);
  place_partials(&a.d, workspace);
  a.d.scores = reinterpret_cast<float*>(static_cast<char*>(workspace) + part);
  a.d.scores_stride = (static_cast<long long>(max_ctx) + KVQ_BLOCK_SIZE - 1) / KVQ_BLOCK_SIZE * KVQ_BLOCK_SIZE;
  a.acc = acc;
  a.acc_stride = acc_stride;
  a.slot_pos = slot_pos;
  a.pos = pos;
  if (!kvq::step_accum_grid_ok(a.d)) return KVQ_ERR_UNSUPPORTED;
  int launched = 0;
  const int rc = cuda_status(kvq::launch_step_accum(a, static_cast<cudaStream_t>(stream), &launched));
  if (o.launches) *o.launches = launched;
  return rc;
}

// The most keys that a windowed step counts of a sequence (window_map): whole pages of the first keys, and of the rows'
// windows, which may begin at the end of a page.
static int32_t window_keys(int32_t max_ctx, int32_t n_new, int32_t window, int32_t n_sink) {
  const long long pages = (static_cast<long long>(n_sink) + KVQ_BLOCK_SIZE - 1) / KVQ_BLOCK_SIZE +
                          (static_cast<long long>(window) + n_new - 1 + 2 * (KVQ_BLOCK_SIZE - 1)) / KVQ_BLOCK_SIZE;
  return static_cast<int32_t>(std::min<long long>(std::max(max_ctx, 1), pages * KVQ_BLOCK_SIZE));
}

// The automatic split size of a step with a window.  All sequences longer than the window have the same number of keys, so that
// what counts is how often a round of resident CTAs goes through them: n splits of a unit take about
// one round of (pages / n + 22) pages where slots CTAs are enough, or units n / slots + 1/2 of them; 22 is for a CTA's start and
// end, and the pages are cut evenly.  Against the rule of the whole contexts, 8 KV heads of 128: batch 64, window 4096, two
// splits 103.8 us, three uneven ones 113.1 us; window 1024, one 35.7 us, three 44.7 us; batch 16, window 4096, two 32.8 us,
// nine 39.8 us.  Batch 128, 4 KV heads of 256, window 4096: one 180.8 us, three 200.9 us.
static int32_t window_split_rows(int32_t batch, int32_t n_kv_heads, int32_t head_dim, int32_t keys, int32_t n_sms) {
  const double slots = static_cast<double>(n_sms) * (head_dim == 256 ? 1 : 2);  // resident stage-1 CTAs
  const double units = static_cast<double>(batch) * n_kv_heads;
  const int pages = keys / KVQ_BLOCK_SIZE + (keys % KVQ_BLOCK_SIZE != 0);
  const int most = std::min(std::max(1, pages / (kAutoSplitMinRows / KVQ_BLOCK_SIZE)),
                            std::max(8, static_cast<int>(std::min(slots / units, 1024.0))));
  int best = 1;
  double least = 0.0;
  for (int n = 1; n <= most; ++n) {
    const double rounds = units * n <= slots ? 1.0 : units * n / slots + 0.5, t = rounds * (pages / static_cast<double>(n) + 22.0);
    if (n == 1 || t < least) {
      best = n;
      least = t;
    }
  }
  return std::max(kAutoSplitMinRows, (pages + best - 1) / best * KVQ_BLOCK_SIZE);
}

size_t kvq_step_window_workspace_bytes(int32_t batch, int32_t n_new, int32_t n_q_heads, int32_t n_kv_heads,
                                       int32_t max_ctx, int32_t window, int32_t n_sink, int32_t head_dim,
                                       const kvq_decode_opts* opts) {
  if (n_kv_heads <= 0 || max_ctx <= 0 || window <= 0 || n_sink < 0) return 0;
  return kvq_verify_workspace_bytes(batch, n_new, n_q_heads, window_keys(max_ctx, n_new, window, n_sink), head_dim, opts);
}

int kvq_decode_step_window_int8kv(const kvq_cache* cache, const void* k_new, const void* v_new, const void* q,
                                  int32_t batch, int32_t n_new, int32_t n_q_heads, const int32_t* block_table,
                                  int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t max_ctx,
                                  float softmax_scale, int32_t window, int32_t n_sink, float* out, void* workspace,
                                  size_t workspace_bytes, const kvq_decode_opts* opts, void* stream) {
  int st = check_decode(cache, k_new, v_new, q, batch, n_new, n_q_heads, block_table, max_blocks_per_seq, ctx_lens,
                        max_ctx, out);
  if (st != KVQ_OK) return st;
  if (window <= 0 || n_sink < 0) return KVQ_ERR_INVALID_ARG;
  const int mc = max_ctx > 0 ? max_ctx : 1;
  const int32_t keys = window_keys(mc, n_new, window, n_sink);
  kvq_decode_opts o = decode_defaults(opts);
  if (o.split_rows % KVQ_BLOCK_SIZE != 0 || o.force_route < 0 || o.force_route > 2) return KVQ_ERR_INVALID_ARG;
  if (decode_split_route(o, keys)) {
    if (!workspace) return KVQ_ERR_WORKSPACE;
    if (o.split_rows == 0) {
      const int sms = device_sm_count();
      if (sms <= 0) return KVQ_ERR_CUDA;
      o.split_rows = window_split_rows(batch, cache->n_kv_heads, cache->head_dim, keys, sms);
    }
  }
  kvq::DecodePlan plan;
  st = kvq::decode_plan(cache, batch, n_new, n_q_heads, keys, &o, &plan);
  if (st != KVQ_OK) return st;
  if (plan.split) {
    if (!workspace || workspace_bytes < plan.bytes) return KVQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  }
  kvq::DecodeArgs a = decode_args(cache, k_new, v_new, q, batch, n_new, n_q_heads, block_table, max_blocks_per_seq,
                                  ctx_lens, mc, softmax_scale, out, o, plan);
  if (plan.split) place_partials(&a, workspace);
  a.window = std::min(window, mc);
  a.n_sink = std::min(n_sink, mc);
  int launched = 0;
  const int rc = cuda_status(kvq::launch_step_window(a, plan.split ? kvq::DecodeRoute::kSplit : kvq::DecodeRoute::kSingle,
                                                     static_cast<cudaStream_t>(stream), &launched));
  if (o.launches) *o.launches = launched;
  return rc;
}

// Largest number of CTAs a pass of the chunk weights runs: more than any GPU the library is built for has
// SMs, so that the workspace size does not depend on the GPU.
constexpr int kChunkWeightsMaxRuns = 160;

static bool chunk_weights_sizes_ok(int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads, int32_t history_len) {
  if (n_tokens <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || history_len < 0 || n_q_heads % n_kv_heads != 0) return false;
  // rows of a KV head and keys are counted in 32 bits, with room for a tile more
  const long long limit = 1LL << 30;
  const long long rows = static_cast<long long>(n_tokens) * (n_q_heads / n_kv_heads), keys = static_cast<long long>(history_len) + n_tokens;
  if (rows >= limit || keys >= limit) return false;
  // and so are a CTA's score tiles
  return (rows + 127) / 128 * ((keys + 127) / 128) < (1LL << 35) / n_kv_heads;
}

size_t kvq_chunk_weights_workspace_bytes(int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads, int32_t history_len,
                                         int32_t head_dim) {
  if (!chunk_weights_sizes_ok(n_tokens, n_q_heads, n_kv_heads, history_len) || (head_dim != 128 && head_dim != 256)) return 0;
  return static_cast<size_t>(
      kvq::chunk_weights_plan(n_tokens, n_q_heads, n_kv_heads, history_len, head_dim, kChunkWeightsMaxRuns).bytes);
}

int kvq_attn_chunk_weights_int8kv(const kvq_cache* cache, const void* q, int32_t n_tokens, int32_t n_q_heads,
                                  int32_t history_len, const int32_t* block_table_row, int32_t n_blocks_row,
                                  float softmax_scale, float* acc, int64_t acc_stride, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!q || !block_table_row || !acc) return KVQ_ERR_INVALID_ARG;
  if (n_tokens <= 0 || n_q_heads <= 0 || history_len < 0 || n_blocks_row <= 0) return KVQ_ERR_INVALID_ARG;
  if (n_q_heads % cache->n_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  const long long n_keys = static_cast<long long>(history_len) + n_tokens;
  if (n_keys > static_cast<long long>(n_blocks_row) * KVQ_BLOCK_SIZE || acc_stride < n_keys) return KVQ_ERR_INVALID_ARG;
  if (!chunk_weights_sizes_ok(n_tokens, n_q_heads, cache->n_kv_heads, history_len) || cache->n_kv_heads > 65535)
    return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned4(acc) || !aligned4(block_table_row)) return KVQ_ERR_MISALIGNED;
  if (!workspace) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  const int sms = std::min(device_sm_count(), kChunkWeightsMaxRuns);
  if (sms <= 0) return KVQ_ERR_CUDA;
  const kvq::ChunkWeightsPlan p = kvq::chunk_weights_plan(n_tokens, n_q_heads, cache->n_kv_heads, history_len, cache->head_dim, sms);
  if (workspace_bytes < static_cast<size_t>(p.bytes)) return KVQ_ERR_WORKSPACE;
  kvq::ChunkWeightsArgs a{};
  a.k = cache->k;
  a.k_scale = cache->k_scale;
  a.num_blocks = cache->num_blocks;
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.q = q;
  a.n_q_heads = n_q_heads;
  a.group = n_q_heads / cache->n_kv_heads;
  a.history_len = history_len;
  a.n_rows = n_tokens * a.group;
  a.n_keys = static_cast<int>(n_keys);
  a.block_table_row = block_table_row;
  a.c2 = softmax_scale * 1.44269504088896341f;
  a.acc = acc;
  a.acc_stride = acc_stride;
  a.row_tiles = p.row_tiles;
  a.key_tiles = p.key_tiles;
  for (int i = 0; i < 2; ++i) {
    a.a_rows[i] = p.a_rows[i];
    a.units[i] = p.units[i];
    a.line[i] = p.line[i];
    a.runs[i] = p.runs[i];
    a.n_part[i] = p.n_part[i];
  }
  char* base = static_cast<char*>(workspace);
  a.row_part = reinterpret_cast<float2*>(base);
  a.row_nm = reinterpret_cast<float*>(base + p.off_nm);
  a.row_il = reinterpret_cast<float*>(base + p.off_il);
  a.q_tiles = reinterpret_cast<uint8_t*>(base + p.off_q);
  a.col_part = reinterpret_cast<float*>(base + p.off_col);
  if (p.widen_once) {
    a.k_tiles = reinterpret_cast<uint8_t*>(base + p.off_k);
    a.k_par = reinterpret_cast<float*>(base + p.off_kpar);
    a.k_valid = reinterpret_cast<uint32_t*>(base + p.off_kvalid);
  }
  a.status = status_ptr();
  a.wait_budget = kvq::debug_wait_budget();
  a.fault = kvq::debug_fault_mode();
  return cuda_status(kvq::launch_chunk_weights(a, static_cast<cudaStream_t>(stream)));
}

size_t kvq_evict_workspace_bytes(int32_t batch, int32_t n_kv_heads, int32_t max_ctx, int32_t keep) {
  if (batch <= 0 || n_kv_heads <= 0 || max_ctx <= 0 || keep <= 0) return 0;
  return static_cast<size_t>(kvq::evict_workspace(batch, n_kv_heads, max_ctx, keep).bytes);
}

int kvq_cache_evict(const kvq_cache* cache, int32_t batch, const int32_t* block_table, int32_t max_blocks_per_seq,
                    const int32_t* ctx_lens, int32_t max_ctx, int32_t keep, int32_t n_sink, int32_t n_recent,
                    const float* acc, const int32_t* slot_pos, int64_t acc_stride, float* acc_out,
                    int32_t* slot_pos_out, int64_t out_stride, int32_t* new_lens, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!block_table || !ctx_lens || !acc || !slot_pos || !acc_out || !slot_pos_out || !new_lens)
    return KVQ_ERR_INVALID_ARG;
  if (batch <= 0 || max_blocks_per_seq <= 0 || max_ctx <= 0 || keep <= 0) return KVQ_ERR_INVALID_ARG;
  if (n_sink < 0 || n_recent < 0 || static_cast<long long>(n_sink) + n_recent > keep) return KVQ_ERR_INVALID_ARG;
  if (acc_stride < max_ctx || out_stride < std::min(keep, max_ctx)) return KVQ_ERR_INVALID_ARG;
  // in place: both arrays, with the same rows
  if ((acc_out == acc) != (slot_pos_out == slot_pos) || (acc_out == acc && out_stride != acc_stride))
    return KVQ_ERR_INVALID_ARG;
  if (new_lens == ctx_lens) return KVQ_ERR_INVALID_ARG;
  if (batch > 65535 || cache->n_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;  // grid y and z
  if (max_ctx > 1 << 30) return KVQ_ERR_UNSUPPORTED;  // slots are counted in 32 bits, a block of them ahead
  if (!aligned4(block_table) || !aligned4(ctx_lens) || !aligned4(acc) || !aligned4(slot_pos) || !aligned4(acc_out) ||
      !aligned4(slot_pos_out) || !aligned4(new_lens))
    return KVQ_ERR_MISALIGNED;
  const kvq::EvictWorkspace w = kvq::evict_workspace(batch, cache->n_kv_heads, max_ctx, keep);
  if (!workspace || workspace_bytes < static_cast<size_t>(w.bytes)) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  const int sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  kvq::EvictArgs a{};
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks;
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.batch = batch;
  a.block_table = block_table;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.ctx_lens = ctx_lens;
  a.max_ctx = max_ctx;
  a.keep = keep;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.acc = acc;
  a.slot_pos = slot_pos;
  a.acc_stride = acc_stride;
  a.acc_out = acc_out;
  a.slot_pos_out = slot_pos_out;
  a.out_stride = out_stride;
  a.new_lens = new_lens;
  char* base = static_cast<char*>(workspace);
  a.max_moves = w.max_moves;
  a.n_pages = w.n_pages;
  a.move_src = reinterpret_cast<int32_t*>(base);
  a.slot_map = reinterpret_cast<int32_t*>(base + w.off_map);
  a.n_moves = reinterpret_cast<int32_t*>(base + w.off_count);
  a.n_words = w.n_words;
  a.words = reinterpret_cast<uint32_t*>(base + w.off_words);
  a.status = status_ptr();
  return cuda_status(kvq::launch_evict(a, sms, static_cast<cudaStream_t>(stream)));
}

int kvq_rope_phases(int32_t rotary_dim, double base, const kvq_rope_scaling* scaling, uint64_t* phases,
                    float* attn_factor) {
  if (!phases || rotary_dim <= 0 || rotary_dim % 2 != 0) return KVQ_ERR_INVALID_ARG;
  if (!(base > 0.0) || !std::isfinite(base)) return KVQ_ERR_INVALID_ARG;
  kvq_rope_scaling z = {KVQ_ROPE_NONE, 1.0, 0.0, 0.0, 0.0, nullptr};
  if (scaling) z = *scaling;
  if (z.kind < KVQ_ROPE_NONE || z.kind > KVQ_ROPE_DIVISORS) return KVQ_ERR_UNSUPPORTED;
  if (z.kind != KVQ_ROPE_NONE && z.kind != KVQ_ROPE_DIVISORS && (!(z.factor > 0.0) || !std::isfinite(z.factor)))
    return KVQ_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586476925;
  const double r = rotary_dim;
  double low = 0.0, high = 0.0, factor_attn = 1.0;
  if (z.kind == KVQ_ROPE_NTK) {
    if (rotary_dim <= 2) return KVQ_ERR_INVALID_ARG;
    base *= std::pow(z.factor, r / (r - 2.0));
  } else if (z.kind == KVQ_ROPE_YARN) {
    if (!(z.original_len > 0.0) || !(z.low > 0.0) || !(z.high > z.low) || !(base > 1.0)) return KVQ_ERR_INVALID_ARG;
    auto dim_of = [&](double turns) { return r * std::log(z.original_len / (turns * kTwoPi)) / (2.0 * std::log(base)); };
    low = std::max(std::floor(dim_of(z.high)), 0.0);
    high = std::min(std::ceil(dim_of(z.low)), r - 1.0);
    if (z.factor > 1.0) factor_attn = 0.1 * std::log(z.factor) + 1.0;
  } else if (z.kind == KVQ_ROPE_BANDS) {
    if (!(z.original_len > 0.0) || !(z.low > 0.0) || !(z.high > z.low)) return KVQ_ERR_INVALID_ARG;
  } else if (z.kind == KVQ_ROPE_DIVISORS) {
    if (!z.divisors) return KVQ_ERR_INVALID_ARG;
  }
  auto frequency = [&](int32_t j) {
    double inv = std::pow(base, -2.0 * j / r);
    if (z.kind == KVQ_ROPE_LINEAR) {
      inv /= z.factor;
    } else if (z.kind == KVQ_ROPE_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (j - low) / std::max(high - low, 1e-3)));
      inv = inv / z.factor * ramp + inv * (1.0 - ramp);
    } else if (z.kind == KVQ_ROPE_BANDS) {
      const double turns = z.original_len * inv / kTwoPi;  // over the original context
      const double mix = std::min(1.0, std::max(0.0, (turns - z.low) / (z.high - z.low)));
      inv = inv / z.factor * (1.0 - mix) + inv * mix;
    } else if (z.kind == KVQ_ROPE_DIVISORS) {
      inv /= z.divisors[j];
    }
    return inv;
  };
  // every frequency before the first phase is written: one past what a double holds has no fraction of a turn
  for (int32_t j = 0; j < rotary_dim / 2; ++j)
    if ((z.kind == KVQ_ROPE_DIVISORS && !(z.divisors[j] > 0.0)) || !std::isfinite(frequency(j))) return KVQ_ERR_INVALID_ARG;
  for (int32_t j = 0; j < rotary_dim / 2; ++j) {
    double turns = frequency(j) / kTwoPi;
    turns -= std::floor(turns);
    const double scaled = std::nearbyint(std::ldexp(turns, 64));
    phases[j] = scaled >= 18446744073709551616.0 ? 0u : static_cast<uint64_t>(scaled);
  }
  if (attn_factor) *attn_factor = static_cast<float>(factor_attn);
  return KVQ_OK;
}

}  // extern "C"

// What the calls that rotate rows check of them, and their arguments but for the positions.
static int rope_rows(const void* q, void* q_out, int64_t q_stride, int64_t q_out_stride, int32_t n_q_heads,
                     const void* k, void* k_out, int64_t k_stride, int64_t k_out_stride, int32_t n_kv_heads,
                     int32_t head_dim, int32_t n_tokens, const int32_t* pos, const uint64_t* phases, int32_t rotary_dim,
                     int32_t rotary_offset, int32_t layout, float attn_factor, kvq::RopeArgs* args, bool* nothing) {
  *nothing = false;
  if (n_tokens < 0 || n_q_heads < 0 || n_kv_heads < 0 || head_dim <= 0) return KVQ_ERR_INVALID_ARG;
  if (layout != KVQ_ROPE_HALF && layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_UNSUPPORTED;
  if (rotary_dim <= 0 || rotary_dim % 2 != 0 || rotary_offset < 0 ||
      static_cast<long long>(rotary_offset) + rotary_dim > head_dim)
    return KVQ_ERR_INVALID_ARG;
  if (head_dim > 1024 || static_cast<long long>(n_q_heads) + n_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  if (n_tokens == 0 || n_q_heads + n_kv_heads == 0) {
    *nothing = true;
    return KVQ_OK;
  }
  if (!pos || !phases) return KVQ_ERR_INVALID_ARG;
  if (n_q_heads && (!q || !q_out)) return KVQ_ERR_INVALID_ARG;
  if (n_kv_heads && (!k || !k_out)) return KVQ_ERR_INVALID_ARG;
  // rows of different tokens do not overlap (one token has no next row)
  const long long qd = static_cast<long long>(n_q_heads) * head_dim, kd = static_cast<long long>(n_kv_heads) * head_dim;
  if (n_tokens > 1 && ((n_q_heads && (q_stride < qd || q_out_stride < qd)) ||
                       (n_kv_heads && (k_stride < kd || k_out_stride < kd))))
    return KVQ_ERR_INVALID_ARG;
  // in place means the same rows
  if (n_tokens > 1 && ((n_q_heads && q == q_out && q_stride != q_out_stride) ||
                       (n_kv_heads && k == k_out && k_stride != k_out_stride)))
    return KVQ_ERR_INVALID_ARG;
  auto odd = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) != 0; };
  if (odd(q) || odd(q_out) || odd(k) || odd(k_out) || !aligned4(pos) || reinterpret_cast<uintptr_t>(phases) % 8 != 0)
    return KVQ_ERR_MISALIGNED;
  kvq::RopeArgs& a = *args;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.q_stride = n_tokens > 1 ? q_stride : qd;
  a.q_out_stride = n_tokens > 1 ? q_out_stride : qd;
  a.k_stride = n_tokens > 1 ? k_stride : kd;
  a.k_out_stride = n_tokens > 1 ? k_out_stride : kd;
  a.n_q_heads = n_q_heads;
  a.n_kv_heads = n_kv_heads;
  a.head_dim = head_dim;
  a.n_tokens = n_tokens;
  a.pos = pos;
  a.phases = reinterpret_cast<const unsigned long long*>(phases);
  a.rotary_dim = rotary_dim;
  a.rotary_offset = rotary_offset;
  a.interleaved = layout == KVQ_ROPE_INTERLEAVED;
  a.attn_factor = attn_factor;
  return KVQ_OK;
}

// Positions on several axes; axis_of (host) names the axis of each of the n frequencies.
static int rope_axes(const int32_t* pos, int64_t pos_stride, int32_t n_axes, const uint8_t* axis_of, int32_t n,
                     int32_t n_tokens, kvq::RopeAxes* ax) {
  if (n_axes < 1 || n_axes > kvq::kMaxAxes) return KVQ_ERR_UNSUPPORTED;
  if (!axis_of || (n_axes > 1 && pos_stride < n_tokens)) return KVQ_ERR_INVALID_ARG;
  ax->pos = pos;
  ax->pos_stride = n_axes > 1 ? pos_stride : 0;
  ax->n = n_axes;
  for (int32_t j = 0; j < n; ++j) {
    if (axis_of[j] >= n_axes) return KVQ_ERR_INVALID_ARG;
    ax->map[j / 16] |= static_cast<uint32_t>(axis_of[j]) << (2 * (j % 16));
  }
  return KVQ_OK;
}

extern "C" {

int kvq_rope_bf16(const void* q, void* q_out, int64_t q_stride, int64_t q_out_stride, int32_t n_q_heads,
                  const void* k, void* k_out, int64_t k_stride, int64_t k_out_stride, int32_t n_kv_heads,
                  int32_t head_dim, int32_t n_tokens, const int32_t* pos, const uint64_t* phases, int32_t rotary_dim,
                  int32_t rotary_offset, int32_t layout, float attn_factor, void* stream) {
  kvq::RopeArgs a{};
  bool nothing;
  const int st = rope_rows(q, q_out, q_stride, q_out_stride, n_q_heads, k, k_out, k_stride, k_out_stride, n_kv_heads,
                           head_dim, n_tokens, pos, phases, rotary_dim, rotary_offset, layout, attn_factor, &a, &nothing);
  if (st != KVQ_OK || nothing) return st;
  const int sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  return cuda_status(kvq::launch_rope(a, sms, static_cast<cudaStream_t>(stream)));
}

int kvq_rope_axes_bf16(const void* q, void* q_out, int64_t q_stride, int64_t q_out_stride, int32_t n_q_heads,
                       const void* k, void* k_out, int64_t k_stride, int64_t k_out_stride, int32_t n_kv_heads,
                       int32_t head_dim, int32_t n_tokens, const int32_t* pos, int64_t pos_stride, int32_t n_axes,
                       const uint64_t* phases, const uint8_t* axis_of, int32_t rotary_dim, int32_t rotary_offset,
                       int32_t layout, float attn_factor, int32_t inverse, void* stream) {
  kvq::RopeAxesArgs a{};
  bool nothing;
  int st = rope_rows(q, q_out, q_stride, q_out_stride, n_q_heads, k, k_out, k_stride, k_out_stride, n_kv_heads, head_dim,
                     n_tokens, pos, phases, rotary_dim, rotary_offset, layout, attn_factor, &a, &nothing);
  if (st != KVQ_OK || nothing) return st;
  st = rope_axes(pos, pos_stride, n_axes, axis_of, rotary_dim / 2, n_tokens, &a.axes);
  if (st != KVQ_OK) return st;
  a.sin_factor = inverse ? -attn_factor : attn_factor;
  const int sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  return cuda_status(kvq::launch_rope_axes(a, sms, static_cast<cudaStream_t>(stream)));
}

int kvq_rope_axes_phases(int32_t n_axes, const int32_t* sections, int32_t order, int32_t ladder, double base,
                         const kvq_rope_scaling* scaling, uint64_t* phases, uint8_t* axis_of, float* attn_factor) {
  if (n_axes < 1 || n_axes > kvq::kMaxAxes) return KVQ_ERR_UNSUPPORTED;
  if (order != KVQ_ROPE_CHUNKED && order != KVQ_ROPE_TURNS) return KVQ_ERR_UNSUPPORTED;
  if (ladder != KVQ_ROPE_SHARED && ladder != KVQ_ROPE_PER_AXIS) return KVQ_ERR_UNSUPPORTED;
  if (!sections || !phases || !axis_of) return KVQ_ERR_INVALID_ARG;
  int32_t n = 0;
  for (int32_t i = 0; i < n_axes; ++i) {
    if (sections[i] < 0 || sections[i] > kvq::kMaxRotaryDim / 2) return KVQ_ERR_INVALID_ARG;
    n += sections[i];
  }
  if (n < 1 || n > kvq::kMaxRotaryDim / 2) return KVQ_ERR_INVALID_ARG;
  // the axis of each frequency, and its place in its axis's own ladder
  uint8_t axis[kvq::kMaxRotaryDim / 2];
  int32_t place[kvq::kMaxRotaryDim / 2], used[kvq::kMaxAxes] = {};
  for (int32_t j = 0, turn = 0; j < n; ++j) {
    while (used[turn] == sections[turn]) turn = (turn + 1) % n_axes;
    axis[j] = static_cast<uint8_t>(turn);
    place[j] = used[turn]++;
    if (order == KVQ_ROPE_TURNS) turn = (turn + 1) % n_axes;
  }
  uint64_t made[kvq::kMaxRotaryDim / 2];
  float factor = 1.0f;
  if (ladder == KVQ_ROPE_SHARED) {
    const int st = kvq_rope_phases(2 * n, base, scaling, made, &factor);
    if (st != KVQ_OK) return st;
  } else {
    if (scaling && scaling->kind == KVQ_ROPE_DIVISORS) return KVQ_ERR_UNSUPPORTED;
    uint64_t own[kvq::kMaxRotaryDim / 2];
    for (int32_t i = 0; i < n_axes; ++i) {
      if (sections[i] == 0) continue;
      const int st = kvq_rope_phases(2 * sections[i], base, scaling, own, &factor);
      if (st != KVQ_OK) return st;
      for (int32_t j = 0; j < n; ++j)
        if (axis[j] == i) made[j] = own[place[j]];
    }
  }
  for (int32_t j = 0; j < n; ++j) {
    phases[j] = made[j];
    axis_of[j] = axis[j];
  }
  if (attn_factor) *attn_factor = factor;
  return KVQ_OK;
}

int kvq_rope_append_int8kv(const kvq_cache* cache, const void* q, void* q_out, int64_t q_stride, int64_t q_out_stride,
                           int32_t n_q_heads, const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                           int32_t n_tokens, const int32_t* seq_idx, const int32_t* slot, const int32_t* block_table,
                           int32_t num_seqs, int32_t max_blocks_per_seq, const int32_t* pos, int64_t pos_stride,
                           int32_t n_axes, const uint64_t* phases, const uint8_t* axis_of, int32_t rotary_dim,
                           int32_t rotary_offset, int32_t layout, float attn_factor, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  const int D = cache->head_dim, H = cache->n_kv_heads;
  if (n_tokens < 0 || n_q_heads < 0 || num_seqs <= 0 || max_blocks_per_seq <= 0) return KVQ_ERR_INVALID_ARG;
  if (layout != KVQ_ROPE_HALF && layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_UNSUPPORTED;
  if (rotary_dim <= 0 || rotary_dim % 2 != 0 || rotary_offset < 0 ||
      static_cast<long long>(rotary_offset) + rotary_dim > D)
    return KVQ_ERR_INVALID_ARG;
  if (rotary_dim % 16 != 0 || rotary_offset % 8 != 0) return KVQ_ERR_UNSUPPORTED;  // whole 16-byte words of pairs
  if (static_cast<long long>(n_q_heads) + H > 65535) return KVQ_ERR_UNSUPPORTED;
  if (!decode_row_ok(max_blocks_per_seq)) return KVQ_ERR_UNSUPPORTED;
  if (!std::isfinite(attn_factor)) return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return KVQ_OK;
  if (!k_new || !v_new || !seq_idx || !slot || !block_table || !pos || !phases) return KVQ_ERR_INVALID_ARG;
  if (n_q_heads && (!q || !q_out)) return KVQ_ERR_INVALID_ARG;
  const long long qd = static_cast<long long>(n_q_heads) * D, kd = static_cast<long long>(H) * D;
  if (n_tokens > 1) {
    if (k_stride < kd || v_stride < kd || (n_q_heads && (q_stride < qd || q_out_stride < qd))) return KVQ_ERR_INVALID_ARG;
    if (n_q_heads && q == q_out && q_stride != q_out_stride) return KVQ_ERR_INVALID_ARG;  // in place means the same rows
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || (n_q_heads && (q_stride % 8 != 0 || q_out_stride % 8 != 0)))
      return KVQ_ERR_MISALIGNED;
  }
  if (!aligned16(k_new) || !aligned16(v_new) || (n_q_heads && (!aligned16(q) || !aligned16(q_out)))) return KVQ_ERR_MISALIGNED;
  if (!aligned4(seq_idx) || !aligned4(slot) || !aligned4(block_table) || !aligned4(pos) ||
      reinterpret_cast<uintptr_t>(phases) % 8 != 0)
    return KVQ_ERR_MISALIGNED;
  kvq::RopeAppendArgs a{};
  st = rope_axes(pos, pos_stride, n_axes, axis_of, rotary_dim / 2, n_tokens, &a.axes);
  if (st != KVQ_OK) return st;
  const int sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks;
  a.n_kv_heads = H;
  a.head_dim = D;
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.q_stride = n_tokens > 1 ? q_stride : qd;
  a.q_out_stride = n_tokens > 1 ? q_out_stride : qd;
  a.k_stride = n_tokens > 1 ? k_stride : kd;
  a.v_stride = n_tokens > 1 ? v_stride : kd;
  a.n_q_heads = n_q_heads;
  a.n_tokens = n_tokens;
  a.seq_idx = seq_idx;
  a.slot = slot;
  a.block_table = block_table;
  a.num_seqs = num_seqs;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.phases = reinterpret_cast<const unsigned long long*>(phases);
  a.rotary_dim = rotary_dim;
  a.rotary_offset = rotary_offset;
  a.interleaved = layout == KVQ_ROPE_INTERLEAVED;
  a.attn_factor = attn_factor;
  a.status = status_ptr();
  return cuda_status(kvq::launch_rope_append(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t kvq_prefill_workspace_bytes(int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads, int32_t history_len,
                                   int32_t head_dim) {
  if (n_tokens <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || history_len < 0 || head_dim <= 0) return 0;
  return static_cast<size_t>(kvq::prefill_workspace(n_tokens, n_q_heads, n_kv_heads, history_len, head_dim).bytes);
}

static kvq::PrefillArgs prefill_args(const kvq_cache* cache, const void* q, int32_t n_tokens,
                                     int32_t n_q_heads, int32_t history_len,
                                     const int32_t* block_table_row, int32_t n_blocks_row,
                                     float softmax_scale, float* out, void* workspace) {
  kvq::PrefillArgs a{};
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks;
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.q = q;
  a.n_tokens = n_tokens;
  a.n_q_heads = n_q_heads;
  a.history_len = history_len;
  a.block_table_row = block_table_row;
  a.n_blocks_row = n_blocks_row;
  a.softmax_scale = softmax_scale;
  a.out = out;
  if (workspace) {
    const kvq::PrefillWorkspace w =
        kvq::prefill_workspace(n_tokens, n_q_heads, cache->n_kv_heads, history_len, cache->head_dim);
    char* base = static_cast<char*>(workspace);
    a.q_codes = reinterpret_cast<int8_t*>(base);
    a.q_scales = reinterpret_cast<float*>(base + w.off_q_scales);
    a.n_kv_tiles = w.n_kv_tiles;
    a.kw = reinterpret_cast<uint8_t*>(base + w.off_kw);
    a.vw = reinterpret_cast<uint8_t*>(base + w.off_vw);
    a.skw = reinterpret_cast<float*>(base + w.off_skw);
    a.svw = reinterpret_cast<float*>(base + w.off_svw);
    if (w.can_split) {
      a.part = reinterpret_cast<float*>(base + w.off_part);
      a.part_ml = reinterpret_cast<float*>(base + w.off_part_ml);
      a.part_cnt = reinterpret_cast<unsigned int*>(base + w.off_part_flags);
      a.part_ready = a.part_cnt + static_cast<long long>((n_tokens + 127) / 128) * n_q_heads;
      a.split_tail = kvq::prefill_split_tail(n_tokens, n_q_heads, history_len, device_sm_count());
    }
  }
  a.status = status_ptr();
  a.wait_budget = kvq::debug_wait_budget();
  a.fault = kvq::debug_fault_mode();
  return a;
}

int32_t kvq_device_accessible(const void* p) {
  if (!p) return 0;
  cudaPointerAttributes attr{};
  if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
    (void)cudaGetLastError();  // not a sticky error: clear it so the caller's next check is clean
    return 0;
  }
  if (attr.type == cudaMemoryTypeDevice || attr.type == cudaMemoryTypeManaged) return 1;
  return attr.type == cudaMemoryTypeHost && attr.devicePointer == p ? 1 : 0;
}

int32_t kvq_prefill_split_tiles(int32_t n_tokens, int32_t n_q_heads, int32_t history_len, int32_t n_sms) {
  return kvq::prefill_split_tail(n_tokens, n_q_heads, history_len, n_sms);
}

int kvq_attn_prefill_int8(const kvq_cache* cache, const void* q, int32_t n_tokens, int32_t n_q_heads,
                          int32_t history_len, const int32_t* block_table_row, int32_t n_blocks_row,
                          float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!q || !block_table_row || !out) return KVQ_ERR_INVALID_ARG;
  if (n_tokens <= 0 || n_q_heads <= 0 || history_len < 0 || n_blocks_row <= 0) return KVQ_ERR_INVALID_ARG;
  if (n_q_heads % cache->n_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if (static_cast<long long>(history_len) + n_tokens > static_cast<long long>(n_blocks_row) * KVQ_BLOCK_SIZE)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned4(block_table_row)) return KVQ_ERR_MISALIGNED;
  const size_t need = kvq_prefill_workspace_bytes(n_tokens, n_q_heads, cache->n_kv_heads, history_len,
                                                  cache->head_dim);
  if (!workspace || workspace_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  kvq::PrefillArgs a = prefill_args(cache, q, n_tokens, n_q_heads, history_len, block_table_row,
                                    n_blocks_row, softmax_scale, out, workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = kvq::launch_prefill_q_quant(a, s);
  if (e != cudaSuccess) return e == cudaErrorNotSupported ? KVQ_ERR_UNSUPPORTED : KVQ_ERR_CUDA;
  e = kvq::launch_prefill(a, s);
  if (e != cudaSuccess) return e == cudaErrorNotSupported ? KVQ_ERR_UNSUPPORTED : KVQ_ERR_CUDA;
  return KVQ_OK;
}

// Rows, keys, tile pairs and the elements of 128 queries' rows are counted in 32 bits, a tile of them ahead.
static bool prefill_window_sizes_ok(int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads, int32_t history_len, int32_t head_dim) {
  if (n_kv_heads > 65535 || n_q_heads / n_kv_heads > 1024 || n_q_heads >= (1 << 24) / head_dim) return false;
  constexpr long long kMost = 1LL << 30;
  const long long rows = static_cast<long long>(n_tokens) * (n_q_heads / n_kv_heads), keys = static_cast<long long>(history_len) + n_tokens;
  if (rows >= kMost || keys >= kMost) return false;
  return ((rows + 127) / 128) * ((keys + 127) / 128 + 1) * n_kv_heads < 1LL << 35;
}

// The plan of checked sizes on a GPU of n_sms SMs (any number gives the same workspace).
static kvq::PrefillWindowPlan prefill_window_plan_of(int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads,
                                                     int32_t history_len, int32_t window, int32_t n_sink, int32_t head_dim,
                                                     int n_sms) {
  constexpr int32_t kMost = 1 << 30;  // more keys than there are
  return kvq::prefill_window_plan(n_tokens, n_q_heads, n_kv_heads, history_len, std::min(window, kMost),
                                  std::min(n_sink, kMost), head_dim, n_sms);
}

size_t kvq_prefill_window_workspace_bytes(int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads, int32_t history_len,
                                          int32_t window, int32_t n_sink, int32_t head_dim) {
  if (n_tokens <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || history_len < 0 || window <= 0 || n_sink < 0) return 0;
  if (n_q_heads % n_kv_heads != 0 || (head_dim != 128 && head_dim != 256)) return 0;
  if (!prefill_window_sizes_ok(n_tokens, n_q_heads, n_kv_heads, history_len, head_dim)) return 0;
  return static_cast<size_t>(
      prefill_window_plan_of(n_tokens, n_q_heads, n_kv_heads, history_len, window, n_sink, head_dim, 1).bytes);
}

int kvq_attn_prefill_window_int8kv(const kvq_cache* cache, const void* q, int32_t n_tokens, int32_t n_q_heads,
                                   int32_t history_len, const int32_t* block_table_row, int32_t n_blocks_row,
                                   float softmax_scale, int32_t window, int32_t n_sink, void* out, int32_t out_type,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!q || !block_table_row || !out) return KVQ_ERR_INVALID_ARG;
  if (n_tokens <= 0 || n_q_heads <= 0 || history_len < 0 || n_blocks_row <= 0) return KVQ_ERR_INVALID_ARG;
  if (window <= 0 || n_sink < 0) return KVQ_ERR_INVALID_ARG;
  if (out_type != KVQ_OUT_FP32 && out_type != KVQ_OUT_BF16) return KVQ_ERR_UNSUPPORTED;
  const int H = cache->n_kv_heads, D = cache->head_dim;
  if (n_q_heads % H != 0) return KVQ_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if (static_cast<long long>(history_len) + n_tokens > static_cast<long long>(n_blocks_row) * KVQ_BLOCK_SIZE)
    return KVQ_ERR_INVALID_ARG;
  if (!prefill_window_sizes_ok(n_tokens, n_q_heads, H, history_len, D)) return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(out) || !aligned4(block_table_row)) return KVQ_ERR_MISALIGNED;
  if (!workspace) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  const int sms = device_sm_count();
  const kvq::PrefillWindowPlan p = prefill_window_plan_of(n_tokens, n_q_heads, H, history_len, window, n_sink, D, std::max(sms, 1));
  if (workspace_bytes < static_cast<size_t>(p.bytes)) return KVQ_ERR_WORKSPACE;
  if (sms <= 0) return KVQ_ERR_CUDA;
  kvq::PrefillWindowArgs a{};
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks;
  a.n_kv_heads = H;
  a.q = q;
  a.n_q_heads = n_q_heads;
  a.group = n_q_heads / H;
  a.history_len = history_len;
  a.group_inv = a.group == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + a.group - 1) / a.group);
  a.n_rows = n_tokens * a.group;
  a.n_keys = history_len + n_tokens;
  a.window = std::min(window, 1 << 30);
  a.n_sink = std::min(n_sink, 1 << 30);
  a.block_table_row = block_table_row;
  a.c2 = softmax_scale * 1.44269504088896341f;
  a.out = out;
  a.out_bf16 = out_type == KVQ_OUT_BF16;
  a.row_tiles = p.row_tiles;
  a.first_tile = p.first_tile;
  a.sink_tiles = p.sink_tiles;
  a.key_tiles = p.key_tiles;
  a.line = p.line;
  char* ws = static_cast<char*>(workspace);
  a.k_tiles = reinterpret_cast<uint8_t*>(ws);
  a.v_tiles = reinterpret_cast<uint8_t*>(ws + p.off_v);
  a.par = reinterpret_cast<float*>(ws + p.off_par);
  a.part_ml = reinterpret_cast<float2*>(ws + p.off_ml);
  a.part = reinterpret_cast<float4*>(ws + p.off_part);
  a.status = status_ptr();
  a.wait_budget = kvq::debug_wait_budget();
  a.fault = kvq::debug_fault_mode();
  return cuda_status(kvq::launch_prefill_window(a, D, p.runs, static_cast<cudaStream_t>(stream)));
}

size_t kvq_prefill_first_workspace_bytes(int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads,
                                         int32_t head_dim) {
  if (n_tokens <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || (head_dim != 128 && head_dim != 256)) return 0;
  return static_cast<size_t>(kvq::prefill_workspace(n_tokens, n_q_heads, n_kv_heads, 0, head_dim, 2).bytes);
}

int kvq_attn_prefill_first_bf16(const kvq_cache* cache, const void* q, const void* k_new, const void* v_new,
                                int32_t n_tokens, int32_t n_q_heads, const int32_t* block_table_row,
                                int32_t n_blocks_row, float softmax_scale, float* out, void* workspace,
                                size_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!q || !k_new || !v_new || !block_table_row || !out) return KVQ_ERR_INVALID_ARG;
  if (n_tokens <= 0 || n_q_heads <= 0 || n_blocks_row <= 0) return KVQ_ERR_INVALID_ARG;
  if (n_q_heads % cache->n_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if (static_cast<long long>(n_tokens) > static_cast<long long>(n_blocks_row) * KVQ_BLOCK_SIZE)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(out) || !aligned4(block_table_row))
    return KVQ_ERR_MISALIGNED;
  const kvq::PrefillWorkspace w = kvq::prefill_workspace(n_tokens, n_q_heads, cache->n_kv_heads, 0, cache->head_dim, 2);
  if (!workspace || workspace_bytes < static_cast<size_t>(w.bytes)) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  kvq::PrefillArgs a = prefill_args(cache, q, n_tokens, n_q_heads, 0, block_table_row, n_blocks_row,
                                    softmax_scale, out, nullptr);
  char* base = static_cast<char*>(workspace);
  a.q_f16 = reinterpret_cast<uint16_t*>(base);
  a.q_scales = reinterpret_cast<float*>(base + w.off_q_scales);
  a.n_kv_tiles = w.n_kv_tiles;
  a.kw = reinterpret_cast<uint8_t*>(base + w.off_kw);
  a.vw = reinterpret_cast<uint8_t*>(base + w.off_vw);
  a.skw = reinterpret_cast<float*>(base + w.off_skw);
  a.svw = reinterpret_cast<float*>(base + w.off_svw);
  a.k_src = k_new;
  a.v_src = v_new;
  return cuda_status(kvq::launch_prefill_first(a, static_cast<cudaStream_t>(stream)));
}

int kvq_attn_prefill_int8_qcodes(const kvq_cache* cache, const int8_t* q_codes, const float* q_scales,
                                 int32_t n_tokens, int32_t n_q_heads, int32_t history_len,
                                 const int32_t* block_table_row, int32_t n_blocks_row, float softmax_scale,
                                 float* out, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!q_codes || !q_scales || !block_table_row || !out) return KVQ_ERR_INVALID_ARG;
  if (n_tokens <= 0 || n_q_heads <= 0 || history_len < 0 || n_blocks_row <= 0) return KVQ_ERR_INVALID_ARG;
  if (n_q_heads % cache->n_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if (static_cast<long long>(history_len) + n_tokens > static_cast<long long>(n_blocks_row) * KVQ_BLOCK_SIZE)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q_codes) || !aligned4(q_scales) || !aligned16(out) || !aligned4(block_table_row))
    return KVQ_ERR_MISALIGNED;
  const size_t need = kvq_prefill_workspace_bytes(n_tokens, n_q_heads, cache->n_kv_heads, history_len,
                                                  cache->head_dim);
  if (!workspace || workspace_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  kvq::PrefillArgs a = prefill_args(cache, nullptr, n_tokens, n_q_heads, history_len, block_table_row,
                                    n_blocks_row, softmax_scale, out, workspace);
  a.q_codes = const_cast<int8_t*>(q_codes);
  a.q_scales = const_cast<float*>(q_scales);
  return cuda_status(kvq::launch_prefill(a, static_cast<cudaStream_t>(stream)));
}

size_t kvq_sparse_workspace_bytes(int32_t n_blocks_row, int32_t n_kv_heads, int32_t head_dim) {
  if (n_blocks_row <= 0 || n_kv_heads <= 0 || (head_dim != 128 && head_dim != 256)) return 0;
  return kvq::sparse_workspace_bytes(n_blocks_row, n_kv_heads, head_dim);
}

int kvq_attn_sparse_int8kv(const kvq_cache* cache, const void* q, int32_t n_queries, int32_t n_q_heads,
                           const int32_t* cell_offsets, const int32_t* cells,
                           const int32_t* block_table_row, int32_t n_blocks_row, float softmax_scale,
                           float* out, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!q || !cell_offsets || !cells || !block_table_row || !out) return KVQ_ERR_INVALID_ARG;
  if (n_queries <= 0 || n_q_heads <= 0 || n_blocks_row <= 0) return KVQ_ERR_INVALID_ARG;
  if (cache->n_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;  // grid y of both kernels
  if (n_q_heads % cache->n_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  const int G = n_q_heads / cache->n_kv_heads;
  if (G > 16) return KVQ_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < kvq::sparse_workspace_bytes(n_blocks_row, cache->n_kv_heads, cache->head_dim))
    return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  if (!aligned16(q) || !aligned16(out)) return KVQ_ERR_MISALIGNED;
  if (!aligned4(cell_offsets) || !aligned4(cells) || !aligned4(block_table_row)) return KVQ_ERR_MISALIGNED;
  kvq::SparseArgs a{};
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks;
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.q = q;
  a.n_queries = n_queries;
  a.n_q_heads = n_q_heads;
  a.cell_offsets = cell_offsets;
  a.cells = cells;
  a.block_table_row = block_table_row;
  a.n_blocks_row = n_blocks_row;
  a.softmax_scale = softmax_scale;
  a.out = out;
  a.records = static_cast<uint8_t*>(workspace);
  a.status = status_ptr();
  a.wait_budget = kvq::debug_wait_budget();
  a.fault = kvq::debug_fault_mode();
  return cuda_status(kvq::launch_sparse(a, static_cast<cudaStream_t>(stream)));
}

int kvq_debug_stream_floor(const kvq_cache* cache, int32_t batch, const int32_t* block_table,
                           int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t max_ctx, int32_t split_rows,
                           void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!block_table || !ctx_lens || batch <= 0 || batch > 65535 || max_blocks_per_seq <= 0 || max_ctx <= 0)
    return KVQ_ERR_INVALID_ARG;
  if (split_rows < 0 || split_rows % KVQ_BLOCK_SIZE != 0) return KVQ_ERR_INVALID_ARG;
  if (!decode_row_ok(max_blocks_per_seq)) return KVQ_ERR_UNSUPPORTED;
  if (!aligned4(block_table) || !aligned4(ctx_lens)) return KVQ_ERR_MISALIGNED;
  if (split_rows == 0) {
    const int sms = device_sm_count();
    if (sms <= 0) return KVQ_ERR_CUDA;
    split_rows = kvq_decode_auto_split_rows(batch, cache->n_kv_heads, cache->head_dim, max_ctx, sms);
  }
  const long long n_split = (static_cast<long long>(max_ctx) + split_rows - 1) / split_rows;
  if (n_split > kvq::kMaxSplits) return KVQ_ERR_UNSUPPORTED;
  kvq::DecodeArgs a{};
  a.k = cache->k;
  a.v = cache->v;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks;
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.batch = batch;
  a.block_table = block_table;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.ctx_lens = ctx_lens;
  a.max_ctx = max_ctx;
  a.split_rows = split_rows;
  a.n_split = static_cast<int>(n_split);
  a.status = status_ptr();
  a.wait_budget = kvq::debug_wait_budget();
  return cuda_status(kvq::launch_stream_floor(a, static_cast<cudaStream_t>(stream)));
}

int kvq_debug_prefill_q_codes(const void* q, int32_t n_tokens, int32_t n_q_heads, int32_t head_dim,
                              int8_t* q_codes, float* q_scales, void* stream) {
  if (!q || !q_codes || !q_scales || n_tokens <= 0 || n_q_heads <= 0) return KVQ_ERR_INVALID_ARG;
  if (head_dim != 128 && head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(q_codes) || !aligned4(q_scales)) return KVQ_ERR_MISALIGNED;
  kvq::PrefillArgs a{};
  a.head_dim = head_dim;
  a.q = q;
  a.n_tokens = n_tokens;
  a.n_q_heads = n_q_heads;
  a.q_codes = q_codes;
  a.q_scales = q_scales;
  a.status = status_ptr();
  return cuda_status(kvq::launch_prefill_q_quant(a, static_cast<cudaStream_t>(stream)));
}

int kvq_debug_prefill_qk_int32(const kvq_cache* cache, const int8_t* q_codes, const float* q_scales,
                               int32_t n_tokens, int32_t n_q_heads, int32_t history_len,
                               const int32_t* block_table_row, int32_t n_blocks_row, float softmax_scale,
                               int32_t split_tiles, int32_t q_head, int32_t q0, int32_t k0, int32_t nk,
                               int32_t* s_out, float* out, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!q_codes || !q_scales || !block_table_row || !s_out || !out) return KVQ_ERR_INVALID_ARG;
  if (n_tokens <= 0 || n_q_heads <= 0 || history_len < 0 || n_blocks_row <= 0) return KVQ_ERR_INVALID_ARG;
  if (n_q_heads % cache->n_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if (static_cast<long long>(history_len) + n_tokens > static_cast<long long>(n_blocks_row) * KVQ_BLOCK_SIZE)
    return KVQ_ERR_INVALID_ARG;
  // the window: one unit (query tile q0 / 128 of q_head) and whole key tiles it computes
  if (q_head < 0 || q_head >= n_q_heads || q0 < 0 || q0 >= n_tokens || q0 % 128 != 0) return KVQ_ERR_INVALID_ARG;
  const long long unit_tiles = (static_cast<long long>(history_len) + std::min(q0 + 127, n_tokens - 1)) / 128 + 1;
  if (k0 < 0 || nk <= 0 || k0 % 128 != 0 || nk % 128 != 0 || k0 + static_cast<long long>(nk) > 128 * unit_tiles)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q_codes) || !aligned4(q_scales) || !aligned16(out) || !aligned16(s_out) || !aligned4(block_table_row))
    return KVQ_ERR_MISALIGNED;
  const size_t need = kvq_prefill_workspace_bytes(n_tokens, n_q_heads, cache->n_kv_heads, history_len,
                                                  cache->head_dim);
  if (!workspace || workspace_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_MISALIGNED;
  kvq::PrefillArgs a = prefill_args(cache, nullptr, n_tokens, n_q_heads, history_len, block_table_row,
                                    n_blocks_row, softmax_scale, out, workspace);
  if (split_tiles >= 0) {
    // a forced split: every lead segment keeps at least one tile, as the automatic choice does
    const long long shortest = (static_cast<long long>(history_len) + std::min(127, n_tokens - 1)) / 128 + 1;
    const bool can = kvq::prefill_workspace(n_tokens, n_q_heads, cache->n_kv_heads, history_len, cache->head_dim)
                         .can_split;
    if (split_tiles > 0 && (!can || split_tiles > shortest - 1)) return KVQ_ERR_INVALID_ARG;
    a.split_tail = split_tiles;
  }
  a.q_codes = const_cast<int8_t*>(q_codes);
  a.q_scales = const_cast<float*>(q_scales);
  a.dbg_q_head = q_head;
  a.dbg_q0 = q0;
  a.dbg_k0 = k0;
  a.dbg_nk = nk;
  a.dbg_s_out = s_out;
  cudaError_t e = kvq::launch_prefill_qk_debug(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return e == cudaErrorNotSupported ? KVQ_ERR_UNSUPPORTED : KVQ_ERR_CUDA;
  return KVQ_OK;
}

}  // extern "C"
