// kvq_launch.h — internal launcher interface between the C ABI (api.cu) and the kernels.
// Host-side validation happens in api.cu; the launchers assume valid arguments.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "kvq.h"

namespace kvq {

struct QuantWriteArgs {
  int8_t* k;
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int num_blocks, n_kv_heads, head_dim;
  const void* k_new;
  const void* v_new;
  int n_tokens;
  const int32_t* seq_idx;
  const int32_t* pos;
  const int32_t* block_table;
  int num_seqs, max_blocks_per_seq;
  unsigned int* status;
};
cudaError_t launch_quant_write(const QuantWriteArgs& a, cudaStream_t stream);

// Fused producer: RoPE on Q and K, the quantisation rule on Q, K and V; K/V into the cache.
struct RopeQuantArgs {
  QuantWriteArgs kv;      // the cache, k_new / v_new, tokens, slots
  const void* q;          // bf16 [T][Hq][D] or nullptr
  int n_q_heads;
  const float* cos_sin;   // fp32 [max_pos][rotary_dim]: cos of rotary_dim / 2 frequencies, then sin
  int max_pos, rotary_dim;
  int8_t* q_codes;        // [T][Hq][D] or nullptr
  float* q_scales;        // [T][Hq] or nullptr
  uint16_t* q_rot;        // bf16 [T][Hq][D] or nullptr
  int q_heads_per_warp;   // set by launch_rope_quant_write
};
cudaError_t launch_rope_quant_write(const RopeQuantArgs& a, cudaStream_t stream);

// Decode: nq query rows per sequence (1 for plain decode; row i sees keys
// t < ctx - nq + 1 + i).  Stage 1 (both routes) walks a key range of one (sequence, KV head)
// for all G * nq rows; the single-CTA route writes `out` directly, the split route writes
// partials that stage 2 merges.
struct DecodeArgs {
  int8_t* k;          // the cache (written only by the fused step)
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int num_blocks, n_kv_heads, head_dim;
  const void* q;  // bf16 [B][nq][Hq][D]
  int batch, nq, n_q_heads;
  const int32_t* block_table;
  int max_blocks_per_seq;
  const int32_t* ctx_lens;
  int max_ctx;
  float softmax_scale;
  // fused step: bf16 [B][nq][Hkv][D] K / V of each sequence's nq newest tokens, quantised
  // into the cache by stage 1 before it reads their page; nullptr for attention only
  const void* k_new;
  const void* v_new;
  float* out;          // fp32 [B][nq][Hq][D]
  float* part_acc;     // fp32 [B][nq][Hq][n_split][D]  (split route)
  float* part_stats;   // fp32 [B][nq][Hq][n_split][4]  (split route: m_s, m_z, l, with scores: l with NaN kept)
  int split_rows;      // keys per split (split route); ignored by the single route
  int n_split;         // splits per sequence in the grid (split route)
  unsigned int* status;
  cudaEvent_t ev_begin;  // optional events around the stage-1 launch
  cudaEvent_t ev_end;
  // bounded waits: budget in SM clock cycles; fault: test-only injection (kvq_debug_fault_inject),
  // 1 = CTA 0's first team does not issue the copy of its second page
  long long wait_budget;
  int fault;
  // step with accumulated weights only: the scores of every (sequence, KV head, query row) in log2
  // units, fp32 [B][Hkv][G * nq][scores_stride]
  float* scores;
  long long scores_stride;
  // windowed step only: a row at position p sees keys t <= p with t > p - window or t < n_sink; both at most max_ctx
  int window, n_sink;
};
// Pages that a windowed step does not read: of a sequence of ctx keys whose first of nq rows is at ctx - nq, those
// behind the pages of the first n_sink keys and before the first row's window.  The others are counted without them
// (a virtual length ctx - 16 * skipped, virtual pages): page v is page v of the block-table row below `sink_pages`, else
// page v + skipped.
struct WindowMap {
  int sink_pages, skipped;
};
__host__ __device__ inline WindowMap window_map(int ctx, int nq, int window, int n_sink) {
  WindowMap m;
  m.sink_pages = n_sink / KVQ_BLOCK_SIZE + (n_sink % KVQ_BLOCK_SIZE != 0);
  const int low = (ctx >= nq ? ctx - nq + 1 : 0) - window;  // the first key of the first row's window (no row's: below 0)
  m.skipped = low > 0 && low / KVQ_BLOCK_SIZE > m.sink_pages ? low / KVQ_BLOCK_SIZE - m.sink_pages : 0;
  return m;
}
enum class DecodeRoute { kSingle = 1, kSplit = 2 };
// Test-only fault injection and wait budget of the kernels launched next (kvq_debug_fault_inject).
int debug_fault_mode();
long long debug_wait_budget();
constexpr int kMaxSplits = 16384;  // decode_plan makes no more: a merging CTA has a weight for each in shared memory
size_t decode_workspace_bytes(int batch, int n_q_heads, int max_ctx, int head_dim, int split_rows);
// The route, split size and workspace bytes a decode call with these (checked) arguments takes:
// the automatic split size of this GPU when opts->split_rows is 0.  A kvq_status.
struct DecodePlan {
  bool split;
  int split_rows, n_split;
  size_t bytes;
};
int decode_plan(const kvq_cache* cache, int32_t batch, int32_t nq, int32_t n_q_heads, int32_t max_ctx,
                const kvq_decode_opts* opts, DecodePlan* plan);
cudaError_t launch_decode(const DecodeArgs& a, DecodeRoute route, cudaStream_t stream, int* launched);
cudaError_t launch_step_window(const DecodeArgs& a, DecodeRoute route, cudaStream_t stream, int* launched);
// the stage-1 kernel's K/V stream alone, split route geometry (kvq_debug_stream_floor)
cudaError_t launch_stream_floor(const DecodeArgs& a, cudaStream_t stream);

// The split route's stage 1 that also writes the scores, then one launch that merges the splits and adds
// each key's weight (summed over the rows of its KV head) to acc.
struct StepAccumArgs {
  DecodeArgs d;
  float* acc;          // fp32 [B][Hkv][acc_stride]
  long long acc_stride;
  int32_t* slot_pos;   // int32 [B][Hkv][acc_stride] or nullptr: positions of the new tokens go here
  const int32_t* pos;  // int32 [B]: position of each sequence's first new token
  int merge_blocks, key_blocks;  // set by launch_step_accum: CTAs that merge, CTAs of keys per (sequence, KV head)
};
// The tail's CTAs can be counted (the grid's x).
bool step_accum_grid_ok(const DecodeArgs& d);
cudaError_t launch_step_accum(const StepAccumArgs& a, cudaStream_t stream, int* launched);

// Attention weights of a chunk of queries, summed per key.  [0]: the row pass, [1]: the column pass.
struct ChunkWeightsPlan {
  int row_tiles, key_tiles;   // 128 (query, head) rows of a KV head; 128 keys
  int a_rows[2], units[2];    // rows of an A unit (128 or 256), A units of a KV head
  long long line[2];          // (A unit, B tile) pairs of one KV head
  int runs[2], n_part[2];     // CTAs, and the most parts one 128-row A tile is cut into
  bool widen_once;            // the key tiles are widened by a pass of their own
  long long off_nm, off_il, off_q, off_col, off_k, off_kpar, off_kvalid, bytes;
};
ChunkWeightsPlan chunk_weights_plan(int n_tokens, int n_q_heads, int n_kv_heads, int history_len, int head_dim,
                                    int n_sms);
struct ChunkWeightsArgs {
  const int8_t* k;
  const float* k_scale;
  int num_blocks, n_kv_heads, head_dim;
  const void* q;  // bf16 [T][Hq][D]
  int n_q_heads, group, history_len, n_rows, n_keys;  // n_rows = T * group
  const int32_t* block_table_row;
  float c2;       // softmax_scale * log2(e)
  float* acc;     // fp32 [Hkv][acc_stride]
  long long acc_stride;
  int row_tiles, key_tiles;
  int a_rows[2], units[2];
  long long line[2];
  int runs[2], n_part[2];
  float2* row_part;  // workspace [Hkv][A tiles][n_part[0]][128]: (max, sum) parts, sum < 0: dropped
  float* row_nm;     // workspace [Hkv * row_tiles][128]: minus the row's maximum
  float* row_il;     // workspace: 1 / the row's sum, 0 for a row that gives nothing
  uint8_t* q_tiles;  // workspace [Hkv * row_tiles][D / 64 pieces of 16 KB]: the queries, bf16, in tile order
  float* col_part;   // workspace [Hkv][A tiles][n_part[1]][128]
  // workspace, when the key tiles are widened once (else nullptr): bf16 in tile order, score factors, key bits
  uint8_t* k_tiles;   // [Hkv * key_tiles][D / 64 pieces of 16 KB]
  float* k_par;       // [Hkv * key_tiles][128]
  uint32_t* k_valid;  // [Hkv * key_tiles][4]
  unsigned int* status;
  long long wait_budget;
  int fault;
};
cudaError_t launch_chunk_weights(const ChunkWeightsArgs& a, cudaStream_t stream);

// A chunk of prompt queries with a sliding window and first keys that stay visible.
struct PrefillWindowPlan {
  int row_tiles;         // 128 (query, head) rows of a KV head
  int first_tile;        // the first 128-key tile of any query's window
  int sink_tiles;        // tiles of first keys before it that are kept as well
  int key_tiles;         // tiles of a KV head in the workspace: sink_tiles, then first_tile on
  long long line;        // (row tile, key tile) pairs of one KV head
  int runs;              // CTAs, each with an equal run of all KV heads' pairs
  long long off_v, off_par, off_ml, off_part, bytes;
};
PrefillWindowPlan prefill_window_plan(int n_tokens, int n_q_heads, int n_kv_heads, int history_len, int window,
                                      int n_sink, int head_dim, int n_sms);
struct PrefillWindowArgs {
  const int8_t* k;
  const int8_t* v;
  const float* k_scale;
  const float* v_scale;
  int num_blocks, n_kv_heads;
  const void* q;  // bf16 [T][Hq][D]
  int n_q_heads, group, history_len, n_rows, n_keys;  // n_rows = T * group
  uint32_t group_inv;  // ceil(2^32 / group), 0 for 1
  int window, n_sink;
  const int32_t* block_table_row;
  float c2;       // softmax_scale * log2(e)
  void* out;      // [T][Hq][D], bf16 or fp32
  int out_bf16;
  int row_tiles, first_tile, sink_tiles, key_tiles;
  long long line;
  uint8_t* k_tiles;   // workspace [Hkv][key_tiles][D / 64 pieces of 16 KB]: codes in bf16, tile order
  uint8_t* v_tiles;   // workspace, likewise in fp16
  float* par;         // workspace [Hkv][key_tiles][3][128]: score factor, log2 of the V scale, its inverse
  float2* part_ml;    // workspace [runs][2][128]: (reference, sum) of a unit's part, sum < 0: dropped
  float4* part;       // workspace [runs][2][128 * D / 4]: its numerator, as the softmax threads hold it
  unsigned int* status;
  long long wait_budget;
  int fault;
};
cudaError_t launch_prefill_window(const PrefillWindowArgs& a, int head_dim, int runs, cudaStream_t stream);

// Eviction by accumulated weight.
struct EvictArgs {
  int8_t* k;
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int num_blocks, n_kv_heads, head_dim;
  int batch;
  const int32_t* block_table;
  int max_blocks_per_seq;
  const int32_t* ctx_lens;
  int max_ctx, keep, n_sink, n_recent;
  const float* acc;          // [B][Hkv][acc_stride]
  const int32_t* slot_pos;   // [B][Hkv][acc_stride]
  long long acc_stride;
  float* acc_out;            // [B][Hkv][out_stride]
  int32_t* slot_pos_out;
  long long out_stride;
  int32_t* new_lens;         // [B]
  // workspace: per (sequence, KV head) the slots that move (ascending), for every slot of the pages below
  // the budget the physical slot that moves into it, whether anything moves, and which slots are kept
  int max_moves, n_pages;
  int32_t* move_src;         // [units][max_moves]
  int32_t* slot_map;         // [units][16 * n_pages]
  int32_t* n_moves;          // [units]
  int n_words;               // > 0: words of 32 slots, when a CTA's range can pass what it keeps in shared memory
  uint32_t* words;           // [units][n_words][2]
  unsigned int* status;
};
struct EvictWorkspace {
  int max_moves, n_pages, n_words;
  long long off_map, off_count, off_words, bytes;
};
EvictWorkspace evict_workspace(int batch, int n_kv_heads, int max_ctx, int keep);
cudaError_t launch_evict(const EvictArgs& a, int n_sms, cudaStream_t stream);

// Rotation of bf16 rows by position.
struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  long long q_stride, k_stride, q_out_stride, k_out_stride;  // elements from a token to the next
  int n_q_heads, n_kv_heads, head_dim, n_tokens;
  const int32_t* pos;
  const unsigned long long* phases;  // [rotary_dim / 2]: turns per position * 2^64
  int rotary_dim, rotary_offset, interleaved;
  float attn_factor;
  int columns, head_groups;  // set by launch_rope
};
cudaError_t launch_rope(const RopeArgs& a, int n_sms, cudaStream_t stream);

// Positions on several axes, and the axis of each frequency: two bits each.
constexpr int kMaxAxes = 4;
constexpr int kMaxRotaryDim = 1024;
struct RopeAxes {
  const int32_t* pos;    // [n][pos_stride]
  long long pos_stride;
  int n;
  uint32_t map[kMaxRotaryDim / 2 / 16];
};
struct RopeAxesArgs : RopeArgs {  // pos is not used
  RopeAxes axes;
  float sin_factor;  // attn_factor, negative for the inverse
};
cudaError_t launch_rope_axes(const RopeAxesArgs& a, int n_sms, cudaStream_t stream);

// Rotation, quantisation and append of new tokens.
struct RopeAppendArgs {
  int8_t* k;
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int num_blocks, n_kv_heads, head_dim;
  const uint16_t* q;      // bf16 rows, a token's q_stride elements after the one before
  uint16_t* q_out;
  const uint16_t* k_new;
  const uint16_t* v_new;
  long long q_stride, q_out_stride, k_stride, v_stride;
  int n_q_heads, n_tokens;
  const int32_t* seq_idx;
  const int32_t* slot;
  const int32_t* block_table;
  int num_seqs, max_blocks_per_seq;
  const unsigned long long* phases;  // [rotary_dim / 2]
  int rotary_dim, rotary_offset, interleaved;
  float attn_factor;
  RopeAxes axes;
  unsigned int* status;
  int q_heads, kv_heads, kv_first;  // of a block, set by launch_rope_append
};
cudaError_t launch_rope_append(const RopeAppendArgs& a, int n_sms, cudaStream_t stream);

struct SparseArgs {
  const int8_t* k;
  const int8_t* v;
  const float* k_scale;
  const float* v_scale;
  int num_blocks, n_kv_heads, head_dim;
  const void* q;  // bf16 [N][Hq][D]
  int n_queries, n_q_heads;
  const int32_t* cell_offsets;
  const int32_t* cells;
  const int32_t* block_table_row;
  int n_blocks_row;
  float softmax_scale;
  float* out;
  uint8_t* records;  // workspace: gather records [n_blocks_row][Hkv][16][2D + 16]
  unsigned int* status;
  long long wait_budget;  // SM clock cycles a bounded wait may take
  int fault;              // test-only fault injection (kvq_debug_fault_inject), 0: none
};
size_t sparse_workspace_bytes(int n_blocks_row, int n_kv_heads, int head_dim);
cudaError_t launch_sparse(const SparseArgs& a, cudaStream_t stream);

struct PrefillArgs {
  int8_t* k;          // the cache (written only by the first-chunk pass)
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int num_blocks, n_kv_heads, head_dim;
  const void* q;  // bf16 [T][Hq][D]
  int n_tokens, n_q_heads, history_len;
  const int32_t* block_table_row;
  int n_blocks_row;
  float softmax_scale;
  float* out;        // fp32 [T][Hq][D]
  int8_t* q_codes;   // workspace int8 [T][Hq][D]
  float* q_scales;   // workspace fp32 [T][Hq]
  // first chunk in high precision: fp16 Q (q * 2^e per row) in place of the codes, and the
  // chunk's own bf16 K/V [T][Hkv][D] (also written into the int8 cache by the pre-pass)
  uint16_t* q_f16;   // workspace fp16 [T][Hq][D]
  const void* k_src;
  const void* v_src;
  // workspace: K/V of every (KV head, 128-key tile) widened to the attention kernel's
  // shared-memory operand image, and the tiles' key / value scales
  int n_kv_tiles;
  uint8_t* kw;       // [Hkv][n_kv_tiles][D/64 pieces of 16 KB]
  uint8_t* vw;       // [Hkv][n_kv_tiles][D/64 pieces of 16 KB]
  float* skw;        // [Hkv][n_kv_tiles][128]
  float* svw;        // [Hkv][n_kv_tiles][128]
  unsigned int* status;
  // key-range split (int8 path): with split_tail > 0 each unit (128 query rows, query head) runs
  // as two CTAs, a lead segment (key tiles [0, js)) and a tail segment (tiles [js, n_tiles)),
  // js = min(n_tiles - split_tail, history_len / 128); whichever finishes first leaves its
  // numerator and (m, l) in part / part_ml, and the other merges them into out
  int split_tail;
  float* part;               // workspace fp32 [units][128][D]
  float* part_ml;            // workspace fp32 [units][128][2]
  unsigned int* part_cnt;    // workspace [units]: segments arrived (zeroed by the widen pass)
  unsigned int* part_ready;  // workspace [units]: the first segment's values are written
  // debug QK tile (kvq_debug_prefill_qk_int32)
  int dbg_q_head, dbg_q0, dbg_k0, dbg_nk;
  int32_t* dbg_s_out;
  // bounded waits: budget in SM clock cycles; fault: test-only injection (kvq_debug_fault_inject),
  // 2 = the producer of attention CTA 0 does not issue its fourth piece copy
  long long wait_budget;
  int fault;
};
struct PrefillWorkspace {
  int n_kv_tiles;
  long long off_q_scales, off_kw, off_vw, off_skw, off_svw;
  long long off_part, off_part_ml, off_part_flags;  // only when the key range may be split
  bool can_split;
  long long bytes;
};
PrefillWorkspace prefill_workspace(int n_tokens, int n_q_heads, int n_kv_heads, int history_len, int head_dim,
                                   int q_elem_bytes = 1);
// Tail length (in 128-key tiles) of the key-range split of the int8 prefill at this shape on
// n_sms SMs, 0 for no split: the choice that minimises the modelled finish time of the
// longest-first dispatch (one attention CTA per SM).
int prefill_split_tail(int n_tokens, int n_q_heads, int history_len, int n_sms);
cudaError_t launch_prefill_q_quant(const PrefillArgs& a, cudaStream_t stream);
cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream);
// first chunk: Q to fp16, the chunk's K/V into the cache and into fp16 operand pieces, then the
// attention in high precision (fp16 P)
cudaError_t launch_prefill_first(const PrefillArgs& a, cudaStream_t stream);
cudaError_t launch_prefill_qk_debug(const PrefillArgs& a, cudaStream_t stream);

}  // namespace kvq
