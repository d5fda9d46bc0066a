// rope_append.cu — new tokens into the int8 paged cache in one call: q and k rotated by positions that need not be
// slots (one axis or several), k and v quantised and written to their slots, q written rotated in bf16.
//
// "gfx936 DCU上实现INT8 KV与INT8 MMAC Attention推理优化" §2.2 has one producer read Q/K/V, rotate, quantise and write;
// kvq_rope_quant_write is that producer for positions that are slots and a cos / sin table.  A cache that has evicted
// tokens, and positions with several axes, have neither: here the position comes from the plan of kvq_rope_axes_bf16.
//
// The codes are decided by fp32 values, so these are specified to the bit: cos and sin are the fp32 numbers nearest to
// factor cos(2 pi turns) and factor sin(2 pi turns), and
//     x' = RN(RN(x c) - RN(y s)),   y' = RN(RN(y c) + RN(x s)),
// then the rule of kvq_quant_write on the fp32 row.  cos_sin_exact below gives those numbers: a table of 256 angles
// in pairs of fp32 and a short polynomial of what is left, about 50 operations a pair, within 2^-45 of the value, which
// leaves one cos in some 2^19 rounded the other way (and a code only where its quotient lies at a tie as well).
//
// Bound: bytes, each row in once, q out once, half a byte out for each byte of k and v in.  A block takes 16 tokens and
// some query heads, or one KV head; a thread owns one column of a token (8 pairs, two 16-byte words of a row), so its 8 cos and sin serve all
// its heads and stay in registers.  The 16 tokens are counted from a page boundary where the first token's slot says
// where one is, so that a chunk's V codes leave a page at a time, 16 bytes a dimension.
#include "kvq_dev.cuh"
#include "kvq_launch.h"
#include "quant_rule.cuh"
#include "rope_dev.cuh"

namespace kvq {

namespace {

// ---------------------------------------------------------------- cos and sin to the nearest fp32
constexpr int kAngles = 256;  // entries of a turn
struct alignas(16) AngleEntry {
  float ch, cl, sh, sl;  // cos and sin as hi + lo
};
struct AngleTable {
  AngleEntry e[kAngles];
};

// Taylor series in double for |x| <= pi / 4 (the terms left out are below 1e-19).
constexpr double taylor(double x, bool sine) {
  double term = sine ? x : 1.0, sum = 0.0, n = sine ? 1.0 : 0.0;
  double terms[12] = {};
  for (int i = 0; i < 12; ++i) {
    terms[i] = term;
    term *= -x * x / ((n + 1.0) * (n + 2.0));
    n += 2.0;
  }
  for (int i = 11; i >= 0; --i) sum += terms[i];  // the small ones first
  return sum;
}

constexpr AngleTable make_angles() {
  AngleTable t{};
  for (int k = 0; k < kAngles; ++k) {
    const int q = (k + kAngles / 8) / (kAngles / 4);  // nearest quarter turn
    const double x = (k - q * (kAngles / 4)) * (6.283185307179586477 / kAngles);
    const double cr = taylor(x, false), sr = taylor(x, true);
    const double c = q % 4 == 0 ? cr : q % 4 == 1 ? -sr : q % 4 == 2 ? -cr : sr;
    const double s = q % 4 == 0 ? sr : q % 4 == 1 ? cr : q % 4 == 2 ? -sr : -cr;
    t.e[k].ch = static_cast<float>(c);
    t.e[k].cl = static_cast<float>(c - static_cast<double>(static_cast<float>(c)));
    t.e[k].sh = static_cast<float>(s);
    t.e[k].sl = static_cast<float>(s - static_cast<double>(static_cast<float>(s)));
  }
  return t;
}

__device__ constexpr AngleTable kTable = make_angles();

// hi + lo - p - v, rounded once after the multiplication by f.  |hi| >= |p| >= |v| or hi = 0 (then v = 0 too).
__device__ __forceinline__ float join(float hi, float p, float v, float lo, float f) {
  const float s1 = __fsub_rn(hi, p), t1 = __fsub_rn(__fsub_rn(hi, s1), p);
  const float s2 = __fsub_rn(s1, v), t2 = __fsub_rn(__fsub_rn(s1, s2), v);
  const float low = t1 + t2 + lo;
  const float h = __fadd_rn(s2, low), l = __fadd_rn(__fsub_rn(s2, h), low);
  const float m = __fmul_rn(h, f);
  return __fadd_rn(m, __fmaf_rn(h, f, -m) + l * f);
}

// The fp32 numbers nearest to f cos(2 pi t / 2^64) and f sin(2 pi t / 2^64).  The nearest table angle leaves b, at most
// pi / 256 = 2^-6.3, in fp32 pairs; with v = 1 - cos b (2^-13.7 at most)
//     cos(a + b) = C - S sin b - C v,   sin(a + b) = S + C sin b - S v,
// products and sums of the leading parts with their rounding errors, the rest in plain fp32.
__device__ __forceinline__ void cos_sin_exact(unsigned long long t, float f, float& c, float& s) {
  const unsigned long long k = (t + (1ull << 55)) >> 56;
  const long long r = static_cast<long long>(t - (k << 56));  // in [-2^55, 2^55)
  const uint4 raw = __ldg(reinterpret_cast<const uint4*>(&kTable.e[k & (kAngles - 1)]));
  const float ch = __uint_as_float(raw.x), cl = __uint_as_float(raw.y);
  const float sh = __uint_as_float(raw.z), sl = __uint_as_float(raw.w);
  // b = r 2 pi / 2^64, r's magnitude in pieces that fp32 holds (24, 16 and 16 bits): h + l = |r| / 2^16
  constexpr double kUnit = 6.283185307179586477 / 281474976710656.0;
  constexpr float kUnitH = static_cast<float>(kUnit), kUnitL = static_cast<float>(kUnit - static_cast<double>(kUnitH));
  const unsigned long long m = static_cast<unsigned long long>(r < 0 ? -r : r);
  const float m2 = static_cast<float>(static_cast<uint32_t>(m >> 32)), m1 = static_cast<float>(static_cast<uint32_t>(m) >> 16);
  const float m0 = static_cast<float>(static_cast<uint32_t>(m) & 0xFFFFu);
  const float h = __fmaf_rn(m2, 65536.0f, m1);
  const float l = __fadd_rn(__fmaf_rn(m2, 65536.0f, -h), m1) + m0 * 1.52587890625e-5f;
  const float unit = r < 0 ? -kUnitH : kUnitH, unit_l = r < 0 ? -kUnitL : kUnitL;
  const float bh = __fmul_rn(h, unit);
  const float bl = __fmaf_rn(h, unit, -bh) + __fmaf_rn(h, unit_l, l * unit);
  const float b2 = __fmul_rn(bh, bh), b2l = __fmaf_rn(bh, bh, -b2);
  // sin b = bh + sbl, 1 - cos b = vh + vl
  const float sbl = bl - bh * b2 * (0.16666667f - b2 * 0.0083333333f);
  const float vh = 0.5f * b2;
  const float vl = 0.5f * b2l + bh * bl - b2 * b2 * (0.041666667f - b2 * 0.0013888889f);
  // products of the leading parts, then their errors and the small parts
  const float sb = __fmul_rn(sh, bh), cb = __fmul_rn(ch, bh), cv = __fmul_rn(ch, vh), sv = __fmul_rn(sh, vh);
  const float c_lo = cl - (__fmaf_rn(sh, bh, -sb) + sh * sbl + sl * bh) - (__fmaf_rn(ch, vh, -cv) + ch * vl + cl * vh);
  const float s_lo = sl + (__fmaf_rn(ch, bh, -cb) + ch * sbl + cl * bh) - (__fmaf_rn(sh, vh, -sv) + sh * vl + sl * vh);
  c = join(ch, sb, cv, c_lo, f);
  s = join(sh, -cb, sv, s_lo, f);
}

constexpr int kTokens = 16;  // of a block
constexpr int kAppendThreads = 256;

// A lane's two words of a row, 8 values each; the pair of its frequency i.
template <bool INTER>
__device__ __forceinline__ void rotate_words(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + 8;
    const float a = x[ia], b = x[ib];
    x[ia] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
    x[ib] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
  }
}

__device__ __forceinline__ void unpack_words(const uint4& w0, const uint4& w1, float (&x)[16]) {
  float lo[8], hi[8];
  unpack<8>(w0, lo);
  unpack<8>(w1, hi);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = lo[i];
    x[8 + i] = hi[i];
  }
}

}  // namespace

// Blocks y < q_blocks: query heads q_heads_per_block * y ..; the others: KV head y - q_blocks.  D / 16 lanes hold a row.
template <int D, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) rope_append_kernel(const __grid_constant__ RopeAppendArgs a) {
  constexpr int LANES = D / 16, ROWS = kAppendThreads / LANES;  // rows the block holds at a time: 16 or 32
  __shared__ __align__(16) int8_t vs[kTokens][D];
  __shared__ long long tok_ph[kTokens];  // page * n_kv_heads + head, -1: not written
  __shared__ int tok_slot[kTokens], tok_seq[kTokens], tok_at[kTokens];
  const int row = threadIdx.x / LANES, col = threadIdx.x % LANES;
  const int k = row % kTokens;  // token of the block
  const bool is_q = static_cast<int>(blockIdx.y) < a.q_blocks;
  grid_dep_wait();
  grid_dep_trigger();
  // tokens from a page boundary on (one token more than a whole number of blocks is no reason to shift)
  int shift = 0;
  if (a.n_tokens > kTokens) shift = a.slot[0] & (KVQ_BLOCK_SIZE - 1);
  const long long tok = static_cast<long long>(blockIdx.x) * kTokens - shift + k;
  const bool live = tok >= 0 && tok < a.n_tokens;
  int slot = -1, seq = 0;
  if (live) {
    slot = a.slot[tok];
    if (!is_q) seq = a.seq_idx[tok];
  }
  const bool take = live && slot != -1;  // -1: a padding token
  const int half = a.rotary_dim / 2, n_rot = half / 8;
  int e0, e1;
  const bool rotated = col < n_rot;
  if (rotated) {
    e0 = a.rotary_offset + (INTER ? 16 * col : 8 * col);
    e1 = INTER ? e0 + 8 : e0 + half;
  } else {
    const int u = 16 * (col - n_rot);
    e0 = u < a.rotary_offset ? u : u + a.rotary_dim;
    e1 = u + 8 < a.rotary_offset ? u + 8 : u + 8 + a.rotary_dim;
  }
  const bool is_v = !is_q && ROWS > kTokens && row >= kTokens;  // head_dim 128: K rows and V rows side by side
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  if (rotated && take && !is_v) {
    int32_t p[kMaxAxes];
    load_axes(a.axes, tok, p);
    const uint32_t map = a.axes.map[col / 2] >> (16 * (col % 2));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      cos_sin_exact(position_bits(axis_position(p, map, i)) * __ldg(a.phases + col * 8 + i), a.attn_factor, c[i], s[i]);
  }

  if (is_q) {
    if (!take) return;
    constexpr int STEP = ROWS / kTokens, IN_FLIGHT = 4;
    const int h0 = static_cast<int>(blockIdx.y) * a.q_heads_per_block, h1 = min(a.n_q_heads, h0 + a.q_heads_per_block);
    const uint16_t* src = a.q + tok * a.q_stride;
    uint16_t* dst = a.q_out + tok * a.q_out_stride;
    for (int h = h0 + row / kTokens; h < h1; h += STEP * IN_FLIGHT) {
      uint4 w0[IN_FLIGHT], w1[IN_FLIGHT];
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u)
        if (h + u * STEP < h1) {
          w0[u] = *reinterpret_cast<const uint4*>(src + static_cast<long long>(h + u * STEP) * D + e0);
          w1[u] = *reinterpret_cast<const uint4*>(src + static_cast<long long>(h + u * STEP) * D + e1);
        }
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u)
        if (h + u * STEP < h1) {
          if (rotated) {
            float x[16], lo[8], hi[8];
            unpack_words(w0[u], w1[u], x);
            rotate_words<INTER>(x, c, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              lo[i] = x[i];
              hi[i] = x[8 + i];
            }
            w0[u] = pack<8>(lo);
            w1[u] = pack<8>(hi);
          }
          *reinterpret_cast<uint4*>(dst + static_cast<long long>(h + u * STEP) * D + e0) = w0[u];
          *reinterpret_cast<uint4*>(dst + static_cast<long long>(h + u * STEP) * D + e1) = w1[u];
        }
    }
    return;
  }

  // ---- one KV head
  const int kvh = static_cast<int>(blockIdx.y) - a.q_blocks, H = a.n_kv_heads;
  long long ph = -1;
  if (take) {
    unsigned bad = 0;
    if (seq < 0 || seq >= a.num_seqs) {
      bad = KVQ_DEV_BAD_SEQ;
    } else if (slot < 0 || slot / KVQ_BLOCK_SIZE >= a.max_blocks_per_seq) {
      bad = KVQ_DEV_BAD_POS;
    } else {
      const int page = a.block_table[static_cast<long long>(seq) * a.max_blocks_per_seq + slot / KVQ_BLOCK_SIZE];
      if (page < 0 || page >= a.num_blocks) bad = KVQ_DEV_BAD_BLOCK;
      else ph = static_cast<long long>(page) * H + kvh;
    }
    if (bad && col == 0) set_status(a.status, bad);
  }
  const int at = slot & (KVQ_BLOCK_SIZE - 1);
  if (col == 0 && row < kTokens) {
    tok_ph[k] = ph;
    tok_at[k] = at;
    tok_slot[k] = slot;
    tok_seq[k] = seq;
  }
  const long long src = tok, head = static_cast<long long>(kvh) * D;
  auto load = [&](const uint16_t* rows, long long stride, float (&x)[16]) {
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (ph >= 0) {
      w0 = *reinterpret_cast<const uint4*>(rows + src * stride + head + e0);
      w1 = *reinterpret_cast<const uint4*>(rows + src * stride + head + e1);
    }
    unpack_words(w0, w1, x);
  };
  // every lane of a warp takes part in the rows' maxima
  if (!is_v) {
    float x[16];
    load(a.k_new, a.k_stride, x);
    if (rotated) rotate_words<INTER>(x, c, s);
    uint32_t code[4];
    const float scale = quant_rule_rows_packed<16, LANES>(x, code);
    if (ph >= 0) {
      int8_t* page = a.k + ph * (D * KVQ_BLOCK_SIZE);
      *reinterpret_cast<uint2*>(page + ((e0 / 16) * KVQ_BLOCK_SIZE + at) * 16 + e0 % 16) = make_uint2(code[0], code[1]);
      *reinterpret_cast<uint2*>(page + ((e1 / 16) * KVQ_BLOCK_SIZE + at) * 16 + e1 % 16) = make_uint2(code[2], code[3]);
      if (col == 0) a.k_scale[ph * KVQ_BLOCK_SIZE + at] = scale;
    }
  }
  if (is_v || ROWS == kTokens) {
    float x[16];
    load(a.v_new, a.v_stride, x);
    uint32_t code[4];
    const float scale = quant_rule_rows_packed<16, LANES>(x, code);
    *reinterpret_cast<uint2*>(&vs[k][e0]) = make_uint2(code[0], code[1]);
    *reinterpret_cast<uint2*>(&vs[k][e1]) = make_uint2(code[2], code[3]);
    if (ph >= 0 && col == 0) a.v_scale[ph * KVQ_BLOCK_SIZE + at] = scale;
  }
  __syncthreads();
  // The V codes: where the block's tokens fill a page in order, 16 bytes a dimension; else a byte each.
  bool full = true;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) full = full && tok_ph[i] == tok_ph[0] && tok_at[i] == i;
  full = full && tok_ph[0] >= 0;
  if (full) {
    for (int d = threadIdx.x; d < D; d += kAppendThreads) {
      uint32_t w[4];
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4)
        w[q4] = static_cast<uint32_t>(static_cast<uint8_t>(vs[4 * q4][d])) |
                (static_cast<uint32_t>(static_cast<uint8_t>(vs[4 * q4 + 1][d])) << 8) |
                (static_cast<uint32_t>(static_cast<uint8_t>(vs[4 * q4 + 2][d])) << 16) |
                (static_cast<uint32_t>(static_cast<uint8_t>(vs[4 * q4 + 3][d])) << 24);
      *reinterpret_cast<uint4*>(a.v + (tok_ph[0] * D + d) * KVQ_BLOCK_SIZE) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    for (int it = threadIdx.x; it < kTokens * D; it += kAppendThreads) {
      const int i = it / D, d = it % D;
      if (tok_ph[i] >= 0) a.v[(tok_ph[i] * D + d) * KVQ_BLOCK_SIZE + tok_at[i]] = vs[i][d];
    }
  }
}

template <int D>
static cudaError_t launch_append_d(RopeAppendArgs a, int n_sms, cudaStream_t stream) {
  const long long groups = a.n_tokens > kTokens ? (static_cast<long long>(a.n_tokens) + KVQ_BLOCK_SIZE - 1 + kTokens - 1) / kTokens : 1;
  int per = 16;
  while (per > 256 / D && groups * ((a.n_q_heads + per - 1) / per + a.n_kv_heads) < 4LL * n_sms) per /= 2;
  a.q_heads_per_block = per;
  a.q_blocks = (a.n_q_heads + per - 1) / per;
  if (groups > 0x7fffffffLL || a.q_blocks + a.n_kv_heads > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(groups), a.q_blocks + a.n_kv_heads);
  return a.interleaved ? launch_pdl(rope_append_kernel<D, true>, grid, dim3(kAppendThreads), 0, stream, a)
                       : launch_pdl(rope_append_kernel<D, false>, grid, dim3(kAppendThreads), 0, stream, a);
}

cudaError_t launch_rope_append(const RopeAppendArgs& a, int n_sms, cudaStream_t stream) {
  return a.head_dim == 256 ? launch_append_d<256>(a, n_sms, stream) : launch_append_d<128>(a, n_sms, stream);
}

}  // namespace kvq
