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
// in pairs of fp32 and a short polynomial of what is left, about 100 instructions a pair, within 2^-45 of the value, which
// leaves one cos in some 2^19 rounded the other way (and a code only where its quotient lies at a tie as well).
//
// Bound: bytes, each row in once, q out once, half a byte out for each byte of k and v in; a token's cos and sin cost as many
// instructions as the rotation of eight heads.  So a block takes 16 tokens and as many heads as leave the GPU full: it makes
// the cos and sin once, into shared memory, its first query rows on their way meanwhile, and then a thread owns one column
// of a token (8 pairs, two 16-byte words of a row) for all its heads.  With 8 pairs of cos and sin in each thread's own registers,
// again for every two heads of a token, 2048 tokens of 24 + 4 + 4 heads of 256 took 18.0 us; so 13.8 us (63 MB: 4.6 TB/s), of
// which 7 us are instructions to issue (7.7 M warp instructions; 11.5 M before).  Two blocks an SM leave a thread 64 registers, 36
// bytes of which are spilled beside the three rows on their way.  One token: 4.3 us in a captured graph.
// The 16 tokens are counted from a page boundary where the first token's slot says where one is, so that a chunk's V codes
// leave a page at a time, 16 bytes a dimension.
#include <algorithm>

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
constexpr int kAppendThreads = 512;

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

// Block y: query heads q_heads y .. and, from y = kv_first on, KV heads kv_heads (y - kv_first) ..  First the cos and sin of
// its tokens, into shared memory; then D / 16 lanes a row, RS rows of each token at a time.
template <int D, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, 2) rope_append_kernel(const __grid_constant__ RopeAppendArgs a) {
  constexpr int LANES = D / 16, RS = kAppendThreads / (kTokens * LANES);  // 2 or 4
  __shared__ __align__(16) float cs_s[2][kTokens][D / 2 + 4];
  __shared__ __align__(16) int8_t vs[RS / 2][kTokens][D];
  __shared__ int tok_slot[kTokens], tok_page[kTokens];  // -1: a padding token or none; -1: nothing written to the cache
  __shared__ bool page_s;
  const int tid = threadIdx.x, rs = tid / (kTokens * LANES), k = tid / LANES % kTokens, col = tid % LANES;
  const int h0 = static_cast<int>(blockIdx.y) * a.q_heads, h1 = min(a.n_q_heads, h0 + a.q_heads);
  const int kv0 = (static_cast<int>(blockIdx.y) - a.kv_first) * a.kv_heads;
  const int n_kv = kv0 < 0 ? 0 : min(a.n_kv_heads - kv0, a.kv_heads);  // (0 or less: none)
  grid_dep_wait();
  grid_dep_trigger();
  // more than one block: tokens from a page boundary on, as the first token's slot has it
  int shift = 0;
  if (a.n_tokens > kTokens) shift = a.slot[0] & (KVQ_BLOCK_SIZE - 1);
  const long long base = static_cast<long long>(blockIdx.x) * kTokens - shift;
  const int lo = base < 0 ? static_cast<int>(-base) : 0, hi = static_cast<int>(min(static_cast<long long>(kTokens), a.n_tokens - base));
  if (tid < 32) {
    int slot = -1, seq = 0, page = -1;
    if (tid >= lo && tid < hi) {
      slot = a.slot[base + tid];
      seq = a.seq_idx[base + tid];
    }
    if (slot != -1 && n_kv > 0) {
      unsigned bad = 0;
      if (seq < 0 || seq >= a.num_seqs) {
        bad = KVQ_DEV_BAD_SEQ;
      } else if (slot < 0 || slot / KVQ_BLOCK_SIZE >= a.max_blocks_per_seq) {
        bad = KVQ_DEV_BAD_POS;
      } else {
        page = a.block_table[static_cast<long long>(seq) * a.max_blocks_per_seq + slot / KVQ_BLOCK_SIZE];
        if (page < 0 || page >= a.num_blocks) {
          bad = KVQ_DEV_BAD_BLOCK;
          page = -1;
        }
      }
      if (bad) set_status(a.status, bad);
    }
    // whether the tokens fill a page in order: their V codes leave 16 bytes a dimension then
    const int page0 = __shfl_sync(0xffffffffu, page, 0);
    const bool fill = __all_sync(0xffffffffu, tid >= kTokens || (page >= 0 && page == page0 && slot % KVQ_BLOCK_SIZE == tid));
    if (tid < kTokens) {
      tok_slot[tid] = slot;
      tok_page[tid] = page;
      if (tid == 0) page_s = fill;
    }
  }
  const int half = a.rotary_dim / 2, n_live = hi - lo, n_rot = half / 8;
  const bool rotated = col < n_rot;
  int e0, e1;
  if (rotated) {
    e0 = a.rotary_offset + (INTER ? 16 * col : 8 * col);
    e1 = INTER ? e0 + 8 : e0 + half;
  } else {
    const int u = 16 * (col - n_rot);
    e0 = u < a.rotary_offset ? u : u + a.rotary_dim;
    e1 = u + 8 < a.rotary_offset ? u + 8 : u + 8 + a.rotary_dim;
  }
  // the first query rows are on their way meanwhile
  constexpr int IN_FLIGHT = 3;
  const long long tok = base + k;
  const uint16_t* q_src = a.q + tok * a.q_stride;
  uint4 w0[IN_FLIGHT], w1[IN_FLIGHT];
  auto fetch = [&](int h) {
#pragma unroll
    for (int u = 0; u < IN_FLIGHT; ++u)
      if (h + u * RS < h1 && k >= lo && k < hi) {
        w0[u] = *reinterpret_cast<const uint4*>(q_src + static_cast<long long>(h + u * RS) * D + e0);
        w1[u] = *reinterpret_cast<const uint4*>(q_src + static_cast<long long>(h + u * RS) * D + e1);
      }
  };
  fetch(h0 + rs);
  for (int i = tid; i < n_live * half; i += kAppendThreads) {
    const int pair = i / n_live, t = lo + (i - pair * n_live), axis = a.axes.map[pair / 16] >> (2 * (pair % 16)) & 3;
    const int32_t p = a.axes.pos[axis * a.axes.pos_stride + base + t];
    float c, s;
    cos_sin_exact(position_bits(p) * __ldg(a.phases + pair), a.attn_factor, c, s);
    cs_s[0][t][pair] = c;
    cs_s[1][t][pair] = s;
  }
  __syncthreads();

  float c[8], s[8];
  if (rotated) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c4 = *reinterpret_cast<const float4*>(&cs_s[0][k][8 * col + 4 * i]);
      const float4 s4 = *reinterpret_cast<const float4*>(&cs_s[1][k][8 * col + 4 * i]);
      c[4 * i] = c4.x, c[4 * i + 1] = c4.y, c[4 * i + 2] = c4.z, c[4 * i + 3] = c4.w;
      s[4 * i] = s4.x, s[4 * i + 1] = s4.y, s[4 * i + 2] = s4.z, s[4 * i + 3] = s4.w;
    }
  }
  const int slot = tok_slot[k], page = tok_page[k], at = slot & (KVQ_BLOCK_SIZE - 1);

  if (slot != -1) {
    uint16_t* dst = a.q_out + tok * a.q_out_stride;
    for (int h = h0 + rs; h < h1; h += RS * IN_FLIGHT) {
      if (h != h0 + rs) fetch(h);
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u)
        if (h + u * RS < h1) {
          if (rotated) {
            float x[16], low[8], high[8];
            unpack_words(w0[u], w1[u], x);
            rotate_words<INTER>(x, c, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              low[i] = x[i];
              high[i] = x[8 + i];
            }
            w0[u] = pack<8>(low);
            w1[u] = pack<8>(high);
          }
          *reinterpret_cast<uint4*>(dst + static_cast<long long>(h + u * RS) * D + e0) = w0[u];
          *reinterpret_cast<uint4*>(dst + static_cast<long long>(h + u * RS) * D + e1) = w1[u];
        }
    }
  }

  // ---- KV heads, RS / 2 at a time: K rows and V rows side by side
  const bool is_v = rs & 1, fill = page_s;
  for (int i0 = 0; i0 < n_kv; i0 += RS / 2) {
    const bool real = page >= 0 && i0 + rs / 2 < n_kv;
    const int kvh = kv0 + i0 + rs / 2;
    const long long ph = static_cast<long long>(page) * a.n_kv_heads + kvh;
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (real) {
      const uint16_t* src = (is_v ? a.v_new + tok * a.v_stride : a.k_new + tok * a.k_stride) + static_cast<long long>(kvh) * D;
      w0 = *reinterpret_cast<const uint4*>(src + e0);
      w1 = *reinterpret_cast<const uint4*>(src + e1);
    }
    float x[16];
    unpack_words(w0, w1, x);
    if (!is_v && rotated) rotate_words<INTER>(x, c, s);
    uint32_t code[4];
    const float scale = quant_rule_rows_packed<16, LANES>(x, code);  // every lane of a warp takes part in the rows' maxima
    if (is_v) {
      *reinterpret_cast<uint2*>(&vs[rs / 2][k][e0]) = make_uint2(code[0], code[1]);
      *reinterpret_cast<uint2*>(&vs[rs / 2][k][e1]) = make_uint2(code[2], code[3]);
    } else if (real) {
      int8_t* dst = a.k + ph * (D * KVQ_BLOCK_SIZE);
      *reinterpret_cast<uint2*>(dst + ((e0 / 16) * KVQ_BLOCK_SIZE + at) * 16 + e0 % 16) = make_uint2(code[0], code[1]);
      *reinterpret_cast<uint2*>(dst + ((e1 / 16) * KVQ_BLOCK_SIZE + at) * 16 + e1 % 16) = make_uint2(code[2], code[3]);
    }
    if (real && col == 0) (is_v ? a.v_scale : a.k_scale)[ph * KVQ_BLOCK_SIZE + at] = scale;
    __syncthreads();
    // The V codes
    if (fill) {
      const int b = tid / D, d = tid % D, h = i0 + b;  // (RS / 2 heads of D dimensions: 256 threads)
      if (b < RS / 2 && h < n_kv) {
        uint32_t w[4];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4)
          w[q4] = static_cast<uint32_t>(static_cast<uint8_t>(vs[b][4 * q4][d])) |
                  (static_cast<uint32_t>(static_cast<uint8_t>(vs[b][4 * q4 + 1][d])) << 8) |
                  (static_cast<uint32_t>(static_cast<uint8_t>(vs[b][4 * q4 + 2][d])) << 16) |
                  (static_cast<uint32_t>(static_cast<uint8_t>(vs[b][4 * q4 + 3][d])) << 24);
        *reinterpret_cast<uint4*>(a.v + ((static_cast<long long>(tok_page[0]) * a.n_kv_heads + kv0 + h) * D + d) * KVQ_BLOCK_SIZE) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      for (int it = tid; it < RS / 2 * kTokens * D; it += kAppendThreads) {
        const int d = it % D, t = it / D % kTokens, b = it / (D * kTokens);
        if (tok_page[t] >= 0 && i0 + b < n_kv)
          a.v[((static_cast<long long>(tok_page[t]) * a.n_kv_heads + kv0 + i0 + b) * D + d) * KVQ_BLOCK_SIZE +
              (tok_slot[t] & (KVQ_BLOCK_SIZE - 1))] = vs[b][t][d];
      }
    }
    __syncthreads();
  }
}

// Heads of a block: all of them share its cos and sin, so as many as leave one and a half blocks an SM, and from half a
// block an SM on a KV head and its query heads at least.  Where there are fewer tokens, query heads and KV heads in blocks of their own.
// So | always together | apart up to three blocks an SM, us: 64 sequences' tokens, 8 KV heads of 128 5.2 | 5.6 | 5.2; 64 tokens of
// one sequence, 4 heads of 256 5.3 | 6.3 | 5.3; 200 sequences 6.3 | 6.3 | 7.2; 512 tokens of one 6.5 | 6.5 | 10.1.
template <int D>
static cudaError_t launch_append_d(RopeAppendArgs a, int n_sms, cudaStream_t stream) {
  constexpr int RS = kAppendThreads / D;
  const long long groups = a.n_tokens > kTokens ? (static_cast<long long>(a.n_tokens) + KVQ_BLOCK_SIZE - 1 + kTokens - 1) / kTokens : 1;
  const int H = a.n_kv_heads, Hq = a.n_q_heads;
  long long blocks;
  if (2 * groups * H >= n_sms) {
    const int cut = static_cast<int>(std::min<long long>(H, (3LL * n_sms + 2 * groups - 1) / (2 * groups)));
    a.kv_heads = (H + cut - 1) / cut;
    blocks = (H + a.kv_heads - 1) / a.kv_heads;
    a.q_heads = static_cast<int>((Hq + blocks - 1) / blocks);
    a.kv_first = 0;
  } else {
    int per = 16;
    while (per > RS && groups * ((Hq + per - 1) / per + H) < 2LL * n_sms) per /= 2;
    a.q_heads = per;
    a.kv_heads = 1;
    a.kv_first = (Hq + per - 1) / per;
    blocks = static_cast<long long>(a.kv_first) + H;
  }
  if (groups > 0x7fffffffLL || blocks > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>(blocks));
  return a.interleaved ? launch_pdl(rope_append_kernel<D, true>, grid, dim3(kAppendThreads), 0, stream, a)
                       : launch_pdl(rope_append_kernel<D, false>, grid, dim3(kAppendThreads), 0, stream, a);
}

cudaError_t launch_rope_append(const RopeAppendArgs& a, int n_sms, cudaStream_t stream) {
  return a.head_dim == 256 ? launch_append_d<256>(a, n_sms, stream) : launch_append_d<128>(a, n_sms, stream);
}

}  // namespace kvq
