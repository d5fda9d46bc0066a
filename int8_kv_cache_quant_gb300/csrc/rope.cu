// rope.cu — rotary positions on bf16 query and key rows, by positions that need not be cache slots.
//
// "gfx936 DCU上实现INT8 KV与INT8 MMAC Attention推理优化" §2.2 rotates Q and K inside the quantising
// producer, by the slot's position and a cos / sin table; kvq_rope_quant_write is that producer.
// The decode step and the first prefill chunk take K and Q rows that are already rotated, and a
// cache that evicts tokens holds a token at a slot that is not its position.  This kernel is the
// rotation on its own: for the pair (x, y) of frequency j at position p
//     x' = x c - y s,   y' = y c + x s,   c = factor cos(2 pi turns), s = factor sin(2 pi turns),
//     turns = frac(p * phase[j] / 2^64).
// The phase is the frequency in turns per position as a 64-bit fraction, so p * phase mod 2^64 is
// exact whatever p is, and there is no table whose rows would have to be read (1 KB a token at
// rotary_dim 256) or sized by a largest position.  What a far position multiplies is the plan's own
// rounding: the phases are made in double precision, which leaves an angle of at most 1.1e-6 rad at
// position 2^31 (3.2e-7 measured over bases 500 .. 1e7), against bf16's 2^-9.
//
// Bound: bytes, each row once in and once out.  A thread owns one column of a token (kVec pairs, two
// 16-byte words of a row; the dims that are not rotated are columns without arithmetic), computes its
// cos and sin once and applies them to several heads, with the loads of four heads in flight.
// 2048 tokens x (24 + 4) heads of 256, 64 dims rotated (29 MB in, 29 MB out): 11.9 us, 4.9 TB/s, most of the outputs staying in L2; one
// token 1.8 us, a launch.
#include <cuda_bf16.h>

#include "kvq_dev.cuh"
#include "kvq_launch.h"

namespace kvq {

namespace {

// cos and sin of 2 pi t / 2^32.  The nearest quarter turn n leaves an angle of at most pi / 4 in
// magnitude (an exact integer r of 2^-32 turns, rounded once to fp32), where the Taylor
// polynomials of degree 9 and 8 are within 1.8e-9 and 2.5e-8 of sin and cos (the first terms left
// out, (pi/4)^11 / 11! and (pi/4)^10 / 10!): below half an fp32 step.
__device__ __forceinline__ void cos_sin_turns(int32_t t, float& c, float& s) {
  const uint32_t q = (static_cast<uint32_t>(t) + 0x20000000u) >> 30;
  const int32_t r = static_cast<int32_t>(static_cast<uint32_t>(t) - (q << 30));
  const float x = static_cast<float>(r) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float x2 = x * x;
  float sp = fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);
  sp = fmaf(sp, x2, 8.33333333e-3f);
  sp = fmaf(sp, x2, -1.66666667e-1f);
  sp = fmaf(sp * x2, x, x);
  float cp = fmaf(x2, 2.48015873e-5f, -1.38888889e-3f);
  cp = fmaf(cp, x2, 4.16666667e-2f);
  cp = fmaf(cp, x2, -0.5f);
  cp = fmaf(cp, x2, 1.0f);
  // q quarter turns more
  c = (q & 1u) ? sp : cp;
  s = (q & 1u) ? cp : sp;
  if (q == 1u || q == 2u) c = -c;
  if (q & 2u) s = -s;
}

template <int V>
struct Word;  // V bf16 values as one load or store
template <>
struct Word<8> { using T = uint4; };
template <>
struct Word<4> { using T = uint2; };
template <>
struct Word<2> { using T = uint32_t; };
template <>
struct Word<1> { using T = uint16_t; };

template <int V>
__device__ __forceinline__ void unpack(const typename Word<V>::T& w, float (&x)[V]) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(&w);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = bf16_bits_to_float(h[i]);
}

template <int V>
__device__ __forceinline__ typename Word<V>::T pack(const float (&x)[V]) {
  typename Word<V>::T w;
  uint16_t* h = reinterpret_cast<uint16_t*>(&w);
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x[i]));
  return w;
}

constexpr int kRopeThreads = 128;
constexpr int kInFlight = 4;  // heads whose loads a thread issues before it works on the first

}  // namespace

// Thread (token, head group hg, column): heads hg, hg + head_groups, ... of the token.
// INTER: the pair of frequency j is dims (2j, 2j + 1) of the rotated part; else (j, j + r/2).
template <int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  using W = typename Word<V>::T;
  const long long idx = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  grid_dep_wait();
  grid_dep_trigger();
  const long long tg = idx / a.columns;
  const int col = static_cast<int>(idx - tg * a.columns);
  const long long tok = tg / a.head_groups;
  if (tok >= a.n_tokens) return;
  const int hg = static_cast<int>(tg - tok * a.head_groups);
  const int half = a.rotary_dim / 2, n_rot = half / V;
  // the column's two words: element offsets in the row
  int e0, e1;
  const bool rotated = col < n_rot;
  if (rotated) {
    e0 = a.rotary_offset + (INTER ? 2 * col : col) * V;
    e1 = INTER ? e0 + V : e0 + half;
  } else {  // dims outside the rotated part, two words at a time (the last column may have one)
    const int rest = (a.head_dim - a.rotary_dim) / V, u = 2 * (col - n_rot);
    auto place = [&](int w) { return w * V < a.rotary_offset ? w * V : w * V + a.rotary_dim; };
    e0 = place(u);
    e1 = u + 1 < rest ? place(u + 1) : -1;
  }
  float c[V], s[V];
  if (rotated) {
    const unsigned long long p = static_cast<unsigned long long>(static_cast<long long>(a.pos[tok]));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const unsigned long long ph = p * __ldg(a.phases + col * V + i);
      cos_sin_turns(static_cast<int32_t>((ph + 0x80000000ull) >> 32), c[i], s[i]);
      c[i] *= a.attn_factor;
      s[i] *= a.attn_factor;
    }
  }
  const int H = a.n_q_heads + a.n_kv_heads;
  for (int h0 = hg; h0 < H; h0 += kInFlight * a.head_groups) {
    W w0[kInFlight], w1[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int h = h0 + u * a.head_groups;
      if (h < H) {
        const uint16_t* row = h < a.n_q_heads ? a.q + tok * a.q_stride + h * a.head_dim
                                              : a.k + tok * a.k_stride + (h - a.n_q_heads) * a.head_dim;
        w0[u] = *reinterpret_cast<const W*>(row + e0);
        if (e1 >= 0) w1[u] = *reinterpret_cast<const W*>(row + e1);
      }
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int h = h0 + u * a.head_groups;
      if (h < H) {
        uint16_t* dst = h < a.n_q_heads ? a.q_out + tok * a.q_out_stride + h * a.head_dim
                                        : a.k_out + tok * a.k_out_stride + (h - a.n_q_heads) * a.head_dim;
        if (rotated) {
          float x[V], y[V];
          unpack<V>(w0[u], x);
          unpack<V>(w1[u], y);
          if constexpr (INTER) {
            // words hold the pairs side by side: element 2i, 2i + 1 of the 2V values
            float z[2 * V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
              z[i] = x[i];
              z[V + i] = y[i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float xa = z[2 * i], xb = z[2 * i + 1];
              z[2 * i] = fmaf(xa, c[i], -(xb * s[i]));
              z[2 * i + 1] = fmaf(xb, c[i], xa * s[i]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
              x[i] = z[i];
              y[i] = z[V + i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float xa = x[i], xb = y[i];
              x[i] = fmaf(xa, c[i], -(xb * s[i]));
              y[i] = fmaf(xb, c[i], xa * s[i]);
            }
          }
          w0[u] = pack<V>(x);
          w1[u] = pack<V>(y);
        }
        *reinterpret_cast<W*>(dst + e0) = w0[u];
        if (e1 >= 0) *reinterpret_cast<W*>(dst + e1) = w1[u];
      }
    }
  }
}

template <int V>
static cudaError_t launch_rope_v(RopeArgs a, int n_sms, cudaStream_t stream) {
  const int H = a.n_q_heads + a.n_kv_heads;
  const int rest = (a.head_dim - a.rotary_dim) / V;
  a.columns = a.rotary_dim / (2 * V) + (rest + 1) / 2;
  // Heads per thread: as many (up to 8) as leave a thousand threads for every SM.  More of them share
  // one evaluation of cos and sin; fewer spread a short call over the GPU.  Always
  // one | always 8, us: one token 1.9 | 3.0, 64 x (32 + 8) heads of 128 2.1 | 3.4, 2048 x (24 + 4) of 256 19.0 |
  // 12.3; at most 2 or 16: 13.5 and 12.0 for the last.
  int per = 8;
  while (per > 1 && static_cast<long long>(a.n_tokens) * ((H + per - 1) / per) * a.columns < 1024LL * n_sms) per /= 2;
  a.head_groups = (H + per - 1) / per;
  const long long threads = static_cast<long long>(a.n_tokens) * a.head_groups * a.columns;
  const long long blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks));
  return a.interleaved ? launch_pdl(rope_kernel<V, true>, grid, dim3(kRopeThreads), 0, stream, a)
                       : launch_pdl(rope_kernel<V, false>, grid, dim3(kRopeThreads), 0, stream, a);
}

cudaError_t launch_rope(const RopeArgs& a, int n_sms, cudaStream_t stream) {
  // the widest word that every row, the rotated part and both its halves are whole numbers of
  long long bits = a.rotary_dim / 2 | a.rotary_offset | a.head_dim | 8;
  if (a.n_q_heads) bits |= a.q_stride | a.q_out_stride | static_cast<long long>(reinterpret_cast<uintptr_t>(a.q) / 2) |
                           static_cast<long long>(reinterpret_cast<uintptr_t>(a.q_out) / 2);
  if (a.n_kv_heads) bits |= a.k_stride | a.k_out_stride | static_cast<long long>(reinterpret_cast<uintptr_t>(a.k) / 2) |
                            static_cast<long long>(reinterpret_cast<uintptr_t>(a.k_out) / 2);
  switch (bits & -bits) {
    case 8: return launch_rope_v<8>(a, n_sms, stream);
    case 4: return launch_rope_v<4>(a, n_sms, stream);
    case 2: return launch_rope_v<2>(a, n_sms, stream);
    default: return launch_rope_v<1>(a, n_sms, stream);
  }
}

}  // namespace kvq
