// rope_dev.cuh — device helpers of the kernels that rotate bf16 rows by position (rope.cu, rope_append.cu): bf16 words,
// and the position that a frequency takes.
#pragma once

#include <cuda_bf16.h>

#include "kvq_dev.cuh"
#include "kvq_launch.h"

namespace kvq {

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

// A position as the factor of a phase: modulo 2^64, negative ones too.
__device__ __forceinline__ unsigned long long position_bits(int32_t p) {
  return static_cast<unsigned long long>(static_cast<long long>(p));
}

// The positions of token tok on every axis (0 on the axes that the call does not have).
__device__ __forceinline__ void load_axes(const RopeAxes& ax, long long tok, int32_t (&p)[kMaxAxes]) {
#pragma unroll
  for (int i = 0; i < kMaxAxes; ++i) p[i] = i < ax.n ? ax.pos[i * ax.pos_stride + tok] : 0;
}

// The position of the frequency whose axis is the i-th pair of bits of map.
__device__ __forceinline__ int32_t axis_position(const int32_t (&p)[kMaxAxes], uint32_t map, int i) {
  const uint32_t lo = map >> (2 * i) & 1u, hi = map >> (2 * i + 1) & 1u;
  return hi ? (lo ? p[3] : p[2]) : (lo ? p[1] : p[0]);
}

}  // namespace kvq
