// decode_window.cu — the decode step over the int8 paged K/V cache with a sliding window and first tokens that stay
// visible: the row at position p sees the keys t <= p with t > p - window or t < n_sink.
//
// The kernels are those of decode.cu (stage 1 and the merge, described there), compiled with the window: the pages that
// no row of a sequence sees are left out of the walk, whether or not the block table still names them, so that the time
// goes by the window and not by the sequence, and a row's mask is two bounds a thread holds in registers.
//
// Bound: the bytes of the keys that are seen.  64 sequences of 512 .. 16384 keys, W = 4096, 32 / 8 heads of 128 (498 MB): 100 us,
// 5.0 TB/s; the step without a window over as many keys takes 2 % less (102.0 against 103.8 us at 4112 keys a sequence).
// One sequence, W = 1024, 24 / 4 heads of 256: 7.9 us in a captured graph, two dependent launches; four rows, W = 8191: 16.9 us.
#include "decode_merge.cuh"
#include "decode_stage1.cuh"

namespace kvq {

template <int D, bool SPLIT>
static cudaError_t launch_stage1_window(const DecodeArgs& a, dim3 grid, cudaStream_t stream) {
  const int group = a.n_q_heads / a.n_kv_heads;
  if (a.nq == 1 && group <= 8) {
    if (a.k_new) return launch_stage1<D, 1, SPLIT, false, true, false, true>(a, grid, stream);
    return launch_stage1<D, 1, SPLIT, false, false, false, true>(a, grid, stream);
  }
  switch ((group * a.nq + 7) / 8) {
    case 1: return launch_stage1<D, 1, SPLIT, true, true, false, true>(a, grid, stream);
    case 2: return launch_stage1<D, 2, SPLIT, true, true, false, true>(a, grid, stream);
    case 3: return launch_stage1<D, 3, SPLIT, true, true, false, true>(a, grid, stream);
    case 4: return launch_stage1<D, 4, SPLIT, true, true, false, true>(a, grid, stream);
    case 5: return launch_stage1<D, 5, SPLIT, true, true, false, true>(a, grid, stream);
    case 6: return launch_stage1<D, 6, SPLIT, true, true, false, true>(a, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <int D>
static cudaError_t launch_step_window_d(const DecodeArgs& a, DecodeRoute route, cudaStream_t stream) {
  if (route == DecodeRoute::kSingle) return launch_stage1_window<D, false>(a, dim3(1, a.n_kv_heads, a.batch), stream);
  cudaError_t e = prepare_merge<D, true>(a);
  if (e != cudaSuccess) return e;
  e = launch_stage1_window<D, true>(a, dim3(a.n_split, a.n_kv_heads, a.batch), stream);
  if (e != cudaSuccess) return e;
  return launch_decode_merge<D, true>(a, stream);
}

cudaError_t launch_step_window(const DecodeArgs& a, DecodeRoute route, cudaStream_t stream, int* launched) {
  *launched = route == DecodeRoute::kSingle ? 1 : 2;
  return a.head_dim == 256 ? launch_step_window_d<256>(a, route, stream) : launch_step_window_d<128>(a, route, stream);
}

}  // namespace kvq
