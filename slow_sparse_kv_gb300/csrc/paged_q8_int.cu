// Attention over an 8-bit paged cache, int8 codes, and the choice between the two formats.
#include "paged_q8_impl.cuh"

namespace sfi {

template cudaError_t launch_q8_of<false>(const PagedAttnArgs&, int, bool, bool, int, cudaStream_t);
extern template cudaError_t launch_q8_of<true>(const PagedAttnArgs&, int, bool, bool, int, cudaStream_t);

cudaError_t launch_paged_attn_q8(const PagedAttnArgs& a, int D, bool e4m3, bool q_f32, bool use_tma, int grid,
                                 cudaStream_t st) {
  return e4m3 ? launch_q8_of<true>(a, D, q_f32, use_tma, grid, st) : launch_q8_of<false>(a, D, q_f32, use_tma, grid, st);
}

}  // namespace sfi
