// Attention over an 8-bit paged cache, e4m3 codes.
#include "paged_q8_impl.cuh"

namespace sfi {

template cudaError_t launch_q8_of<true>(const PagedAttnArgs&, int, bool, bool, int, cudaStream_t);

}  // namespace sfi
