// Attention over a paged MXFP8 cache for up to 32 query heads of a cache head at a time.
#include "mxq_paged_attention.cuh"

namespace mxq {
namespace paged {
template cudaError_t launch_heads<32>(const CUtensorMap&, const CUtensorMap&, const Args&, cudaStream_t);
}  // namespace paged
}  // namespace mxq
