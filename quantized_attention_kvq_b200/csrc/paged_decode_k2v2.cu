// Paged split decode, INT2 keys and INT2 values.
#include "paged_decode.cuh"

namespace kvq {
namespace paged {

cudaError_t launch_22(const PagedDecodeArgs& a, cudaStream_t s) { return launch_bits<2, 2>(a, s); }
KVQ_BOUNDS_COUNTER(bounds_22)

}  // namespace paged
}  // namespace kvq
