// Paged split decode, INT4 keys and INT2 values.
#include "paged_decode.cuh"

namespace kvq {
namespace paged {

cudaError_t launch_42(const PagedDecodeArgs& a, cudaStream_t s) { return launch_bits<4, 2>(a, s); }
KVQ_BOUNDS_COUNTER(bounds_42)

}  // namespace paged
}  // namespace kvq
