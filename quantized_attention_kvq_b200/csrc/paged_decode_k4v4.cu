// Paged split decode, INT4 keys and INT4 values.
#include "paged_decode.cuh"

namespace kvq {
namespace paged {

cudaError_t launch_44(const PagedDecodeArgs& a, cudaStream_t s) { return launch_bits<4, 4>(a, s); }
KVQ_BOUNDS_COUNTER(bounds_44)

}  // namespace paged
}  // namespace kvq
