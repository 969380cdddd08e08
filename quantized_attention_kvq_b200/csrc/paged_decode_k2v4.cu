// Paged split decode, INT2 keys and INT4 values.
#include "paged_decode.cuh"

namespace kvq {
namespace paged {

cudaError_t launch_24(const PagedDecodeArgs& a, cudaStream_t s) { return launch_bits<2, 4>(a, s); }
KVQ_BOUNDS_COUNTER(bounds_24)

}  // namespace paged
}  // namespace kvq
