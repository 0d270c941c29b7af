// Tensor-core path of the decayed attention: not taken by any call yet.
#include "decay.cuh"

namespace la {
namespace decay {

bool tc_supported(const Args&, la_dtype) { return false; }
int tc_segments(int64_t, int, int, int) { return 1; }
cudaError_t tc_run(Args, void*, cudaStream_t) { return cudaErrorNotSupported; }

}  // namespace decay
}  // namespace la
