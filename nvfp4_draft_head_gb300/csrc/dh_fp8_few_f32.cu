// The FP8 block-scaled product of few tokens with float32 results.
#include "dh_fp8_few.cuh"

namespace dh {
namespace f8 {

template cudaError_t launch_few<float>(const Fp8BlockArgs&, const FewPlan&, const uint8_t*, int, const float*, cudaStream_t);

}  // namespace f8
}  // namespace dh
