// rms_norm.cu -- the root-mean-square norm and its gradient (norm.cuh).
#include "norm.cuh"

namespace dgr {

cudaError_t launch_rms_norm(const DeviceInfo &dev, const NormCall &c, cudaStream_t stream) {
  return launch_norm_form<false>(dev, c, stream);
}

cudaError_t launch_rms_norm_grad(const DeviceInfo &dev, const NormGradCall &c,
                                  cudaStream_t stream) {
  return launch_grad_form<false>(dev, c, stream);
}

}  // namespace dgr
