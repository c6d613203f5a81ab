// layer_norm.cu -- the layer norm and its gradient (norm.cuh).
#include "norm.cuh"

namespace dgr {

cudaError_t launch_layer_norm(const DeviceInfo &dev, const NormCall &c, cudaStream_t stream) {
  return launch_norm_form<true>(dev, c, stream);
}

cudaError_t launch_layer_norm_grad(const DeviceInfo &dev, const NormGradCall &c,
                                  cudaStream_t stream) {
  return launch_grad_form<true>(dev, c, stream);
}

}  // namespace dgr
