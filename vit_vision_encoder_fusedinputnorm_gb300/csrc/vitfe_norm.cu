// Layer norm: the forward pass.
#include "vitfe_norm.cuh"

namespace vitfe {

cudaError_t launch_layer_norm(const NormArgs& a, cudaStream_t s) {
  return a.rows == 0 ? cudaSuccess : launch_any<false>(a, s);
}

}  // namespace vitfe
