// Layer norm: the backward pass.
#include "vitfe_norm.cuh"

namespace vitfe {
namespace {

// Sum of the blocks' partial rows, [2][width] each: 32 columns by 32 slices of the rows a block, so
// that few loads follow one another (304 rows of 2 x 1280: 4.5 us, latency; set up while the
// kernel before it runs).
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ partial, int blocks, int width,
                                                           float* __restrict__ dweight, float* __restrict__ dbias) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  grid_dep_wait();
  if (c < 2 * width) {
#pragma unroll 8
    for (int b = w; b < blocks; b += 32) s += partial[(int64_t)b * 2 * width + c];
  }
  red[w][lane] = s;
  __syncthreads();
  s = warp_sum(red[lane][w]);                  // warp w sums column w of the 32
  const int col = blockIdx.x * 32 + w;
  if (lane == 0 && col < 2 * width) {
    if (col < width) {
      if (dweight) dweight[col] = s;
    } else if (dbias) {
      dbias[col - width] = s;
    }
  }
}

}  // namespace

int64_t layer_norm_workspace(int64_t rows, int width) {
  return backward_blocks(rows, width) * 2 * width * (int64_t)sizeof(float);
}

cudaError_t launch_layer_norm_backward(const NormArgs& a, cudaStream_t s) {
  if (a.rows == 0 && a.partial == nullptr) return cudaSuccess;
  cudaError_t e = launch_any<true>(a, s);
  if (e != cudaSuccess || a.partial == nullptr) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((2 * a.width + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_reduce_kernel, (const float*)a.partial, (int)backward_blocks(a.rows, a.width),
                            (int)a.width, a.dweight, a.dbias);
}

}  // namespace vitfe
