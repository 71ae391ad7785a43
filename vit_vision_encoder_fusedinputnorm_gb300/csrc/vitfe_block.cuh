// Definitions shared by the encoder-block operators (layer norm, multi-axis rotary, attention).
#pragma once

#include <atomic>

#include <cuda_fp16.h>

#include "vitfe_internal.cuh"

namespace vitfe {

// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------
__host__ __device__ constexpr int dtype_bytes(vitfe_dtype d) { return d == VITFE_F32 ? 4 : 2; }

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

// Two floats rounded to nearest even and packed, `lo` in the lower half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// V consecutive elements as one access of V * sizeof(T) bytes (at most 16).
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// Two fp32 lanes in one 64-bit register.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float lo_f32(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_f32(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// VITFE_TEST_STALL_BLOCK_LOADS=1: the kernels of this call issue no copies.
bool stall_loads();
// SMs of the current device, asked for once per device.
cudaError_t current_sms(int* sms);
// Allow `kernel` up to `smem` bytes of dynamic shared memory on the current device, once per device
// (`done`: a bit for each device below 64, of this kernel alone).  `regs` > 0: the registers a thread
// that the kernel has to be launched with (it shares them out anew); an error when it is not.
cudaError_t allow_smem(const void* kernel, int smem, std::atomic<uint64_t>& done, int regs = 0);

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
struct NormArgs {
  const void* x;
  int64_t x_stride;
  vitfe_dtype dtype;
  int64_t rows;
  int width;
  const void* weight;
  const void* bias;
  vitfe_dtype param_dtype;
  float eps;
  void* out;            // y, or dx
  int64_t out_stride;
  float* mean;          // written by the forward pass, read by the backward pass
  float* rstd;
  const void* dout;     // backward only, as the next ones
  int64_t dout_stride;
  float* dweight;
  float* dbias;
  float* partial;       // [CTA][2][width]
  uint64_t wait_ns;     // bound of a wait
  bool stall;           // tests: load nothing, so that the waits run out
};
cudaError_t launch_layer_norm(const NormArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm_backward(const NormArgs& a, cudaStream_t s);
int64_t layer_norm_workspace(int64_t rows, int width);

struct MropeArgs {
  const int32_t* pos;
  int axes;
  const uint8_t* axis_of_pair;   // host
  int rotary_dim;
  float theta;
  bool inverse;
  int64_t rows;
  int head_dim;
  vitfe_dtype dtype;
  const void* x[2];              // Q, K
  void* y[2];
  int heads[2];
  int64_t x_stride[2], y_stride[2];
};
cudaError_t launch_mrope_apply(const MropeArgs& a, cudaStream_t s);
cudaError_t launch_mrope_positions(const vitfe_span* spans, const int32_t* n_spans, int max_spans,
                                   const vitfe_item* items, const int32_t* n_items, int max_items, int merge,
                                   int64_t rows, int32_t* pos, int32_t* status, cudaStream_t s);

}  // namespace vitfe
