// Layer norm, forward and backward.
#include "vitfe_block.cuh"

namespace vitfe {
namespace {

constexpr int kNormThreads = 256;

// One row is held by a group of T threads (a warp, or the whole block), K vectors of V
// elements each: thread t owns columns (k * T + t) * V ..., so the row is read once and both
// statistics passes run on registers.
template <int T>
__device__ __forceinline__ float group_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (T > 32) {
    const int w = threadIdx.x >> 5;
    __syncthreads();                       // red may still be read from the call before
    if ((threadIdx.x & 31) == 0) red[w] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < T / 32; ++i) v += red[i];
  }
  return v;
}

template <typename X, int V, int T, int K>
__global__ void __launch_bounds__(T > kNormThreads ? T : kNormThreads) norm_kernel(const NormArgs a) {
  __shared__ float red[32];
  const int t = threadIdx.x % T;
  const int64_t groups = (int64_t)gridDim.x * (blockDim.x / T);
  for (int64_t r = (int64_t)blockIdx.x * (blockDim.x / T) + threadIdx.x / T; r < a.rows; r += groups) {
    const X* x = static_cast<const X*>(a.x) + r * a.x_stride;
    float f[K][V];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * T + t) * V;
      if (c < a.width) {
        const Vec<X, V> v = *reinterpret_cast<const Vec<X, V>*>(x + c);
#pragma unroll
        for (int e = 0; e < V; ++e) f[k][e] = to_f32(v.v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[k][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) sum += f[k][e];
    }
    const float mean = group_sum<T>(sum, red) / (float)a.width;
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if ((k * T + t) * V < a.width) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = f[k][e] - mean;
          sq = fmaf(d, d, sq);
        }
      }
    }
    const float rstd = 1.0f / sqrtf(group_sum<T>(sq, red) / (float)a.width + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    X* y = static_cast<X*>(a.out) + r * a.out_stride;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * T + t) * V;
      if (c >= a.width) continue;
      float w[V], b[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[e] = 1.f;
        b[e] = 0.f;
      }
      if (a.weight) load_params<V>(a.weight, a.param_dtype, c, w);
      if (a.bias) load_params<V>(a.bias, a.param_dtype, c, b);
      Vec<X, V> v;
#pragma unroll
      for (int e = 0; e < V; ++e) v.v[e] = from_f32<X>(fmaf((f[k][e] - mean) * rstd, w[e], b[e]));
      *reinterpret_cast<Vec<X, V>*>(y + c) = v;
    }
  }
}

// dx row by row; the weight's and bias's gradients are summed over the block's rows in
// registers (each thread owns its columns), then over the block's groups in shared memory,
// and written as one partial row per block.
template <typename X, int V, int T, int K>
__global__ void __launch_bounds__(T > kNormThreads ? T : kNormThreads) norm_backward_kernel(const NormArgs a) {
  extern __shared__ float part[];          // [2][width] when the block holds several groups
  __shared__ float red[32];
  const int t = threadIdx.x % T;
  const int g = threadIdx.x / T;
  const int64_t groups = (int64_t)gridDim.x * (blockDim.x / T);
  float dw[K][V], db[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int e = 0; e < V; ++e) dw[k][e] = db[k][e] = 0.f;
  }
  const float inv_n = 1.0f / (float)a.width;
  for (int64_t r = (int64_t)blockIdx.x * (blockDim.x / T) + g; r < a.rows; r += groups) {
    const X* x = static_cast<const X*>(a.x) + r * a.x_stride;
    const X* dy = static_cast<const X*>(a.dout) + r * a.dout_stride;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float xh[K][V], gr[K][V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * T + t) * V;
      if (c >= a.width) continue;
      const Vec<X, V> vx = *reinterpret_cast<const Vec<X, V>*>(x + c);
      const Vec<X, V> vd = *reinterpret_cast<const Vec<X, V>*>(dy + c);
      float w[V];
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = 1.f;
      if (a.weight) load_params<V>(a.weight, a.param_dtype, c, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float h = (to_f32(vx.v[e]) - mean) * rstd;
        const float d = to_f32(vd.v[e]);
        dw[k][e] = fmaf(d, h, dw[k][e]);
        db[k][e] += d;
        xh[k][e] = h;
        gr[k][e] = d * w[e];
        s1 += gr[k][e];
        s2 = fmaf(gr[k][e], h, s2);
      }
    }
    s1 = group_sum<T>(s1, red) * inv_n;
    s2 = group_sum<T>(s2, red) * inv_n;
    X* dx = static_cast<X*>(a.out) + r * a.out_stride;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * T + t) * V;
      if (c >= a.width) continue;
      Vec<X, V> v;
#pragma unroll
      for (int e = 0; e < V; ++e) v.v[e] = from_f32<X>(rstd * (gr[k][e] - s1 - xh[k][e] * s2));
      *reinterpret_cast<Vec<X, V>*>(dx + c) = v;
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.width;
  if constexpr (T >= kNormThreads) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * T + t) * V;
      if (c >= a.width) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        out[c + e] = dw[k][e];
        out[a.width + c + e] = db[k][e];
      }
    }
  } else {
    for (int i = 0; i < kNormThreads / T; ++i) {   // group after group: a fixed order of sums
      if (g == i) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int c = (k * T + t) * V;
          if (c >= a.width) continue;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            part[c + e] = (i ? part[c + e] : 0.f) + dw[k][e];
            part[a.width + c + e] = (i ? part[a.width + c + e] : 0.f) + db[k][e];
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * a.width; c += kNormThreads) out[c] = part[c];
  }
}

// Sum of the blocks' partial rows: a block of 32 x 8 threads takes 32 columns.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* __restrict__ partial, int blocks, int width,
                                                          float* __restrict__ dweight, float* __restrict__ dbias) {
  __shared__ float red[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31);
  const int w = threadIdx.x >> 5;
  float s = 0.f;
  if (c < 2 * width)
    for (int b = w; b < blocks; b += 8) s += partial[(int64_t)b * 2 * width + c];
  red[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w == 0 && c < 2 * width) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x & 31];
    if (c < width) {
      if (dweight) dweight[c] = s;
    } else if (dbias) {
      dbias[c - width] = s;
    }
  }
}

// The widest access that every row and parameter start allows.
bool rows_vec16(const NormArgs& a, bool backward) {
  const int v = 16 / dtype_bytes(a.dtype);
  auto ok = [&](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows <= 1 || stride % v == 0);
  };
  auto par = [&](const void* p) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  return a.width % v == 0 && ok(a.x, a.x_stride) && ok(a.out, a.out_stride) && par(a.weight) && par(a.bias) &&
         (!backward || ok(a.dout, a.dout_stride));
}

template <typename X, int V, int T, int K>
cudaError_t launch_one(const NormArgs& a, bool backward, int blocks, cudaStream_t s) {
  constexpr int threads = T > kNormThreads ? T : kNormThreads;
  if (!backward) {
    norm_kernel<X, V, T, K><<<blocks, threads, 0, s>>>(a);
  } else {
    const size_t smem = (T < kNormThreads && a.partial) ? (size_t)2 * a.width * sizeof(float) : 0;
    norm_backward_kernel<X, V, T, K><<<blocks, threads, smem, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename X, int V>
cudaError_t launch_typed(const NormArgs& a, bool backward, int blocks, cudaStream_t s) {
  const int vecs = (a.width + V - 1) / V;
  // a warp per row while a thread holds at most 8 vectors; then the block, then a block of 1024
  const int k32 = (vecs + 31) / 32, k256 = (vecs + 255) / 256;
  if (k32 <= 1) return launch_one<X, V, 32, 1>(a, backward, blocks, s);
  if (k32 <= 2) return launch_one<X, V, 32, 2>(a, backward, blocks, s);
  if (k32 <= 3) return launch_one<X, V, 32, 3>(a, backward, blocks, s);
  if (k32 <= 5) return launch_one<X, V, 32, 5>(a, backward, blocks, s);
  if (k32 <= 8) return launch_one<X, V, 32, 8>(a, backward, blocks, s);
  if (k256 <= 2) return launch_one<X, V, 256, 2>(a, backward, blocks, s);
  if (k256 <= 4) return launch_one<X, V, 256, 4>(a, backward, blocks, s);
  if (k256 <= 8) return launch_one<X, V, 256, 8>(a, backward, blocks, s);
  return launch_one<X, V, 1024, 16>(a, backward, blocks, s);   // 16384 columns one by one
}

template <typename X>
cudaError_t launch_width(const NormArgs& a, bool backward, int blocks, cudaStream_t s) {
  if (rows_vec16(a, backward)) return launch_typed<X, 16 / sizeof(X)>(a, backward, blocks, s);
  return launch_typed<X, 1>(a, backward, blocks, s);
}

cudaError_t launch_any(const NormArgs& a, bool backward, int blocks, cudaStream_t s) {
  switch (a.dtype) {
    case VITFE_BF16: return launch_width<__nv_bfloat16>(a, backward, blocks, s);
    case VITFE_F16: return launch_width<__half>(a, backward, blocks, s);
    default: return launch_width<float>(a, backward, blocks, s);
  }
}

int64_t backward_blocks(int64_t rows) {
  const int64_t want = (rows + 7) / 8;
  return want < 304 ? (want > 0 ? want : 1) : 304;
}

}  // namespace

int64_t layer_norm_workspace(int64_t rows, int width) {
  return backward_blocks(rows) * 2 * width * (int64_t)sizeof(float);
}

cudaError_t launch_layer_norm(const NormArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  const int64_t blocks = (a.rows + 7) / 8;
  return launch_any(a, false, (int)(blocks < 1216 ? blocks : 1216), s);
}

cudaError_t launch_layer_norm_backward(const NormArgs& a, cudaStream_t s) {
  const int blocks = (int)backward_blocks(a.rows);
  if (a.rows > 0 || a.partial) {
    cudaError_t e = launch_any(a, true, blocks, s);
    if (e != cudaSuccess) return e;
  }
  if (a.partial) {
    norm_reduce_kernel<<<(2 * a.width + 31) / 32, 256, 0, s>>>(a.partial, blocks, a.width, a.dweight, a.dbias);
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace vitfe
