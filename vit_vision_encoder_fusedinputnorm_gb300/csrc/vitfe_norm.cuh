// Layer norm's kernels.  With xh = (x - mean) rstd, rstd = 1 / sqrt(mean((x - mean)^2) + eps):
//   y = xh w + b
//   g = dout w;  dx = rstd (g - mean(g) - xh mean(g xh));  dw = sum over rows of dout xh;  db = of dout
// Some ten operations an element either way: memory bound.  All of it is held in fp32, and what is
// stored in fewer bits is rounded once.
//
// A group of T threads holds one row: each thread owns at most 64 of its columns, so the row's
// statistics are passes over registers, and the weight's gradient is summed in registers over all
// rows of the group.
#pragma once

#include "vitfe_block.cuh"

namespace vitfe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormStages = 8;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// The lanes of a thread's group; a warp may hold several, each at a row of its own.
template <int T>
__device__ __forceinline__ unsigned group_lanes() {
  if constexpr (T >= 32) return 0xffffffffu;
  else return ((1u << T) - 1u) << (threadIdx.x & 31 & ~(T - 1));
}

template <int T>
__device__ __forceinline__ void group_sync(int g) {
  if constexpr (T <= 32) __syncwarp(group_lanes<T>());
  else if constexpr (T == kNormThreads) __syncthreads();
  else named_bar_sync(1 + g, T);
}

// Sums over the group of N values a thread.  Two buffers in turn, so one barrier a call is enough.
template <int T, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*red)[kNormThreads / 32][2], int g, int& turn) {
#pragma unroll
  for (int d = T < 32 ? T / 2 : 16; d >= 1; d >>= 1) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(group_lanes<T>(), v[n], d);
  }
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) red[turn][threadIdx.x >> 5][n] = v[n];
    }
    group_sync<T>(g);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) v[n] += red[turn][g * W + i][n];
    }
    turn ^= 1;
  }
}

// A row's place in memory, widened to whole 16-byte words (each of which holds a byte of it).
struct RowSpan {
  const char* from;
  uint32_t bytes, skip;
};
__device__ __forceinline__ RowSpan row_span(const void* p, int64_t r, int64_t stride, int width, int size) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p) + (uintptr_t)(r * stride * size);
  const uintptr_t lo = at & ~(uintptr_t)15, hi = (at + (uintptr_t)(width * size) + 15) & ~(uintptr_t)15;
  return RowSpan{reinterpret_cast<const char*>(lo), (uint32_t)(hi - lo), (uint32_t)(at - lo)};
}

// Elements are handled as pairs (packed fp32 arithmetic): a chunk is one access of V elements, or,
// where rows allow only single elements (V = 1), two of them T columns apart.  A thread has
// C columns; the launch picks the least C of a short list, so all but the last few chunks lie
// inside the row for every thread: no test there.
__host__ __device__ constexpr int least_columns(int T, int C) { return T <= 64 ? (C == 64 ? 48 : C - 8) : C / 2; }

template <int V, int T, int C>
struct Chunks {
  static constexpr int E = V == 1 ? 2 : V;      // elements of a chunk
  static constexpr int P = E / 2;
  static constexpr int N = C / E;
  // column of element e of thread t's i-th chunk
  static __device__ __forceinline__ int col(int i, int t, int e) { return V == 1 ? (2 * i + e) * T + t : (i * T + t) * V + e; }
  static __device__ __forceinline__ bool full(int i) { return (i + 1) * E <= least_columns(T, C); }
  static __device__ __forceinline__ bool has(int i, int t, int e, int width) { return full(i) || col(i, t, e) < width; }
};

template <typename X>
__device__ __forceinline__ uint64_t unpack2(uint32_t v);
template <>
__device__ __forceinline__ uint64_t unpack2<__nv_bfloat16>(uint32_t v) {
  return (uint64_t)(v << 16) | ((uint64_t)(v & 0xffff0000u) << 32);
}
template <>
__device__ __forceinline__ uint64_t unpack2<__half>(uint32_t v) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return f32x2(f.x, f.y);
}

// Chunk i of a row, or 0 past its end; `p` points at the thread's first column.
template <typename X, int V, int T, int C>
__device__ __forceinline__ void load_chunk(const X* p, int i, int t, int width, uint64_t (&v)[Chunks<V, T, C>::P]) {
  using Ch = Chunks<V, T, C>;
  if constexpr (V == 1) {
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) f[e] = Ch::has(i, t, e, width) ? to_f32(p[(2 * i + e) * T]) : 0.f;
    v[0] = f32x2(f[0], f[1]);
  } else if (Ch::has(i, t, 0, width)) {
    p += i * T * V;
    if constexpr (sizeof(X) == 4) {
      const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(p);
      v[0] = x.x;
      v[1] = x.y;
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      v[0] = unpack2<X>(x.x);
      v[1] = unpack2<X>(x.y);
      v[2] = unpack2<X>(x.z);
      v[3] = unpack2<X>(x.w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < Ch::P; ++e) v[e] = 0;
  }
}

template <typename X, int V, int T, int C>
__device__ __forceinline__ void store_chunk(X* p, int i, int t, int width, const uint64_t (&v)[Chunks<V, T, C>::P]) {
  using Ch = Chunks<V, T, C>;
  if constexpr (V == 1) {
    if (Ch::has(i, t, 0, width)) p[2 * i * T] = from_f32<X>(lo_f32(v[0]));
    if (Ch::has(i, t, 1, width)) p[(2 * i + 1) * T] = from_f32<X>(hi_f32(v[0]));
  } else if (Ch::has(i, t, 0, width)) {
    p += i * T * V;
    if constexpr (sizeof(X) == 4)
      *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v[0], v[1]);
    else
      *reinterpret_cast<uint4*>(p) = make_uint4(pack2<X>(lo_f32(v[0]), hi_f32(v[0])), pack2<X>(lo_f32(v[1]), hi_f32(v[1])),
                                                pack2<X>(lo_f32(v[2]), hi_f32(v[2])), pack2<X>(lo_f32(v[3]), hi_f32(v[3])));
  }
}

// A vector as fp32 in shared memory, laid out so that every warp's chunk is a run of 8 or 16 bytes a
// thread: no bank conflicts.  The place of column c:
template <int V, int T, int C>
__device__ __forceinline__ int staged_at(int c) {
  using Ch = Chunks<V, T, C>;
  int i, t, e;
  if constexpr (V == 1) {
    i = c / (2 * T);
    e = c / T & 1;
    t = c % T;
  } else {
    i = c / (T * V);
    t = c / V % T;
    e = c % V;
  }
  constexpr int W = Ch::E < 4 ? Ch::E : 4;     // floats of one access
  return ((i * (Ch::E / W) + e / W) * T + t) * W + e % W;
}

// A parameter vector laid out so (no conversion and no type test for each row).
template <int V, int T, int C>
__device__ __forceinline__ void stage_params(float* dst, const void* p, vitfe_dtype d, float none, int width) {
  for (int c = threadIdx.x; c < C * T; c += kNormThreads) {
    float f = none;
    if (p != nullptr && c < width)
      f = d == VITFE_F32    ? static_cast<const float*>(p)[c]
          : d == VITFE_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[c])
                            : to_f32(static_cast<const __half*>(p)[c]);
    dst[staged_at<V, T, C>(c)] = f;
  }
}
// (volatile, as the next one: the compiler would keep what it has read in registers, and spill)
template <int V, int T, int C>
__device__ __forceinline__ void load_params(uint32_t src, int i, int t, uint64_t (&v)[Chunks<V, T, C>::P]) {
  if constexpr (V == 1) {
    asm volatile("ld.volatile.shared.b64 %0, [%1];" : "=l"(v[0]) : "r"(src + 8u * (uint32_t)(i * T + t)));
  } else {
#pragma unroll
    for (int q = 0; q < V / 4; ++q)
      asm volatile("ld.volatile.shared.v2.b64 {%0, %1}, [%2];"
                   : "=l"(v[2 * q]), "=l"(v[2 * q + 1])
                   : "r"(src + 16u * (uint32_t)((i * (V / 4) + q) * T + t)));
  }
}

// Chunk i of a row in shared memory (its bytes from `src`, the thread's first column).
template <typename X, int V, int T, int C>
__device__ __forceinline__ void load_staged(uint32_t src, int i, int t, int width, uint64_t (&v)[Chunks<V, T, C>::P]) {
  using Ch = Chunks<V, T, C>;
  if constexpr (V == 1) {
    float f[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!Ch::has(i, t, e, width)) continue;
      const uint32_t at = src + (uint32_t)((2 * i + e) * T * (int)sizeof(X));
      if constexpr (sizeof(X) == 4) {
        asm volatile("ld.volatile.shared.f32 %0, [%1];" : "=f"(f[e]) : "r"(at));
      } else {
        uint16_t h;
        asm volatile("ld.volatile.shared.u16 %0, [%1];" : "=h"(h) : "r"(at));
        f[e] = to_f32(*reinterpret_cast<const X*>(&h));
      }
    }
    v[0] = f32x2(f[0], f[1]);
  } else if (Ch::has(i, t, 0, width)) {
    const uint32_t at = src + (uint32_t)(i * T * 16);
    if constexpr (sizeof(X) == 4) {
      asm volatile("ld.volatile.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(at));
    } else {
      uint32_t x[4];
      asm volatile("ld.volatile.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                   : "r"(at));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = unpack2<X>(x[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < Ch::P; ++e) v[e] = 0;
  }
}

// Blocks of an SM: as many as the row's registers allow.  bf16: 589,824 x 1280 (40 columns a thread)
// takes 521 us with four, which spill a few, and 486 with three; 589,824 x 640 (24) 242 and 266 us.
__host__ __device__ constexpr int forward_per_sm(int C) { return C <= 24 ? 4 : C <= 40 ? 3 : 2; }

// Forward: the row goes straight to registers (the SM's other rows cover the latency), the mean and the
// squared deviations are two passes over them: one read and one write of memory, and no cancellation.
// bf16, 589,824 x 1280: 486 us, 6.2 TB/s, 92% of what a copy reaches; 18,048 x 1280: 20 us.  A ring of
// bulk copies as the backward pass has took 986 us where this form took 584: the reads of shared
// memory come on top, and the registers it frees are of no use here.
template <typename X, int V, int T, int C>
__global__ void __launch_bounds__(kNormThreads, forward_per_sm(C)) norm_kernel(const NormArgs a) {
  using Ch = Chunks<V, T, C>;
  constexpr int N = Ch::N, P = Ch::P, G = kNormThreads / T;
  extern __shared__ __align__(16) float params[];      // [2][C * T]
  __shared__ float red[2][kNormThreads / 32][2];
  const int t = threadIdx.x % T, g = threadIdx.x / T, width = a.width;
  const int64_t step = (int64_t)gridDim.x * G;
  const float inv_n = 1.0f / (float)width;
  stage_params<V, T, C>(params, a.weight, a.param_dtype, 1.f, width);
  stage_params<V, T, C>(params + C * T, a.bias, a.param_dtype, 0.f, width);
  __syncthreads();
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * G + g; r < a.rows; r += step) {
    const X* x = static_cast<const X*>(a.x) + r * a.x_stride + t * V;
    uint64_t f[N][P];
#pragma unroll
    for (int i = 0; i < N; ++i) load_chunk<X, V, T, C>(x, i, t, width, f[i]);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p) sum[(i + p) & 1] = add_f32x2(sum[(i + p) & 1], f[i][p]);
    sum[0] = add_f32x2(sum[0], sum[1]);
    float m[1] = {lo_f32(sum[0]) + hi_f32(sum[0])};
    group_sum<T>(m, red, g, turn);
    // a true division: 1 / width is rounded, and a row of equal values would deviate from its own mean by
    // a unit of the last place, which rstd (up to 1 / sqrt(eps)) makes large
    const float mean = m[0] / (float)width;
    const uint64_t minus = f32x2(-mean, -mean);
    uint64_t sq[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        f[i][p] = add_f32x2(f[i][p], minus);
        if (!Ch::full(i))                                   // columns past the row deviate by nothing
          f[i][p] = f32x2(Ch::has(i, t, 2 * p, width) ? lo_f32(f[i][p]) : 0.f,
                          Ch::has(i, t, 2 * p + 1, width) ? hi_f32(f[i][p]) : 0.f);
        sq[(i + p) & 1] = fma_f32x2(f[i][p], f[i][p], sq[(i + p) & 1]);
      }
    }
    sq[0] = add_f32x2(sq[0], sq[1]);
    float v[1] = {lo_f32(sq[0]) + hi_f32(sq[0])};
    group_sum<T>(v, red, g, turn);
    const float rstd = rsqrtf(v[0] * inv_n + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    X* y = static_cast<X*>(a.out) + r * a.out_stride + t * V;
    const uint64_t rs = f32x2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint64_t w[P], b[P];
      load_params<V, T, C>(smem_u32(params), i, t, w);
      load_params<V, T, C>(smem_u32(params + C * T), i, t, b);
#pragma unroll
      for (int p = 0; p < P; ++p) f[i][p] = fma_f32x2(mul_f32x2(f[i][p], rs), w[p], b[p]);
      store_chunk<X, V, T, C>(y, i, t, width, f[i]);
    }
  }
}

__host__ __device__ constexpr int backward_per_sm(int C) { return C <= 8 ? 3 : C <= 32 ? 2 : 1; }

// Backward: rows of x and dout arrive in shared memory through a ring of bulk copies that the
// group's first thread keeps `stages` rows ahead (registers hold the parameter sums, not rows in
// flight), and are read twice: for the sums, then for
//   dx = rstd (dout w + (x - mean) A + B),  A = -rstd mean(g xh),  B = -mean(g).
// The mean is subtracted first, as in the forward pass: x rstd - mean rstd would lose the digits that
// rows far from zero have in common.  (It costs an addition a pair: 589,824 x 1280 684 -> 687 us, rows of
// 1027, which move single elements, 167 -> 173; rstd inside A and B, a register pair more, 691 and 186.)
// Each block leaves one row of parameter sums, in a fixed order: no atomics, the same bits every time.
// bf16, 589,824 x 1280: 687 us, 6.6 TB/s, 97% of what a copy reaches.  18,048 x 1280: 38 us where the
// bytes need 20: the start, the blocks' sums and the kernel that adds them are some 17 us of it,
// whatever the rows (9 us where only dx is asked for).
template <typename X, int V, int T, int C>
__global__ void __launch_bounds__(kNormThreads, backward_per_sm(C)) norm_backward_kernel(const NormArgs a, int stages,
                                                                                       int slot) {
  using Ch = Chunks<V, T, C>;
  constexpr int N = Ch::N, P = Ch::P, G = kNormThreads / T;
  extern __shared__ __align__(16) char raw[];           // weight [C * T] fp32, then the ring
  __shared__ uint64_t full[G][kNormStages];
  __shared__ float red[2][kNormThreads / 32][2];
  __shared__ int abort_flag;
  const int t = threadIdx.x % T, g = threadIdx.x / T, width = a.width;
  float* weight = reinterpret_cast<float*>(raw);
  char* ring = raw + C * T * sizeof(float);
  if (threadIdx.x == 0) abort_flag = 0;
  if (t == 0)
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&full[g][i]), 1);
  fence_mbar_init();
  __syncthreads();
  grid_dep_trigger();                         // the sum of the partial rows may be set up meanwhile
  char* mine = ring + (size_t)g * stages * 2 * slot;
  const int64_t first = (int64_t)blockIdx.x * G + g, step = (int64_t)gridDim.x * G;
  auto fetch = [&](int64_t r, int st) {       // by the group's first thread
    const uint32_t bar = smem_u32(&full[g][st]), dst = smem_u32(mine + (size_t)st * 2 * slot);
    const RowSpan x = row_span(a.x, r, a.x_stride, a.width, sizeof(X));
    const RowSpan d = row_span(a.dout, r, a.dout_stride, a.width, sizeof(X));
    mbar_arrive_expect_tx(bar, x.bytes + d.bytes);
    bulk_load(dst, x.from, x.bytes, bar);
    bulk_load(dst + (uint32_t)slot, d.from, d.bytes, bar);
  };
  if (t == 0 && !a.stall)
    for (int i = 0; i < stages && first + i * step < a.rows; ++i) fetch(first + i * step, i);
  stage_params<V, T, C>(weight, a.weight, a.param_dtype, 1.f, width);
  __syncthreads();
  uint64_t dw[N][P], db[N][P];
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int p = 0; p < P; ++p) dw[i][p] = db[i][p] = 0;
  }
  const float inv_n = 1.0f / (float)a.width;
  int st = 0, turn = 0;
  uint32_t phase = 0;
  float mean_next = first < a.rows ? __ldg(a.mean + first) : 0.f, rstd_next = first < a.rows ? __ldg(a.rstd + first) : 0.f;
  for (int64_t r = first; r < a.rows; r += step) {
    const float mean = mean_next;
    float rstd = rstd_next;
    if (r + step < a.rows) {
      mean_next = __ldg(a.mean + r + step);
      rstd_next = __ldg(a.rstd + r + step);
    }
    // a bound on a wait for this group's own copy: a row that never came gives NaN
    const bool here = mbar_wait(smem_u32(&full[g][st]), phase, &abort_flag, a.wait_ns);
    if (!here) rstd = __int_as_float(0x7fffffff);
    const uint32_t slot0 = smem_u32(mine + (size_t)st * 2 * slot) + (uint32_t)(t * V * (int)sizeof(X));
    const uint32_t x = slot0 + row_span(a.x, r, a.x_stride, width, sizeof(X)).skip;
    const uint32_t dy = slot0 + (uint32_t)slot + row_span(a.dout, r, a.dout_stride, width, sizeof(X)).skip;
    const uint64_t rs = f32x2(rstd, rstd), minus = f32x2(-mean, -mean);
    uint64_t s1 = 0, s2 = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint64_t fx[P], fd[P], w[P];
      load_staged<X, V, T, C>(x, i, t, width, fx);
      load_staged<X, V, T, C>(dy, i, t, width, fd);         // 0 past the row, so nothing is added there
      load_params<V, T, C>(smem_u32(weight), i, t, w);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint64_t u = mul_f32x2(fd[p], add_f32x2(fx[p], minus));      // dout xh / rstd
        dw[i][p] = fma_f32x2(u, rs, dw[i][p]);
        db[i][p] = add_f32x2(db[i][p], fd[p]);
        s1 = fma_f32x2(fd[p], w[p], s1);
        s2 = fma_f32x2(u, w[p], s2);
      }
    }
    float s[2] = {lo_f32(s1) + hi_f32(s1), lo_f32(s2) + hi_f32(s2)};
    group_sum<T>(s, red, g, turn);
    const float fa = -rstd * rstd * (s[1] * inv_n), fb = -(s[0] * inv_n);
    const uint64_t pa = f32x2(fa, fa), pb = f32x2(fb, fb);
    X* dx = static_cast<X*>(a.out) + r * a.out_stride + t * V;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint64_t fx[P], fd[P], w[P];
      load_staged<X, V, T, C>(x, i, t, width, fx);
      load_staged<X, V, T, C>(dy, i, t, width, fd);
      load_params<V, T, C>(smem_u32(weight), i, t, w);
#pragma unroll
      for (int p = 0; p < P; ++p)
        fx[p] = mul_f32x2(fma_f32x2(fd[p], w[p], fma_f32x2(add_f32x2(fx[p], minus), pa, pb)), rs);
      store_chunk<X, V, T, C>(dx, i, t, width, fx);
    }
    group_sync<T>(g);                         // the slot has been read
    // (a slot whose copy did not come takes no other: its barrier still counts the first one)
    if (t == 0 && here && r + stages * step < a.rows) fetch(r + stages * step, st);
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
  }
  if (*(volatile int*)&abort_flag) {          // copies still in flight: time to land before the block ends
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000ull) __nanosleep(1000);
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.width;
  float* part = reinterpret_cast<float*>(ring);      // [2][C * T], staged; the rows are done with
  constexpr int W = P < 2 ? P : 2;                    // pairs of one access
  __syncthreads();
  for (int j = 0; j < G; ++j) {                       // group after group: a fixed order of sums
    if (g == j) {
      auto add = [&](float* to, const uint64_t (&v)[N][P]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
          for (int q = 0; q < P; q += W) {
            uint64_t* at = reinterpret_cast<uint64_t*>(to) + ((i * (P / W) + q / W) * T + t) * W;
#pragma unroll
            for (int e = 0; e < W; ++e) at[e] = j ? add_f32x2(at[e], v[i][q + e]) : v[i][q + e];
          }
        }
      };
      add(part, dw);
      add(part + C * T, db);
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * a.width; c += kNormThreads) {
    const float sum = c < a.width ? part[staged_at<V, T, C>(c)] : part[C * T + staged_at<V, T, C>(c - a.width)];
    out[c] = abort_flag ? __int_as_float(0x7fffffff) : sum;
  }
}

// Whether every row and parameter vector starts on 16 bytes and holds a multiple of it.
bool rows_vec16(const NormArgs& a, bool backward) {
  const int v = 16 / dtype_bytes(a.dtype);
  auto ok = [&](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows <= 1 || stride % v == 0);
  };
  auto par = [&](const void* p) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  return a.width % v == 0 && ok(a.x, a.x_stride) && ok(a.out, a.out_stride) && par(a.weight) && par(a.bias) &&
         (!backward || ok(a.dout, a.dout_stride));
}

// Blocks of the backward pass (one partial row of parameter sums each).
int64_t backward_blocks(int64_t rows, int width) {
  const int t = width <= 128 ? 8 : width <= 256 ? 16 : width <= 768 ? 32 : width <= 2048 ? 64 : width <= 4096 ? 128 : 256;
  const int64_t want = (rows + kNormThreads / t - 1) / (kNormThreads / t);
  const int64_t most = 152 * (width <= 64 ? 3 : width <= 8192 ? 2 : 1);
  return want < most ? (want > 0 ? want : 1) : most;
}

template <typename X, int V, int T, int C, bool kBackward>
cudaError_t launch_one(const NormArgs& a, cudaStream_t s) {
  constexpr int G = kNormThreads / T;
  if constexpr (!kBackward) {
    const int64_t want = (a.rows + G - 1) / G, most = 152 * (T == 256 ? 1 : forward_per_sm(C));
    const int smem = 2 * C * T * (int)sizeof(float);
    if (smem > 48 * 1024) {
      static std::atomic<uint64_t> allowed{0};
      cudaError_t e = allow_smem(reinterpret_cast<const void*>(norm_kernel<X, V, T, C>), smem, allowed);
      if (e != cudaSuccess) return e;
    }
    norm_kernel<X, V, T, C><<<(unsigned)(want < most ? want : most), kNormThreads, smem, s>>>(a);
    return cudaGetLastError();
  } else {
    // a slot holds the row and what the widening to 16-byte words may add; as many stages as fit
    // beside the SM's other block
    const int slot = (a.width * (int)sizeof(X) + 30 + 15) / 16 * 16;
    const int fixed = C * T * (int)sizeof(float);
    int stages = (216 / backward_per_sm(C) * 1024 - fixed) / (G * 2 * slot);
    stages = stages > kNormStages ? kNormStages : stages < 1 ? 1 : stages;
    int smem = G * stages * 2 * slot;
    if (smem < 2 * C * T * (int)sizeof(float)) smem = 2 * C * T * (int)sizeof(float);
    smem += fixed;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(norm_backward_kernel<X, V, T, C>), 222 * 1024, allowed);
    if (e != cudaSuccess) return e;
    norm_backward_kernel<X, V, T, C><<<(unsigned)backward_blocks(a.rows, a.width), kNormThreads, smem, s>>>(a, stages, slot);
    return cudaGetLastError();
  }
}

// The narrowest group whose threads hold at most 64 columns each (backward: 32, as each column takes
// two registers for the whole call), and for the widths in use the fewest columns that do.
template <typename X, int V>
cudaError_t launch_forward(const NormArgs& a, cudaStream_t s) {
  const int c = (a.width + 31) / 32;
  if (a.width <= 64) return launch_one<X, V, 8, 8, false>(a, s);
  if (a.width <= 128) return launch_one<X, V, 8, 16, false>(a, s);
  if (a.width <= 256) return launch_one<X, V, 16, 16, false>(a, s);
  if (c <= 16) return launch_one<X, V, 32, 16, false>(a, s);
  if (c <= 24) return launch_one<X, V, 32, 24, false>(a, s);
  if (c <= 32) return launch_one<X, V, 32, 32, false>(a, s);
  if (c <= 40) return launch_one<X, V, 32, 40, false>(a, s);
  if (c <= 48) return launch_one<X, V, 32, 48, false>(a, s);
  if (c <= 64) return launch_one<X, V, 32, 64, false>(a, s);
  if (a.width <= 64 * 40) return launch_one<X, V, 64, 40, false>(a, s);
  if (a.width <= 64 * 48) return launch_one<X, V, 64, 48, false>(a, s);
  if (a.width <= 64 * 64) return launch_one<X, V, 64, 64, false>(a, s);
  if (a.width <= 128 * 64) return launch_one<X, V, 128, 64, false>(a, s);
  return launch_one<X, V, 256, 64, false>(a, s);
}
template <typename X, int V>
cudaError_t launch_backward(const NormArgs& a, cudaStream_t s) {
  if (a.width <= 64) return launch_one<X, V, 8, 8, true>(a, s);
  if (a.width <= 128) return launch_one<X, V, 8, 16, true>(a, s);
  if (a.width <= 256) return launch_one<X, V, 16, 16, true>(a, s);
  if (a.width <= 32 * 16) return launch_one<X, V, 32, 16, true>(a, s);
  if (a.width <= 32 * 24) return launch_one<X, V, 32, 24, true>(a, s);
  if (a.width <= 64 * 16) return launch_one<X, V, 64, 16, true>(a, s);
  if (a.width <= 64 * 24) return launch_one<X, V, 64, 24, true>(a, s);
  if (a.width <= 64 * 32) return launch_one<X, V, 64, 32, true>(a, s);
  if (a.width <= 128 * 32) return launch_one<X, V, 128, 32, true>(a, s);
  if (a.width <= 256 * 32) return launch_one<X, V, 256, 32, true>(a, s);
  return launch_one<X, V, 256, 64, true>(a, s);
}
template <typename X, int V, bool kBackward>
cudaError_t launch_group(const NormArgs& a, cudaStream_t s) {
  if constexpr (kBackward) return launch_backward<X, V>(a, s);
  else return launch_forward<X, V>(a, s);
}
template <typename X, bool kBackward>
cudaError_t launch_width(const NormArgs& a, cudaStream_t s) {
  return rows_vec16(a, kBackward) ? launch_group<X, 16 / (int)sizeof(X), kBackward>(a, s)
                                  : launch_group<X, 1, kBackward>(a, s);
}
template <bool kBackward>
cudaError_t launch_any(const NormArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case VITFE_BF16: return launch_width<__nv_bfloat16, kBackward>(a, s);
    case VITFE_F16: return launch_width<__half, kBackward>(a, s);
    default: return launch_width<float, kBackward>(a, s);
  }
}

}  // namespace

}  // namespace vitfe
