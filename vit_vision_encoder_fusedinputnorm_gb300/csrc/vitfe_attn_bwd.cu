// Attention over packed sequences: the backward pass.
#include "vitfe_attn.cuh"

namespace vitfe {
namespace {

// dq and delta: a warp per query row.
template <typename T>
__global__ void __launch_bounds__(256) attn_dq_kernel(const AttnArgs a) {
  const AttnPlanHdr* hdr = reinterpret_cast<const AttnPlanHdr*>(a.plan);
  const AttnItem* items = reinterpret_cast<const AttnItem*>(a.plan + a.l.at_items);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = a.s.heads_kv, g = a.l.group, d = a.s.head_dim;
  float* delta = static_cast<float*>(a.workspace);
  if (a.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0) {
    a.status[0] = kOk;
    a.status[1] = -1;
  }
  for (int w = blockIdx.x; w < hdr->n_items * hk; w += gridDim.x) {
    const AttnItem it = items[w / hk];
    if (it.kb > 0) continue;               // the first piece of a cut item takes all of it
    const int kh = w % hk;
    for (int r = warp; r < it.qn * g; r += 8) {
      const int tok = r / g, head = kh * g + r % g;
      const int lim = a.s.causal ? min(it.kn, it.off + tok + 1) : it.kn;
      const int64_t row = it.q0 + tok;
      const T* q = static_cast<const T*>(a.q) + row * a.q_stride + head * d;
      const T* od = static_cast<const T*>(a.out) + row * a.out_stride + head * d;
      const T* dd = static_cast<const T*>(a.dout) + row * a.dout_stride + head * d;
      float fq[4], fd[4], dq[4] = {0.f, 0.f, 0.f, 0.f}, dl = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = lane + 32 * i < d;
        fq[i] = in ? to_f32(q[lane + 32 * i]) * a.scale : 0.f;
        fd[i] = in ? to_f32(dd[lane + 32 * i]) : 0.f;
        if (in) dl = fmaf(fd[i], to_f32(od[lane + 32 * i]), dl);
      }
      dl = warp_sum(dl);
      if (lane == 0) delta[row * a.s.heads_q + head] = dl;
      const float lse = a.lse[row * a.s.heads_q + head];
      for (int j = 0; j < lim; ++j) {
        const T* k = static_cast<const T*>(a.k) + (int64_t)(it.k0 + j) * a.k_stride + kh * d;
        const T* v = static_cast<const T*>(a.v) + (int64_t)(it.k0 + j) * a.v_stride + kh * d;
        float s = 0.f, dp = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < d) {
            s = fmaf(fq[i], to_f32(k[lane + 32 * i]), s);
            dp = fmaf(fd[i], to_f32(v[lane + 32 * i]), dp);
          }
        s = warp_sum(s);
        dp = warp_sum(dp);
        const float ds = __expf(s - lse) * (dp - dl) * a.scale;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < d) dq[i] = fmaf(ds, to_f32(k[lane + 32 * i]), dq[i]);
      }
      T* o = static_cast<T*>(a.dq) + row * a.dq_stride + head * d;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < d) o[lane + 32 * i] = from_f32<T>(dq[i]);
    }
  }
}

// dk and dv: a warp per key row, over the tokens and query heads that read it.
template <typename T>
__global__ void __launch_bounds__(256) attn_dkv_kernel(const AttnArgs a) {
  const AttnPlanHdr* hdr = reinterpret_cast<const AttnPlanHdr*>(a.plan);
  const AttnKeyItem* items = reinterpret_cast<const AttnKeyItem*>(a.plan + a.l.at_keys);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = a.s.heads_kv, g = a.l.group, d = a.s.head_dim;
  const float* delta = static_cast<const float*>(a.workspace);
  for (int w = blockIdx.x; w < hdr->n_keys * hk; w += gridDim.x) {
    const AttnKeyItem it = items[w / hk];
    const int kh = w % hk;
    for (int j = warp; j < it.kn; j += 8) {
      const T* k = static_cast<const T*>(a.k) + (int64_t)(it.k0 + j) * a.k_stride + kh * d;
      const T* v = static_cast<const T*>(a.v) + (int64_t)(it.k0 + j) * a.v_stride + kh * d;
      float fk[4], fv[4], dk[4] = {0.f, 0.f, 0.f, 0.f}, dv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = lane + 32 * i < d;
        fk[i] = in ? to_f32(k[lane + 32 * i]) * a.scale : 0.f;
        fv[i] = in ? to_f32(v[lane + 32 * i]) : 0.f;
      }
      for (int r = max(0, j - it.off) * g; r < it.qn * g; ++r) {
        const int64_t row = it.q0 + r / g;
        const int head = kh * g + r % g;
        const T* q = static_cast<const T*>(a.q) + row * a.q_stride + head * d;
        const T* dd = static_cast<const T*>(a.dout) + row * a.dout_stride + head * d;
        float s = 0.f, dp = 0.f, fq[4], fd[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = lane + 32 * i < d;
          fq[i] = in ? to_f32(q[lane + 32 * i]) : 0.f;
          fd[i] = in ? to_f32(dd[lane + 32 * i]) : 0.f;
          s = fmaf(fq[i], fk[i], s);
          dp = fmaf(fd[i], fv[i], dp);
        }
        s = warp_sum(s);
        dp = warp_sum(dp);
        const float p = __expf(s - a.lse[row * a.s.heads_q + head]);
        const float ds = p * (dp - delta[row * a.s.heads_q + head]) * a.scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dv[i] = fmaf(p, fd[i], dv[i]);
          dk[i] = fmaf(ds, fq[i], dk[i]);
        }
      }
      T* ok = static_cast<T*>(a.dk) + (int64_t)(it.k0 + j) * a.dk_stride + kh * d;
      T* ov = static_cast<T*>(a.dv) + (int64_t)(it.k0 + j) * a.dv_stride + kh * d;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < d) {
          ok[lane + 32 * i] = from_f32<T>(dk[i]);
          ov[lane + 32 * i] = from_f32<T>(dv[i]);
        }
    }
  }
}

template <typename T>
cudaError_t launch_typed(const AttnArgs& a, cudaStream_t st) {
  const int64_t wq = a.l.cap_items * a.s.heads_kv, wk = a.l.cap_keys * a.s.heads_kv;
  if (wq > 0) attn_dq_kernel<T><<<(unsigned)(wq < 1216 ? wq : 1216), 256, 0, st>>>(a);
  if (wk > 0) attn_dkv_kernel<T><<<(unsigned)(wk < 1216 ? wk : 1216), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_backward(const AttnArgs& a, cudaStream_t st) {
  return a.s.dtype == VITFE_F16 ? launch_typed<__half>(a, st) : launch_typed<__nv_bfloat16>(a, st);
}

}  // namespace vitfe
