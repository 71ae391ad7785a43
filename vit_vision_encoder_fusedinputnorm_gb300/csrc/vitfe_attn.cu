// Attention over packed sequences: the plan and the forward pass.
#include "vitfe_attn.cuh"

namespace vitfe {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;

struct PlanArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int rows_q, rows_k, max_seqs, heads_kv, tok2, causal;
  AttnLayout l;
  char* plan;
  int32_t* status;
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((unsigned)a + (unsigned)b - 1u) / (unsigned)b); }

// Exclusive sum over the block; `total` gets the whole sum.
__device__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  __syncthreads();                     // warp_sums may still be read from the call before
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  if (w == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[31];
  return incl - v + (w ? warp_sums[w - 1] : 0);
}

// The rows [a, b) of sequence s; s == n is what follows the last sequence.
__device__ __forceinline__ int2 seq_rows(const int32_t* cu, int n, int s, int rows) {
  if (n == 0) return make_int2(0, rows);
  return make_int2(cu[s], s < n ? cu[s + 1] : rows);
}

// The t-th query item (before any cut).
__device__ AttnItem query_item(const PlanArgs& a, const int* scan, int n, int t) {
  const int s = find_item(scan, n + 1, t);
  const int2 q = seq_rows(a.cu_q, n, s, a.rows_q);
  AttnItem it;
  const int first = (t - scan[s]) * a.tok2;
  it.q0 = q.x + first;
  it.qn = min(a.tok2, q.y - it.q0);
  it.k0 = 0;
  it.kn = 0;
  if (s < n) {
    const int2 k = seq_rows(a.cu_k, n, s, a.rows_k);
    it.k0 = k.x;
    it.kn = k.y - k.x;
  }
  it.off = it.kn;
  int last = it.kn;                    // keys that the item's last token sees
  if (a.causal && s < n) {
    it.off = it.kn - (q.y - q.x) + first;
    last = min(it.kn, max(0, it.off + it.qn));
  }
  it.kb = 0;
  it.ke = ceil_div(last, kAttnKeys);
  it.slot = -1;
  return it;
}

__device__ AttnKeyItem key_item(const PlanArgs& a, const int* scan, int n, int t) {
  const int s = find_item(scan, n + 1, t);
  const int2 k = seq_rows(a.cu_k, n, s, a.rows_k);
  AttnKeyItem it;
  const int first = (t - scan[s]) * kAttnKeys;
  it.k0 = k.x + first;
  it.kn = min(kAttnKeys, k.y - it.k0);
  it.q0 = 0;
  it.qn = 0;
  it.off = kAttnKeys;                  // every token sees every key of the tile
  if (s < n) {
    const int2 q = seq_rows(a.cu_q, n, s, a.rows_q);
    it.q0 = q.x;
    it.qn = q.y - q.x;
    // local key j is the sequence's key first + j: seen when first + j <= i + keys - tokens
    if (a.causal) it.off = (k.y - k.x) - it.qn - first;
  }
  it.pad[0] = it.pad[1] = it.pad[2] = 0;
  return it;
}

// Tokens of a key item that see any of its keys.
__device__ __forceinline__ int key_item_work(const AttnKeyItem& k) { return max(0, k.qn - max(0, -k.off)); }

// One block: checks the boundaries, lists the query and key items of every sequence, cuts long
// key ranges where there are few items, and sorts by length, longest first, so that the
// attention kernels' fixed deal of items to SMs comes out even.  The order among equal
// lengths may vary from call to call; no result depends on it.
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const PlanArgs a) {
  __shared__ int warp_sums[32];
  __shared__ int bins[kBins];
  __shared__ unsigned bad;
  __shared__ unsigned long long blocks_total;
  __shared__ int slots, joins;
  const int tid = threadIdx.x;
  AttnPlanHdr* hdr = reinterpret_cast<AttnPlanHdr*>(a.plan);
  AttnItem* items = reinterpret_cast<AttnItem*>(a.plan + a.l.at_items);
  AttnKeyItem* keys = reinterpret_cast<AttnKeyItem*>(a.plan + a.l.at_keys);
  AttnJoin* join = reinterpret_cast<AttnJoin*>(a.plan + a.l.at_joins);
  int* scan_q = reinterpret_cast<int*>(a.plan + a.l.at_scan_q);
  int* scan_k = reinterpret_cast<int*>(a.plan + a.l.at_scan_k);
  if (tid == 0) {
    bad = 0xffffffffu;
    blocks_total = 0;
    slots = joins = 0;
  }
  __syncthreads();
  int n = a.max_seqs;
  for (int s = tid; s < n; s += kPlanThreads) {
    const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
    if ((s == 0 && (q0 != 0 || k0 != 0)) || q0 < 0 || k0 < 0 || q1 < q0 || k1 < k0 || q1 > a.rows_q || k1 > a.rows_k) atomicMin(&bad, (unsigned)s);
  }
  __syncthreads();
  if (a.status != nullptr && tid == 0) {
    a.status[0] = bad == 0xffffffffu ? kOk : kDesc;
    a.status[1] = bad == 0xffffffffu ? -1 : (int)bad;
  }
  if (bad != 0xffffffffu) n = 0;
  int nq = 0, nk = 0;
  for (int b = 0; b <= n; b += kPlanThreads) {
    const int s = b + tid;
    int cq = 0, ck = 0;
    if (s <= n) {
      const int2 q = seq_rows(a.cu_q, n, s, a.rows_q), k = seq_rows(a.cu_k, n, s, a.rows_k);
      cq = ceil_div(q.y - q.x, a.tok2);
      ck = ceil_div(k.y - k.x, kAttnKeys);
    }
    int total;
    const int eq = block_scan(cq, warp_sums, total);
    if (s <= n) scan_q[s] = nq + eq;
    nq += total;
    const int ek = block_scan(ck, warp_sums, total);
    if (s <= n) scan_k[s] = nk + ek;
    nk += total;
  }
  if (tid == 0) {
    scan_q[n + 1] = nq;
    scan_k[n + 1] = nk;
  }
  __syncthreads();
  unsigned long long mine = 0;
  for (int t = tid; t < nq; t += kPlanThreads) mine += (unsigned)query_item(a, scan_q, n, t).ke;
  atomicAdd(&blocks_total, mine);
  for (int i = tid; i < kBins; i += kPlanThreads) bins[i] = 0;
  __syncthreads();
  // a piece has at least this many blocks: half an SM's even share of all of them
  const unsigned long long share = (blocks_total * (unsigned)a.heads_kv + 2 * kAttnSMs - 1) / (2 * kAttnSMs);
  const int most = a.l.may_split ? (int)(share > kAttnMinBlocks ? share : kAttnMinBlocks) : 0x7fffffff;
  for (int t = tid; t < nq; t += kPlanThreads) {
    const int len = query_item(a, scan_q, n, t).ke;
    const int p = len > most ? ceil_div(len, most) : 1;
    const int each = ceil_div(len, p);
    for (int i = 0; i < p; ++i) atomicAdd(&bins[min(min(each, len - i * each), kBins - 1)], 1);
  }
  __syncthreads();
  int total;
  {
    const int b = kBins - 1 - tid;               // longest first
    const int e = block_scan(bins[b], warp_sums, total);
    __syncthreads();
    bins[b] = e;
  }
  __syncthreads();
  for (int t = tid; t < nq; t += kPlanThreads) {
    AttnItem it = query_item(a, scan_q, n, t);
    const int len = it.ke;
    const int p = len > most ? ceil_div(len, most) : 1;
    const int each = ceil_div(len, p);
    int slot = -1;
    if (p > 1) {
      slot = atomicAdd(&slots, p);
      join[atomicAdd(&joins, 1)] = AttnJoin{it.q0, it.qn, slot, p};
    }
    for (int i = 0; i < p; ++i) {
      it.kb = i * each;
      it.ke = min(len, it.kb + each);
      it.slot = slot < 0 ? -1 : slot + i;
      items[atomicAdd(&bins[min(it.ke - it.kb, kBins - 1)], 1)] = it;
    }
  }
  __syncthreads();
  const int n_items = total;
  for (int i = tid; i < kBins; i += kPlanThreads) bins[i] = 0;
  __syncthreads();
  // key items by the tokens that see them, in units of 128
  for (int t = tid; t < nk; t += kPlanThreads)
    atomicAdd(&bins[min(ceil_div(key_item_work(key_item(a, scan_k, n, t)), 128), kBins - 1)], 1);
  __syncthreads();
  {
    const int b = kBins - 1 - tid;
    const int e = block_scan(bins[b], warp_sums, total);
    __syncthreads();
    bins[b] = e;
  }
  __syncthreads();
  for (int t = tid; t < nk; t += kPlanThreads) {
    const AttnKeyItem it = key_item(a, scan_k, n, t);
    keys[atomicAdd(&bins[min(ceil_div(key_item_work(it), 128), kBins - 1)], 1)] = it;
  }
  if (tid == 0) {
    __threadfence_block();
    *hdr = AttnPlanHdr{n_items, nk, joins, 0};
  }
}

// ---------------------------------------------------------------------------
// forward: a warp per query row
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) attn_kernel(const AttnArgs a) {
  const AttnPlanHdr* hdr = reinterpret_cast<const AttnPlanHdr*>(a.plan);
  const AttnItem* items = reinterpret_cast<const AttnItem*>(a.plan + a.l.at_items);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = a.s.heads_kv, g = a.l.group, d = a.s.head_dim;
  const int slot_rows = (int)((a.s.rows_q < 2 * a.l.tok ? a.s.rows_q : 2 * a.l.tok) * g);
  if (a.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0) {
    a.status[0] = kOk;
    a.status[1] = -1;
  }
  float2* stat = static_cast<float2*>(a.workspace);
  float* part = reinterpret_cast<float*>(stat + a.l.cap_slots * hk * (int64_t)slot_rows);
  for (int w = blockIdx.x; w < hdr->n_items * hk; w += gridDim.x) {
    const AttnItem it = items[w / hk];
    const int kh = w % hk;
    for (int r = warp; r < it.qn * g; r += 8) {
      const int tok = r / g, head = kh * g + r % g;
      const int lim = a.s.causal ? min(it.kn, it.off + tok + 1) : it.kn;
      const T* q = static_cast<const T*>(a.q) + (int64_t)(it.q0 + tok) * a.q_stride + head * d;
      float fq[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) fq[i] = lane + 32 * i < d ? to_f32(q[lane + 32 * i]) * a.scale : 0.f;
      float m = -INFINITY, l = 0.f;
      for (int j = it.kb * kAttnKeys; j < min(lim, it.ke * kAttnKeys); ++j) {
        const T* k = static_cast<const T*>(a.k) + (int64_t)(it.k0 + j) * a.k_stride + kh * d;
        const T* v = static_cast<const T*>(a.v) + (int64_t)(it.k0 + j) * a.v_stride + kh * d;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < d) s = fmaf(fq[i], to_f32(k[lane + 32 * i]), s);
        s = warp_sum(s);
        const float mn = fmaxf(m, s);
        const float mz = mn == -INFINITY ? 0.f : mn;
        const float c = __expf(m - mz), p = __expf(s - mz);
        l = l * c + p;
        m = mn;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < d) o[i] = fmaf(o[i], c, p * to_f32(v[lane + 32 * i]));
      }
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const float lse = l > 0.f || l != l ? m + logf(l) : -INFINITY;
      if (it.slot < 0) {
        T* out = static_cast<T*>(a.out) + (int64_t)(it.q0 + tok) * a.out_stride + head * d;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < d) out[lane + 32 * i] = from_f32<T>(o[i] * inv);
        if (a.lse && lane == 0) a.lse[(int64_t)(it.q0 + tok) * a.s.heads_q + head] = lse;
      } else {
        const int64_t at = ((int64_t)it.slot * hk + kh) * slot_rows + r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < d) part[at * d + lane + 32 * i] = o[i] * inv;
        if (lane == 0) stat[at] = make_float2(m, l);
      }
    }
  }
}

// Joins the pieces of a cut item, in their order.  A piece holds its rows' maximum m, sum l and
// normalised output: out = sum of w_i out_i / sum of w_i, w_i = l_i exp(m_i - top).  (m and l
// stay apart: m + log l would lose l next to a large score.)  A warp per row.
template <typename T>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a) {
  const AttnPlanHdr* hdr = reinterpret_cast<const AttnPlanHdr*>(a.plan);
  const AttnJoin* joins = reinterpret_cast<const AttnJoin*>(a.plan + a.l.at_joins);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = a.s.heads_kv, g = a.l.group, d = a.s.head_dim;
  const int slot_rows = (int)((a.s.rows_q < 2 * a.l.tok ? a.s.rows_q : 2 * a.l.tok) * g);
  const float2* stat = static_cast<const float2*>(a.workspace);
  const float* part = reinterpret_cast<const float*>(stat + a.l.cap_slots * hk * (int64_t)slot_rows);
  for (int w = blockIdx.x; w < hdr->n_joins * hk; w += gridDim.x) {
    const AttnJoin jn = joins[w / hk];
    const int kh = w % hk;
    for (int r = warp; r < jn.qn * g; r += 8) {
      const int64_t at = ((int64_t)jn.slot * hk + kh) * slot_rows + r, step = (int64_t)hk * slot_rows;
      float top = -INFINITY;
      for (int p = 0; p < jn.pieces; ++p) top = fmaxf(top, stat[at + p * step].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
      for (int p = 0; p < jn.pieces; ++p) {
        const float2 ml = stat[at + p * step];
        if (ml.y == 0.f) continue;             // no key of this piece weighs anything (NaN goes on)
        const float wgt = ml.y * __expf(ml.x - ref);
        sum += wgt;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < d) o[i] = fmaf(wgt, part[(at + p * step) * d + lane + 32 * i], o[i]);
      }
      const int tok = r / g, head = kh * g + r % g;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      T* out = static_cast<T*>(a.out) + (int64_t)(jn.q0 + tok) * a.out_stride + head * d;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < d) out[lane + 32 * i] = from_f32<T>(o[i] * inv);
      if (a.lse && lane == 0)
        a.lse[(int64_t)(jn.q0 + tok) * a.s.heads_q + head] = sum == 0.f ? -INFINITY : ref + logf(sum);
    }
  }
}

template <typename T>
cudaError_t launch_typed(const AttnArgs& a, cudaStream_t st) {
  const int64_t work = a.l.cap_items * a.s.heads_kv;
  attn_kernel<T><<<(unsigned)(work < 1216 ? work : 1216), 256, 0, st>>>(a);
  if (a.l.may_split)
    attn_join_kernel<T><<<2 * kAttnSMs, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_plan(const vitfe_attention_shape& s, const int32_t* cu_q, const int32_t* cu_k,
                                  void* plan, int32_t* status, cudaStream_t st) {
  PlanArgs a;
  a.l = attn_layout(s);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.rows_q = (int)s.rows_q;
  a.rows_k = (int)s.rows_k;
  a.max_seqs = s.max_seqs;
  a.heads_kv = s.heads_kv;
  a.tok2 = 2 * a.l.tok;
  a.causal = s.causal;
  a.plan = static_cast<char*>(plan);
  a.status = status;
  attn_plan_kernel<<<1, kPlanThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t st) {
  if (a.s.rows_q == 0) return cudaSuccess;
  return a.s.dtype == VITFE_F16 ? launch_typed<__half>(a, st) : launch_typed<__nv_bfloat16>(a, st);
}

}  // namespace vitfe
