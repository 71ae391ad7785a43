// Rotary positions with several axes: the positions of a packed prompt, and their rotation of
// Q and K.
#include <cmath>

#include "vitfe_block.cuh"

namespace vitfe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSpans = VITFE_MAX_SPANS;
constexpr int kMaxPairs = VITFE_ROPE_MAX_HEAD_DIM / 2;

// ---------------------------------------------------------------------------
// positions
// ---------------------------------------------------------------------------
struct SpanScan {          // an inclusive scan's element: positions restart at a `first` span
  long long tokens;
  long long reach;         // positions since the last restart
  int restart;
};

__device__ __forceinline__ SpanScan scan_join(const SpanScan& a, const SpanScan& b) {
  return SpanScan{a.tokens + b.tokens, b.restart ? b.reach : a.reach + b.reach, a.restart | b.restart};
}

// A span is text, then a grid of t x h x w tokens (after merging) at position p = the text's end: token
// (tg, y, x) of it has (p + tg step, p + y, p + x), and the next span begins one past the largest
// position.  So a span's first position is a sum over those before it, back to the last restart: a
// scan.  Every block scans the span table (it is small) and then places its own tokens: one launch,
// no pass between the blocks.  Launch-bound: 5,000 rows take 3.7 us.
__global__ void __launch_bounds__(kThreads) mrope_positions_kernel(
    const vitfe_span* __restrict__ spans, const int32_t* __restrict__ n_spans, int max_spans,
    const vitfe_item* __restrict__ items, const int32_t* __restrict__ n_items, int max_items, int merge, int rows,
    int32_t* __restrict__ pos, int32_t* __restrict__ status) {
  __shared__ int start[kMaxSpans + 1];           // first token, clamped to rows
  __shared__ int base[kMaxSpans];                // position of the span's first token
  __shared__ int text[kMaxSpans], step[kMaxSpans], height[kMaxSpans], wide[kMaxSpans];
  __shared__ SpanScan warp_total[kThreads / 32];
  __shared__ unsigned first_bad;                 // (span << 4) | code of the first bad span
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = *n_spans;
  int code = kOk;
  if (n < 0 || n > max_spans) {
    code = kDesc;
    n = 0;
  }
  int ni = max_items > 0 ? *n_items : 0;
  if (ni < 0 || ni > max_items) {
    code = kDesc;
    n = 0;
  }
  if (tid == 0) first_bad = 0xffffffffu;
  __syncthreads();
  SpanScan carry{0, 0, 0};
  for (int b = 0; b < n; b += kThreads) {
    const int i = b + tid;
    SpanScan e{0, 0, 0};
    if (i < n) {
      const vitfe_span sp = spans[i];
      bool bad = sp.text < 0 || sp.item < -1 || sp.item >= ni || sp.step < 0 || sp.step > 65536;
      long long t = 0, h = 0, w = 0;
      if (!bad && sp.item >= 0) {
        t = items[sp.item].t;
        h = items[sp.item].h;
        w = items[sp.item].w;
        bad = t < 0 || h < 0 || w < 0 || h % merge || w % merge || (h > 0 && w > 0 && t * h > 0x7fffffffLL / w);
        h /= merge;
        w /= merge;
      }
      long long words = sp.text;
      if (bad) {
        t = h = w = words = 0;
        atomicMin(&first_bad, ((unsigned)i << 4) | (unsigned)kDesc);
      }
      const long long seen = t * h * w;
      long long reach = 0;
      if (seen > 0) {
        reach = (t - 1) * sp.step + 1;
        reach = reach > h ? reach : h;
        reach = reach > w ? reach : w;
      }
      text[i] = (int)words;
      step[i] = sp.step;
      height[i] = (int)(seen > 0 ? h : 0);
      wide[i] = (int)(seen > 0 ? w : 0);
      e = SpanScan{words + seen, words + reach, sp.first != 0};
    }
    const SpanScan own = e;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      SpanScan o;
      o.tokens = __shfl_up_sync(0xffffffffu, e.tokens, d);
      o.reach = __shfl_up_sync(0xffffffffu, e.reach, d);
      o.restart = __shfl_up_sync(0xffffffffu, e.restart, d);
      if (lane >= d) e = scan_join(o, e);
    }
    if (lane == 31) warp_total[warp] = e;
    __syncthreads();
    SpanScan before = carry;
    for (int w = 0; w < warp; ++w) before = scan_join(before, warp_total[w]);
    e = scan_join(before, e);
    for (int w = 0; w < kThreads / 32; ++w) carry = scan_join(carry, warp_total[w]);
    __syncthreads();
    if (i < n) {
      const long long at = e.tokens - own.tokens, p = e.reach - own.reach;
      start[i] = (int)(at < rows ? at : rows);
      base[i] = (int)(p < 0x7fffffffLL ? p : 0x7fffffffLL);
      if (e.tokens > rows || e.reach > 0x7fffffffLL) atomicMin(&first_bad, ((unsigned)i << 4) | (unsigned)kRange);
    }
  }
  if (tid == 0) start[n] = (int)(carry.tokens < rows ? carry.tokens : rows);
  __syncthreads();
  if (status != nullptr && blockIdx.x == 0 && tid == 0) {
    const bool bad = code == kOk && first_bad != 0xffffffffu;
    status[0] = bad ? (int)(first_bad & 15u) : code;
    status[1] = bad ? (int)(first_bad >> 4) : -1;
  }
  const int live = start[n];
  for (int r = blockIdx.x * kThreads + tid; r < rows; r += gridDim.x * kThreads) {
    long long p0 = -1, p1 = -1, p2 = -1;
    if (r < live) {
      const int s = find_item(start, n, r);
      const int local = r - start[s] - text[s];
      p0 = p1 = p2 = (long long)base[s] + (r - start[s]);
      if (local >= 0) {
        const int hw = height[s] * wide[s];
        const int tg = local / hw, rem = local - tg * hw;
        const int y = rem / wide[s], x = rem - y * wide[s];
        const long long p = (long long)base[s] + text[s];
        p0 = p + (long long)tg * step[s];
        p1 = p + y;
        p2 = p + x;
      }
    }
    pos[r] = (int)(p0 < 0x7fffffffLL ? p0 : 0x7fffffffLL);
    pos[(size_t)rows + r] = (int)(p1 < 0x7fffffffLL ? p1 : 0x7fffffffLL);
    pos[2 * (size_t)rows + r] = (int)(p2 < 0x7fffffffLL ? p2 : 0x7fffffffLL);
  }
}

// ---------------------------------------------------------------------------
// rotation
// ---------------------------------------------------------------------------
struct MropeTable {
  uint64_t turn[kMaxPairs];    // w_i / (2 pi) in units of 2^-64 turns, from 53-bit arithmetic
  uint8_t axis[kMaxPairs];
};

struct MropeKernelArgs {
  const int32_t* pos;
  int rows, half, head_dim, units_q, units, groups, rest, rows_per_block;
  float sign;
  const void* x[2];
  void* y[2];
  long long x_stride[2], y_stride[2];
};

// (a, b) -> (a cos - b sin, b cos + a sin) for elements i and i + half of each head; `sign` turns back.
// The angle of a pair is position * w_i.  In turns of 2^-64, position * turn[i] wraps as the
// angle does, so a position loses no more than it multiplies turn[i]'s own rounding by (2^-53 turns or
// less for theta >= 500: products of doubles); the phase's top 32 bits become an fp32 number of half
// turns, to 2^-25 of one.
// Memory bound (q and k, in and out).  A block makes the sines of its few rows once, in shared memory,
// for all their heads, while the first rows' elements are on their way.  bf16, 32 + 8 heads of 128:
// 16,384 rows 65 us, 5.2 TB/s, 76% of what a copy reaches; 65,536 rows 228 us, 87%; fp32, 16,384
// rows 94%.  Blocks of twice or half the rows: 69 and 68 us; four rows in flight a thread: 95 us, spilled.
template <typename X, int V>
__global__ void __launch_bounds__(kThreads, 4) mrope_kernel(const __grid_constant__ MropeKernelArgs a, const __grid_constant__ MropeTable tab) {
  extern __shared__ __align__(16) float cs[];    // [rows_per_block][2][half]; half is a multiple of 4
  const int r0 = blockIdx.x * a.rows_per_block;
  const int nr = min(a.rows_per_block, a.rows - r0);
  using XV = Vec<X, V>;
  constexpr int kRows = V == 8 ? 2 : 4;          // rows of a thread in flight
  // unit: (head, group of V pairs), then the copied tail of each head.  A thread keeps its unit over
  // the block's rows; with fewer units than threads, the threads share out the rows as well.
  const int threads = (int)blockDim.x, rot = a.half / V;
  const int lanes = a.units < threads ? a.units : threads, side = threads / lanes;
  const int r_first = threadIdx.x / lanes;
  int u = blockIdx.y * threads + threadIdx.x % lanes;
  if (r_first >= side) u = a.units;
  const X* x = nullptr;
  X* y = nullptr;
  long long xs = 0, ys = 0;
  int g = 0;
  bool turn = false;
  XV va[kRows], vb[kRows];
  auto place = [&]() {
    const int which = u >= a.units_q;
    const int v = u - (which ? a.units_q : 0), head = v / a.groups;
    g = v - head * a.groups;
    turn = g < rot;
    xs = a.x_stride[which];
    ys = a.y_stride[which];
    const int at = head * a.head_dim + (turn ? g * V : 2 * a.half + (g - rot) * V);
    x = static_cast<const X*>(a.x[which]) + r0 * xs + at;
    y = static_cast<X*>(a.y[which]) + r0 * ys + at;
  };
  auto fetch = [&](int r) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int rr = r + i * side;
      if (rr < nr) {
        va[i] = *reinterpret_cast<const XV*>(x + rr * xs);
        if (turn) vb[i] = *reinterpret_cast<const XV*>(x + rr * xs + a.half);
      }
    }
  };
  if (u < a.units) {                             // the first rows are on their way while the table is made
    place();
    fetch(r_first);
  }
  // Read as memory: as constants, the lanes' different entries are fetched one after the other (100,000
  // rows of 1 + 1 heads of 64: 63 us that way, 25 us this way; 16,384 rows of 32 + 8 heads of 128: 70, 65).
  const MropeTable* table = &tab;
  asm("" : "+l"(table));
  for (int i = threadIdx.x; i < nr * a.half; i += threads) {
    const int r = i / a.half, p = i - r * a.half;
    const int64_t at = a.pos[(size_t)table->axis[p] * a.rows + r0 + r];
    const uint64_t phase = (uint64_t)at * table->turn[p];
    const float half_turns = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;   // 2^-31
    float sn, c;
    sincospif(half_turns, &sn, &c);
    cs[(2 * r) * a.half + p] = c;
    cs[(2 * r + 1) * a.half + p] = sn * a.sign;
  }
  __syncthreads();
  for (bool first = true; u < a.units; u += gridDim.y * threads) {
    if (!first) place();
    for (int r = r_first; r < nr; r += kRows * side) {
      if (!first) fetch(r);
      first = false;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int rr = r + i * side;
        if (rr >= nr) break;
        if (turn) {
          const float4* c = reinterpret_cast<const float4*>(cs + 2 * rr * a.half + g * V);
          const float4* s = reinterpret_cast<const float4*>(cs + (2 * rr + 1) * a.half + g * V);
          XV ya, yb;
#pragma unroll
          for (int q = 0; q < V; q += 4) {
            const float4 c4 = c[q / 4], s4 = s[q / 4];
            const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float fa = to_f32(va[i].v[q + e]), fb = to_f32(vb[i].v[q + e]);
              ya.v[q + e] = from_f32<X>(fmaf(fa, cc[e], -(fb * ss[e])));
              yb.v[q + e] = from_f32<X>(fmaf(fb, cc[e], fa * ss[e]));
            }
          }
          *reinterpret_cast<XV*>(y + rr * ys) = ya;
          *reinterpret_cast<XV*>(y + rr * ys + a.half) = yb;
        } else {
          *reinterpret_cast<XV*>(y + rr * ys) = va[i];
        }
      }
    }
  }
}

template <typename X, int V>
cudaError_t launch_typed(const MropeArgs& a, const MropeTable& tab, cudaStream_t s) {
  MropeKernelArgs k;
  k.pos = a.pos;
  k.rows = (int)a.rows;
  k.half = a.rotary_dim / 2;
  k.head_dim = a.head_dim;
  bool moved = false;            // the tail of a head is copied only where out is elsewhere
  for (int i = 0; i < 2; ++i) {
    k.x[i] = a.x[i];
    k.y[i] = a.y[i];
    k.x_stride[i] = a.x_stride[i];
    k.y_stride[i] = a.y_stride[i];
    moved = moved || (a.heads[i] > 0 && a.x[i] != a.y[i]);
  }
  k.rest = moved ? (a.head_dim - a.rotary_dim) / V : 0;
  k.groups = k.half / V + k.rest;
  k.units_q = a.heads[0] * k.groups;
  k.units = (a.heads[0] + a.heads[1]) * k.groups;
  k.sign = a.inverse ? -1.f : 1.f;
  if (k.units == 0) return cudaSuccess;
  // as many threads as share the units (or the rows, where there are few units) out evenly; four rows
  // to a thread, as far as the block's table of sines (32 KB) reaches; few rows: one to a block and
  // its heads over grid.y, so that more SMs take part
  const int passes = (k.units + kThreads - 1) / kThreads, side = passes > 1 ? 1 : kThreads / k.units;
  const int threads = ((k.units * side + passes - 1) / passes + 31) / 32 * 32;
  const int room = 8192 / (2 * k.half);
  int per = 4 * side < room ? 4 * side : room, ysplit = 1;
  if (a.rows < 2 * 152) {
    per = 1;
    ysplit = (k.units + threads - 1) / threads;
    ysplit = ysplit > 16 ? 16 : ysplit;
  }
  k.rows_per_block = per;
  const dim3 grid((unsigned)((a.rows + per - 1) / per), (unsigned)ysplit);
  mrope_kernel<X, V><<<grid, threads, (size_t)per * 2 * k.half * sizeof(float), s>>>(k, tab);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mrope_apply(const MropeArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  MropeTable tab{};
  const int half = a.rotary_dim / 2;
  const double ratio = std::pow((double)a.theta, -2.0 / a.rotary_dim);
  double w = 0.15915494309189535;               // 1 / (2 pi)
  for (int i = 0; i < half; ++i) {
    // turns below 1; the whole part of a larger frequency (theta < 1) turns nothing
    tab.turn[i] = (uint64_t)std::ldexp(w - std::floor(w), 64);
    tab.axis[i] = a.axis_of_pair[i];
    w *= ratio;
  }
  // 8 elements (16 bytes) of a 16-bit type where halves, heads, rows and bases allow it, else 4
  bool wide = a.dtype != VITFE_F32 && half % 8 == 0;
  for (int i = 0; i < 2; ++i)
    if (a.heads[i] > 0)
      wide = wide && reinterpret_cast<uintptr_t>(a.x[i]) % 16 == 0 && reinterpret_cast<uintptr_t>(a.y[i]) % 16 == 0 &&
             a.x_stride[i] % 8 == 0 && a.y_stride[i] % 8 == 0;
  switch (a.dtype) {
    case VITFE_BF16:
      return wide ? launch_typed<__nv_bfloat16, 8>(a, tab, s) : launch_typed<__nv_bfloat16, 4>(a, tab, s);
    case VITFE_F16: return wide ? launch_typed<__half, 8>(a, tab, s) : launch_typed<__half, 4>(a, tab, s);
    default: return launch_typed<float, 4>(a, tab, s);
  }
}

cudaError_t launch_mrope_positions(const vitfe_span* spans, const int32_t* n_spans, int max_spans,
                                   const vitfe_item* items, const int32_t* n_items, int max_items, int merge,
                                   int64_t rows, int32_t* pos, int32_t* status, cudaStream_t s) {
  int64_t blocks = (rows + kThreads - 1) / kThreads;
  blocks = blocks < 1 ? 1 : blocks > 608 ? 608 : blocks;
  mrope_positions_kernel<<<(unsigned)blocks, kThreads, 0, s>>>(spans, n_spans, max_spans, items, n_items, max_items,
                                                               merge, (int)rows, pos, status);
  return cudaGetLastError();
}

}  // namespace vitfe
