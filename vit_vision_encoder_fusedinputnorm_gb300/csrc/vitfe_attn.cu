// Attention over packed sequences: the plan and the forward pass.
#include "vitfe_attn.cuh"

namespace vitfe {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;

struct PlanArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int rows_q, rows_k, max_seqs, heads_kv, group, item_tok, causal;
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
  const int first = (t - scan[s]) * a.item_tok;
  it.q0 = q.x + first;
  it.qn = min(a.item_tok, q.y - it.q0);
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

// One block, since it is all latency (a dozen passes with a barrier each: 8 us for one sequence, 12 for
// eight, 17 for 64 caches) and a plan serves every layer of a model.  It checks the boundaries, lists the
// query and key items of every sequence, cuts long key ranges where there are few items, and sorts by
// length, longest first, for the attention kernels' fixed deal of items to SMs.  Query items come out
// even that way, as those longer than an SM's share are cut; key items are not cut, and few long ones
// do not (eight stills: 397 steps on the fullest SM, 386 on average; causal prompts up to 4100 rows with
// four key heads: 131 and 89.5).  The order among equal lengths may vary from call to call; no result
// depends on it.
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(PlanArgs a) {
  __shared__ int warp_sums[32];
  __shared__ int bins[kBins];
  __shared__ unsigned bad;
  __shared__ unsigned long long blocks_total;
  __shared__ int slots[2], joins;            // of items of many and of few rows
  __shared__ int live;                       // sequences with tokens
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
    slots[0] = joins = live = 0;
    slots[1] = (int)a.l.cap_many;
  }
  __syncthreads();
  int n = a.max_seqs;
  for (int s = tid; s < n; s += kPlanThreads) {
    const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
    if (q1 > q0) atomicAdd(&live, 1);
    if ((s == 0 && (q0 != 0 || k0 != 0)) || q0 < 0 || k0 < 0 || q1 < q0 || k1 < k0 || q1 > a.rows_q || k1 > a.rows_k) atomicMin(&bad, (unsigned)s);
  }
  __syncthreads();
  if (a.status != nullptr && tid == 0) {
    a.status[0] = bad == 0xffffffffu ? kOk : kDesc;
    a.status[1] = bad == 0xffffffffu ? -1 : (int)bad;
  }
  if (bad != 0xffffffffu) n = 0;
  // Two tiles share an item's keys.  Where the sequences have no more tokens than one tile on average
  // (single tokens above all), the second one would stay empty: an item is one tile then, and the
  // kernel works on two items at a time.  bf16, the two-tile item's time first: the 64-token batch below
  // 200 -> 164 us, windows of 64 tokens 417 -> 270 us, one token over 32,768 keys 45.5 -> 40 us; but a
  // sequence of 16,384 715 -> 888 us.
  const bool single = a.l.may_single && n > 0 && a.cu_q[n] <= (long long)live * a.l.tok;
  a.item_tok = (single ? 1 : 2) * a.l.tok;
  int nq = 0, nk = 0;
  for (int b = 0; b <= n; b += kPlanThreads) {
    const int s = b + tid;
    int cq = 0, ck = 0;
    if (s <= n) {
      const int2 q = seq_rows(a.cu_q, n, s, a.rows_q), k = seq_rows(a.cu_k, n, s, a.rows_k);
      cq = ceil_div(q.y - q.x, a.item_tok);
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
  // Items longer than an SM's even share of all blocks are cut: they would be the last to end.  Few rows
  // (single tokens) are cut to a fourth of it, which is half of what each of an SM's two tiles gets, for
  // the evenness (64 tokens over 1..32,768 keys, 8 over 8,192: a half 163/77 us, a third 156/63, a fourth
  // 159/60, a sixth 164/68, a twelfth 183/77).  Joining their pieces costs next to nothing, where for
  // whole tiles it took as long as it saved (71 us beside 107 us, packed prompts up to 4100 rows).
  const unsigned long long all_blocks = blocks_total * (unsigned)a.heads_kv;
  auto pieces_of = [&](const AttnItem& it) {
    if (!a.l.may_split) return 1;
    const unsigned parts = it.qn * a.group <= kAttnFewRows ? kAttnFewCuts * kAttnSMs : kAttnSMs;
    const unsigned long long fair = (all_blocks + parts - 1) / parts;
    const int most = (int)(fair > kAttnMinBlocks ? fair : kAttnMinBlocks);
    return it.ke > most ? ceil_div(it.ke, most) : 1;
  };
  for (int t = tid; t < nq; t += kPlanThreads) {
    const AttnItem it = query_item(a, scan_q, n, t);
    const int len = it.ke, p = pieces_of(it);
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
    const int len = it.ke, p = pieces_of(it);
    const int each = ceil_div(len, p);
    int slot = -1;
    if (p > 1) {
      slot = atomicAdd(&slots[it.qn * a.group <= kAttnFewRows], p);
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
    *hdr = AttnPlanHdr{n_items, nk, joins, single ? 1 : 2};
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// s = scale q.k over the keys that a row sees, p = exp(s - m) with a reference m of the row's, l = sum p,
// out = (sum p v) / l, lse = m + log l; no key: 0 and -inf.  (Any m gives the same quotient; it only has
// to keep p in range.)  One pass over the keys: a block whose
// largest score exceeds m by more than 8 (in powers of 2) moves m, and what has been summed is scaled;
// below that p is at most 2^8, which fp32 sums and 16-bit p hold as well as 1.  s, p's sum and out's sums
// are fp32; p is rounded to the tensors' type, as the tensor core takes it.
//
// One CTA per SM works through (item, key head) pairs.  An item has up to two score tiles of 128
// rows (rows = tokens x the query heads of the key head, token-major), so that the tensor core
// runs one tile's products while the other tile's probabilities are computed.  Heads of 128 come
// near the tensor core's rate; below that a block's products are shorter than the way from scores to
// probabilities and back (some 1400 cycles of each tile), which two tiles hide in part.  bf16: four
// sequences of 9216, 16 heads of 80, 1.62 ms, 1.07 PFLOP/s, 55% of a dense product's rate; two of 8192,
// 16 heads of 128, 0.73 ms, 78%; 16,384 causal, 0.71 ms, 80%; 64 tokens over 1..32,768 keys, 8 key heads
// of 128, 159 us, 5.6 TB/s, 83% of what a copy reaches.
//   warps 0-3, 4-7: softmax of tile 0, 1: thread = row.  Reads S from tensor memory, keeps the
//     running maximum and sum in registers, writes P (16-bit) over S, rescales O when its
//     reference maximum has to move, and stores the finished rows.
//   warp 8: TMA loads of Q tiles and of the ring of K and V blocks.
//   warp 9: the matrix instructions: S_t = Q_t K^T, O_t += P_t V.
// Tensor memory: S0, S1 (128 columns each; P_t in the first 64 of them), O0, O1 (128 each).
__global__ void status_ok_kernel(int32_t* status) {
  status[0] = kOk;
  status[1] = -1;
}

constexpr int kFwdThreads = 384;
// Registers a thread: the launch's, then the softmax warpgroups' and the third's.  The shares have to
// add up to what the block was launched with, or the increase would wait for ever.
constexpr int kFwdRegs = 168, kSoftRegs = 208, kIssueRegs = 88;
static_assert(2 * kSoftRegs + kIssueRegs <= 3 * kFwdRegs, "");
constexpr int kMaxStages = 10;
constexpr int kSmemMax = 227 * 1024;

struct FwdShared {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int abort;
};

// Key blocks [kb, kb + n) that tile t of an item reads (0: the tile has no row that sees a key).
__device__ __forceinline__ int tile_blocks(const AttnItem& it, int t, int tok, bool causal) {
  const int have = min(tok, it.qn - t * tok);
  if (have <= 0) return 0;
  const int last = causal ? min(it.kn, max(0, it.off + t * tok + have)) : it.kn;
  return max(0, min(it.ke, ceil_div(last, kAttnKeys)) - it.kb);
}

// The w-th work of worker `id` of n: the list is sorted longest first and dealt back and forth, which
// keeps the workers' sums together.
__device__ __forceinline__ int deal(int round, int id, int n) { return round * n + ((round & 1) ? n - 1 - id : id); }

// The blocks of a worker's works, one after the other (works without any are passed over).
struct WorkStream {
  AttnItem it;
  int kh, n, j, round;
  bool live;
};
__device__ __forceinline__ void next_work(WorkStream& s, const AttnItem* items, int works, int hk, int id, int workers,
                                          int tok, bool causal) {
  s.live = false;
  s.j = 0;
  for (;;) {
    const int w = deal(++s.round, id, workers);
    if (w >= works) return;
    s.it = items[w / hk];
    s.kh = w % hk;
    s.n = tile_blocks(s.it, 0, tok, causal);
    if (s.n > 0) break;
  }
  s.live = true;
}

// kSingle: items of one tile (AttnPlanHdr::tiles), and each of the two tiles works through items of its own.
template <typename T, bool kSingle>
__device__ __forceinline__ void attn_body(const AttnArgs& a, const CUtensorMap& map_q, const CUtensorMap& map_k,
                                          const CUtensorMap& map_v, int stages, uint8_t* raw, FwdShared& sh) {
  const uint32_t tiles = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = a.s.heads_kv, g = a.l.group, d = a.s.head_dim, tok = a.l.tok;
  const bool causal = a.s.causal != 0;
  const int nb = (d + kColBlock - 1) / kColBlock;            // column blocks of a head
  const uint32_t tile_bytes = (uint32_t)nb * kColBlockBytes;
  const uint32_t ring = tiles + 2 * tile_bytes;
  volatile int* abort_flag = &sh.abort;
  if (threadIdx.x == 0) {
    if (a.status != nullptr && blockIdx.x == 0) {      // a wait that runs out overrides it later
      a.status[0] = kOk;
      a.status[1] = -1;
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&sh.q_full[t]), 1);
      mbar_init(smem_u32(&sh.q_empty[t]), 1);
      mbar_init(smem_u32(&sh.s_full[t]), 1);
      mbar_init(smem_u32(&sh.p_full[t]), 4);
      mbar_init(smem_u32(&sh.o_full[t]), 1);
    }
    for (int i = 0; i < stages; ++i) {
      mbar_init(smem_u32(&sh.kv_full[i]), 1);
      mbar_init(smem_u32(&sh.kv_empty[i]), 1);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  grid_dep_trigger();      // the join may be set up meanwhile (it waits for the end)
  const uint32_t tmem = sh.tmem;
  const AttnPlanHdr* hdr = reinterpret_cast<const AttnPlanHdr*>(a.plan);
  const AttnItem* items = reinterpret_cast<const AttnItem*>(a.plan + a.l.at_items);
  const int works = hdr->n_items * hk, workers = (kSingle ? 2 : 1) * (int)gridDim.x;
  // (neighbours in the list are key heads of the same rows: an SM's two tiles read them together)
  auto worker = [&](int t) { return kSingle ? 2 * (int)blockIdx.x + t : (int)blockIdx.x; };

  if (warp < 8) {
    // ------------------------------------------------------------- softmax and output
    more_registers<kSoftRegs>();
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + (uint32_t)t * 128u;
    const uint32_t o_col = tmem + lanes + 256u + (uint32_t)t * 128u;
    const int tile = kSingle ? 0 : t, id = worker(t);
    const int my_tok = tile * tok + row / g, head_in = row % g;
    const float scale2 = a.scale * 1.4426950408889634f;      // exponents of 2
    const AttnSlots slots(a.s, a.l);
    float2* stat = static_cast<float2*>(a.workspace);
    float* part = reinterpret_cast<float*>(stat + slots.rows(a.l));
    uint32_t ns = 0, no = 0;                                 // phases of s_full, o_full
    bool ok = true;
    for (int r = 0, w = deal(0, id, workers); ok && w < works; w = deal(++r, id, workers)) {
      const AttnItem it = items[w / hk];
      const int kh = w % hk;
      if (it.qn <= tile * tok) continue;
      const int n = tile_blocks(it, tile, tok, causal);
      const bool live = row < tok * g && my_tok < it.qn;
      int lim = causal ? min(it.kn, it.off + my_tok + 1) : it.kn;   // keys that the row sees
      if (!live) lim = 0;
      float m = -INFINITY, l = 0.f;                          // m: the reference of the exponents
      for (int j = 0; j < n; ++j, ++ns) {
        if (!wait_inline(&sh.s_full[t], ns & 1u, abort_flag, a.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(s_col + 32u * c, sr[c]);
        tmem_wait_ld();
        const int left = lim - (it.kb + j) * kAttnKeys;
        if (__any_sync(0xffffffffu, left < kAttnKeys)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e >= left) sr[c][e] = 0xff800000u;   // -inf: weighs 0, whatever was there
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; e += 2)
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = max3(mx[c], __uint_as_float(sr[c][e]), __uint_as_float(sr[c][e + 1]));
        const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], m);
        // The exponents' reference moves only when the maximum has outgrown it by 2^8: until then
        // P is at most 2^8 and the fp32 sums hold it exactly as well, and O need not be touched.
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, (top - m) * scale2 > 8.0f)) {
          const float f = top == -INFINITY ? 1.f : exp2_approx((m - top) * scale2);
          m = top;
          l *= f;
          // s_full of this block also says that the product before it is in O
          for (int c = 0; c < d; c += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(o_col + (uint32_t)c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st_32x32b_x16(o_col + (uint32_t)c, o);
          }
        }
        const float neg = m == -INFINITY ? 0.f : -(m * scale2);
        const uint64_t sc = f32x2(scale2, scale2), off = f32x2(neg, neg);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t x = fma_f32x2(f32x2(__uint_as_float(sr[c][e]), __uint_as_float(sr[c][e + 1])), sc, off);
            const float p0 = exp2_approx(lo_f32(x)), p1 = exp2_approx(hi_f32(x));
            sum[(e >> 1) & 1] = add_f32x2(sum[(e >> 1) & 1], f32x2(p0, p1));
            // the row sums are of the unrounded p; P is rounded for the product, as its type asks
            sr[c][e >> 1] = pack2<T>(p0, p1);
          }
          tmem_st_32x32b_x16(s_col + 16u * c, sr[c]);
        }
        const uint64_t both = add_f32x2(sum[0], sum[1]);
        l += lo_f32(both) + hi_f32(both);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[t]));
      }
      if (!ok) break;
      if (n > 0) {
        if (!wait_inline(&sh.o_full[t], no & 1u, abort_flag, a.wait_ns)) {
          ok = false;
          break;
        }
        ++no;
        tc_fence_after();
      }
      const float m2 = m == -INFINITY ? -INFINITY : m * scale2;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int head = kh * g + head_in;
      const int64_t qrow = (int64_t)it.q0 + my_tok;
      const int64_t at = slots.at(max(it.slot, 0), kh) + my_tok * g + head_in;
      for (int c = 0; c < d; c += 16) {
        uint32_t o[16];
        if (n > 0) {
          tmem_ld_32x32b_x16(o_col + (uint32_t)c, o);
          tmem_wait_ld();
        }
        float f[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = l == 0.f ? 0.f : __uint_as_float(o[e]) * inv;
        if (!live) continue;
        if (it.slot < 0) {
          T* out = static_cast<T*>(a.out) + qrow * a.out_stride + head * d + c;
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            if (c + e < d)
              *reinterpret_cast<uint4*>(out + e) = make_uint4(pack2<T>(f[e], f[e + 1]), pack2<T>(f[e + 2], f[e + 3]),
                                                              pack2<T>(f[e + 4], f[e + 5]), pack2<T>(f[e + 6], f[e + 7]));
        } else {
          float* out = part + at * d + c;
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            if (c + e < d) *reinterpret_cast<float4*>(out + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
      }
      tc_fence_before();
      if (live) {
        if (it.slot >= 0) stat[at] = make_float2(m2, l);
        else if (a.lse) a.lse[qrow * a.s.heads_q + head] = l == 0.f ? -INFINITY : (m2 + log2f(l)) * 0.6931471805599453f;
      }
    }
  } else {
    fewer_registers<kIssueRegs>();
  }
  if (warp == 8) {
    // ------------------------------------------------------------- loads
    if (lane == 0 && !a.stall) {
      uint32_t nq[2] = {0, 0}, nk = 0;
      RingPos pos;
      bool ok = true;
      const uint32_t q_bytes = (uint32_t)(nb * tok * g) * 128u;
      auto load = [&](const CUtensorMap* map, int head, int key) {
        const uint32_t st = pos.i;
        if (!mbar_wait(smem_u32(&sh.kv_empty[st]), pos.parity ^ 1u, abort_flag, a.wait_ns)) return false;
        pos = pos.next((uint32_t)stages);
        const uint32_t bar = smem_u32(&sh.kv_full[st]);
        mbar_arrive_expect_tx(bar, tile_bytes);
        for (int b = 0; b < nb; ++b)
          tma_load_3d(ring + st * tile_bytes + (uint32_t)b * kColBlockBytes, map, bar, b * kColBlock, head, key);
        ++nk;
        return true;
      };
      auto load_q = [&](const AttnItem& it, int kh, int t) {
        const uint32_t bar = smem_u32(&sh.q_full[t]);
        if (!mbar_wait(smem_u32(&sh.q_empty[t]), (nq[t] & 1u) ^ 1u, abort_flag, a.wait_ns)) return false;
        mbar_arrive_expect_tx(bar, q_bytes);
        for (int b = 0; b < nb; ++b)
          tma_load_3d(tiles + (uint32_t)t * tile_bytes + (uint32_t)b * kColBlockBytes, &map_q, bar, b * kColBlock,
                      kh * g, it.q0 + (kSingle ? 0 : t * tok));
        ++nq[t];
        return true;
      };
      if constexpr (kSingle) {
        WorkStream s[2];
        auto begin = [&](int t) {      // the next work's Q and first K
          next_work(s[t], items, works, hk, worker(t), workers, tok, causal);
          if (s[t].live) ok = load_q(s[t].it, s[t].kh, t) && load(&map_k, s[t].kh, s[t].it.k0 + s[t].it.kb * kAttnKeys);
        };
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          s[t].round = -1;
          if (ok) begin(t);
        }
        while (ok && (s[0].live || s[1].live)) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || !s[t].live) continue;
            const int key = s[t].it.k0 + (s[t].it.kb + s[t].j) * kAttnKeys;
            ok = load(&map_v, s[t].kh, key);
            if (!ok) continue;
            if (++s[t].j < s[t].n) ok = load(&map_k, s[t].kh, key + kAttnKeys);
            else begin(t);
          }
        }
      }
      for (int r = 0, w = deal(0, blockIdx.x, workers); !kSingle && ok && w < works; w = deal(++r, blockIdx.x, workers)) {
        const AttnItem it = items[w / hk];
        const int kh = w % hk;
        const int n0 = tile_blocks(it, 0, tok, causal), n1 = tile_blocks(it, 1, tok, causal);
        const int n = max(n0, n1);
        if (n0 > 0) ok = load_q(it, kh, 0);
        if (ok && n > 0) ok = load(&map_k, kh, it.k0 + it.kb * kAttnKeys);
        if (ok && n1 > 0) ok = load_q(it, kh, 1);
        for (int j = 0; ok && j < n; ++j) {
          ok = load(&map_v, kh, it.k0 + (it.kb + j) * kAttnKeys);
          if (ok && j + 1 < n) ok = load(&map_k, kh, it.k0 + (it.kb + j + 1) * kAttnKeys);
        }
      }
      if (*abort_flag) {
        // this warp's last loads land on their own; wait for them before the CTA ends
        const uint64_t t0 = global_timer_ns();
        for (int t = 0; t < 2; ++t)
          while (nq[t] > 0 && !mbar_try_wait(smem_u32(&sh.q_full[t]), (nq[t] - 1) & 1u) &&
                 global_timer_ns() - t0 < kAttnDrainNs) {
          }
        const uint32_t back = nk < (uint32_t)stages ? nk : (uint32_t)stages;
        for (uint32_t i = nk - back; i < nk; ++i)
          while (!mbar_try_wait(smem_u32(&sh.kv_full[i % (uint32_t)stages]), (i / (uint32_t)stages) & 1u) &&
                 global_timer_ns() - t0 < kAttnDrainNs) {
          }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------- matrix instructions
    const uint32_t id_s = idesc_16<T>(128, kAttnKeys, false);
    const uint32_t id_o = idesc_16<T>(128, (d + 15) / 16 * 16, true);
    const int ksteps = (d + 15) / 16;
    const uint64_t q_desc = sw128_desc(tiles), k_desc = sw128_desc(ring), v_desc = sw128_desc_rows(ring);
    const uint64_t tile_step = (uint64_t)(tile_bytes >> 4);
    const uint32_t nst = (uint32_t)stages;
    uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
    RingPos kp, vp = kp.next(nst);                // the next K and V tile: K0 V0 K1 V1 ...
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && wait_inline(bar, parity, abort_flag, a.wait_ns);
      return ok;
    };
    // S_t = Q_t K^T, announced on s_full; then `also` and `release`, when given
    auto scores = [&](int t, uint32_t st, uint64_t* also, uint64_t* release) {
      if (elect_one()) {
        issue_scores(tmem + (uint32_t)t * 128u, q_desc + (uint64_t)t * tile_step, k_desc + st * tile_step, id_s, ksteps);
        umma_commit(smem_u32(&sh.s_full[t]));
        if (also) umma_commit(smem_u32(also));
        if (release) umma_commit(smem_u32(release));
      }
      __syncwarp();
    };
    auto output = [&](int t, uint32_t st, bool first, uint64_t* also, uint64_t* release) {      // O_t (+)= P_t V
      if (elect_one()) {
        issue_sum<128>(tmem + 256u + (uint32_t)t * 128u, tmem + (uint32_t)t * 128u, v_desc + st * tile_step, id_o, !first);
        if (also) umma_commit(smem_u32(also));
        if (release) umma_commit(smem_u32(release));
      }
      __syncwarp();
    };
    if constexpr (kSingle) {
      // tiles in the order that the loads come in: K0 of each, then V(j) and the next K of each in turn
      WorkStream s[2];
      RingPos pos;
      auto begin = [&](int t) {
        next_work(s[t], items, works, hk, worker(t), workers, tok, causal);
        s[t].n = uniform(s[t].n);
        s[t].live = uniform(s[t].live) != 0;
        if (s[t].live) {
          wait(&sh.q_full[t], nq[t]++ & 1u);
          tc_fence_after();
        }
      };
      auto next_scores = [&](int t) {
        if (!ok || !s[t].live) return;
        const RingPos k = pos;
        pos = pos.next(nst);
        if (wait(&sh.kv_full[k.i], k.parity))
          scores(t, k.i, s[t].j + 1 == s[t].n ? &sh.q_empty[t] : nullptr, &sh.kv_empty[k.i]);
      };
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t].round = -1;
        begin(t);
        next_scores(t);
      }
      while (ok && (s[0].live || s[1].live)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || !s[t].live) continue;
          const RingPos v = pos;
          pos = pos.next(nst);
          if (!wait(&sh.kv_full[v.i], v.parity)) continue;
          const int have = uniform(s[t].it.kn - (s[t].it.kb + s[t].j) * kAttnKeys);      // as below
          if (have < kAttnKeys) zero_tile_rows(ring + v.i * tile_bytes, nb, have);
          if (!wait(&sh.p_full[t], np[t]++ & 1u)) continue;
          tc_fence_after();
          const bool last = s[t].j + 1 == s[t].n;
          output(t, v.i, s[t].j == 0, last ? &sh.o_full[t] : nullptr, &sh.kv_empty[v.i]);
          if (last) begin(t);
          else ++s[t].j;
          next_scores(t);
        }
      }
    }
    for (int r = 0, w = deal(0, blockIdx.x, workers); !kSingle && ok && w < works; w = deal(++r, blockIdx.x, workers)) {
      const AttnItem it = items[w / hk];
      const int n0 = uniform(tile_blocks(it, 0, tok, causal)), n1 = uniform(tile_blocks(it, 1, tok, causal));
      const int n = max(n0, n1), keys = uniform(it.kn - it.kb * kAttnKeys);
      if (n == 0) continue;
      if (!wait(&sh.kv_full[kp.i], kp.parity)) break;
      if (n0 > 0) {
        if (!wait(&sh.q_full[0], nq[0]++ & 1u)) break;
        scores(0, kp.i, n0 == 1 ? &sh.q_empty[0] : nullptr, n1 == 0 ? &sh.kv_empty[kp.i] : nullptr);
      }
      if (n1 > 0) {
        if (!wait(&sh.q_full[1], nq[1]++ & 1u)) break;
        scores(1, kp.i, n1 == 1 ? &sh.q_empty[1] : nullptr, &sh.kv_empty[kp.i]);
      }
      for (int j = 0; j < n; ++j) {
        const RingPos kn = vp.next(nst), vn = kn.next(nst);      // K(j + 1), V(j + 1)
        const bool more = j + 1 < n;
        bool v_here = false, k_here = false;
        // which tile is the last to read V(j), K(j + 1)
        const bool v_last1 = j < n1, k_last1 = j + 1 < n1;
        auto v_wait = [&]() {
          if (v_here) return true;
          if (!wait(&sh.kv_full[vp.i], vp.parity)) return false;
          const int have = keys - j * kAttnKeys;        // rows past the sequence's end weigh 0 in P,
          if (have < kAttnKeys) zero_tile_rows(ring + vp.i * tile_bytes, nb, have);   // but 0 * NaN is NaN
          return v_here = true;
        };
        auto k_wait = [&]() { return k_here || (k_here = wait(&sh.kv_full[kn.i], kn.parity)); };
        if (j < n0) {
          if (!wait(&sh.p_full[0], np[0]++ & 1u) || !v_wait()) break;
          tc_fence_after();
          output(0, vp.i, j == 0, j + 1 == n0 ? &sh.o_full[0] : nullptr, v_last1 ? nullptr : &sh.kv_empty[vp.i]);
          if (j + 1 < n0) {
            if (!k_wait()) break;
            scores(0, kn.i, j + 2 == n0 ? &sh.q_empty[0] : nullptr, k_last1 ? nullptr : &sh.kv_empty[kn.i]);
          }
        }
        if (j < n1) {
          if (!wait(&sh.p_full[1], np[1]++ & 1u) || !v_wait()) break;
          tc_fence_after();
          output(1, vp.i, j == 0, j + 1 == n1 ? &sh.o_full[1] : nullptr, &sh.kv_empty[vp.i]);
          if (j + 1 < n1) {
            if (!k_wait()) break;
            scores(1, kn.i, j + 2 == n1 ? &sh.q_empty[1] : nullptr, &sh.kv_empty[kn.i]);
          }
        }
        if (more) {
          kp = kn;
          vp = vn;
        }
      }
      if (!ok) break;
      kp = vp.next(nst);
      vp = kp.next(nst);
    }
    if (!ok) {      // matrix instructions in flight end on their own: wait for them
      if (elect_one()) umma_commit(smem_u32(&sh.drain));
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(smem_u32(&sh.drain), 0) && global_timer_ns() - t0 < kAttnDrainNs) {
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (sh.abort) {
    if (threadIdx.x == 0 && a.status != nullptr) {
      a.status[0] = kTimeout;
      a.status[1] = -1;
    }
    const AttnSlots slots(a.s, a.l);
    for (int t = 0; t < (kSingle ? 2 : 1); ++t) {
      for (int r = 0, w = deal(0, worker(t), workers); w < works; w = deal(++r, worker(t), workers)) {
        const AttnItem it = items[w / hk];
        const int kh = w % hk;
        if (it.slot >= 0) {       // (a piece's sum: the join makes the rows of it)
          fill_nan(static_cast<float*>(a.workspace) + 2 * slots.at(it.slot, kh), it.qn * g, 2, 2);
        } else {
          fill_nan(static_cast<T*>(a.out) + (int64_t)it.q0 * a.out_stride + kh * g * d, it.qn, a.out_stride, g * d);
          if (a.lse) fill_nan(a.lse + (int64_t)it.q0 * a.s.heads_q + kh * g, it.qn, a.s.heads_q, g);
        }
      }
    }
  }
}

// kMaySingle: the shape allows items of one tile, and the plan says whether they are.  (Both ways in one
// kernel cost the two-tile one 2.5%, so shapes that need only that have a kernel of their own.)
template <typename T, bool kMaySingle>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attn_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, int stages) {
  extern __shared__ uint8_t raw[];
  __shared__ FwdShared sh;
  if constexpr (kMaySingle) {
    if (reinterpret_cast<const AttnPlanHdr*>(a.plan)->tiles == 1) {
      attn_body<T, true>(a, map_q, map_k, map_v, stages, raw, sh);
      return;
    }
  }
  attn_body<T, false>(a, map_q, map_k, map_v, stages, raw, sh);
}

// Joins the pieces of a cut item, in their order.  A piece holds its rows' maximum m (as an
// exponent of 2), sum l and normalised output: out = sum of w_i out_i / sum of w_i,
// w_i = l_i 2^(m_i - top).  (m and l stay apart: m + log l would lose l next to a large score.)
// A warp per row, its lanes over the pieces, then over the columns.  Latency: 64 tokens over 1..32,768
// keys, 8 key heads of 128, 9.5 us alone; it is set up while the pieces end.
template <typename T>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a) {
  grid_dep_wait();
  const AttnPlanHdr* hdr = reinterpret_cast<const AttnPlanHdr*>(a.plan);
  const AttnJoin* joins = reinterpret_cast<const AttnJoin*>(a.plan + a.l.at_joins);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = a.s.heads_kv, g = a.l.group, d = a.s.head_dim;
  const AttnSlots slots(a.s, a.l);
  const float2* stat = static_cast<const float2*>(a.workspace);
  const float* part = reinterpret_cast<const float*>(stat + slots.rows(a.l));
  for (int w = blockIdx.x; w < hdr->n_joins * hk; w += gridDim.x) {
    const AttnJoin jn = joins[w / hk];
    const int kh = w % hk;
    const int64_t first = slots.at(jn.slot, kh), step = slots.step(jn.slot);
    for (int r = warp; r < jn.qn * g; r += 8) {
      const int64_t at = first + r;
      float top = -INFINITY;
      for (int p = lane; p < jn.pieces; p += 32) top = fmaxf(top, stat[at + p * step].x);
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
      for (int p0 = 0; p0 < jn.pieces; p0 += 32) {
        float wgt = 0.f;                       // a piece without a key that weighs anything adds nothing
        if (p0 + lane < jn.pieces) {
          const float2 ml = stat[at + (p0 + lane) * step];
          if (ml.y != 0.f) wgt = ml.y * exp2_approx(ml.x - ref);
        }
        sum += warp_sum(wgt);
        const int n = min(32, jn.pieces - p0);
#pragma unroll 4
        for (int p = 0; p < n; ++p) {
          const float f = __shfl_sync(0xffffffffu, wgt, p);
          const float* src = part + (at + (p0 + p) * step) * d;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < d) o[i] = fmaf(f, src[lane + 32 * i], o[i]);
        }
      }
      const int tok = r / g, head = kh * g + r % g;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      T* out = static_cast<T*>(a.out) + (int64_t)(jn.q0 + tok) * a.out_stride + head * d;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < d) out[lane + 32 * i] = from_f32<T>(o[i] * inv);
      if (a.lse && lane == 0)
        a.lse[(int64_t)(jn.q0 + tok) * a.s.heads_q + head] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
    }
  }
}

template <typename T, bool kMaySingle>
cudaError_t launch_typed(const AttnArgs& a, cudaStream_t st) {
  const vitfe_attention_shape& s = a.s;
  CUtensorMap mq, mk, mv;
  // without keys no block is ever loaded: any valid map will do
  const bool keys = s.rows_k > 0;
  if (!make_head_map(&mq, a.q, s.dtype, s.head_dim, s.heads_q, s.rows_q, a.q_stride, a.l.group, a.l.tok) ||
      !make_head_map(&mk, keys ? a.k : a.q, s.dtype, s.head_dim, s.heads_kv, keys ? s.rows_k : 1,
                     keys ? a.k_stride : a.q_stride, 1, kAttnKeys) ||
      !make_head_map(&mv, keys ? a.v : a.q, s.dtype, s.head_dim, s.heads_kv, keys ? s.rows_k : 1,
                     keys ? a.v_stride : a.q_stride, 1, kAttnKeys))
    return cudaErrorInvalidValue;
  const int tile = (s.head_dim + kColBlock - 1) / kColBlock * kColBlockBytes;
  int stages = (kSmemMax - 2048 - 2 * tile) / tile;      // 2 KB: alignment and the barriers
  if (stages > kMaxStages) stages = kMaxStages;
  const int smem = (2 + stages) * tile + 1024;
  static std::atomic<uint64_t> allowed{0};
  int sms = 0;
  cudaError_t e = current_sms(&sms);
  if (e == cudaSuccess)
    e = allow_smem(reinterpret_cast<const void*>(attn_kernel<T, kMaySingle>), kSmemMax - (int)sizeof(FwdShared), allowed, kFwdRegs);
  if (e != cudaSuccess) return e;
  const int64_t work = a.l.cap_items * s.heads_kv;
  attn_kernel<T, kMaySingle><<<(unsigned)(work < sms ? work : sms), kFwdThreads, smem, st>>>(a, mq, mk, mv, stages);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.l.may_split) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * kAttnSMs);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_join_kernel<T>, a);
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
  a.group = a.l.group;
  a.item_tok = 2 * a.l.tok;
  a.causal = s.causal;
  a.plan = static_cast<char*>(plan);
  a.status = status;
  attn_plan_kernel<<<1, kPlanThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t st) {
  if (a.s.rows_q == 0) {
    if (a.status != nullptr) status_ok_kernel<<<1, 1, 0, st>>>(a.status);
    return cudaGetLastError();
  }
  if (a.l.may_single)
    return a.s.dtype == VITFE_F16 ? launch_typed<__half, true>(a, st) : launch_typed<__nv_bfloat16, true>(a, st);
  return a.s.dtype == VITFE_F16 ? launch_typed<__half, false>(a, st) : launch_typed<__nv_bfloat16, false>(a, st);
}

}  // namespace vitfe
