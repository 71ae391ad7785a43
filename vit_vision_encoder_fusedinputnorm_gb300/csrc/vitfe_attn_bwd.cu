// Attention over packed sequences: the backward pass, in three kernels.
//   rows: delta = sum(dout * out) and the exponents' references, per query row and head.
//   keys: dk and dv of 128 keys, over the query tiles that see them (4 products a tile).
//   queries: dq of 128 rows, over the key blocks that they see (3 products a block).
// S and dP are computed in both of the last two, so that every sum has one owner: no atomics, no
// partial results, the same bits every time, for 7 products instead of 5.
//   p = exp(s - lse), dp = dout.v, ds = p (dp - delta); dv = sum p dout, dk = scale sum ds q,
//   dq = scale sum ds k; a key head's sums run over all its query heads.
// s, dp and all sums are fp32, p and ds are rounded to the tensors' type, as the tensor core takes them.
// bf16, eight sequences of 256 to 5184, 16 heads of 80: 24 + 500 + 440 us, 0.95 ms overlapped, 41% of a
// dense product's rate counting five products (57% counting seven); two sequences of 8192, 16 heads of
// 128: 2.5 ms, 56%.
#include "vitfe_attn.cuh"

namespace vitfe {
namespace {

// Warps of both kernels: 16 on scores (four to a row of the score tile, 32 columns each: their passes
// are latency, and a scheduler with four of them at hand hides more of it than with two), one on
// loads, two on matrix instructions (one is held up whenever it has filled the tensor core's short
// queue; the other one's waits then cost nothing), one that lays out row values and cleans tiles.
constexpr int kScoreWarps = 16, kLoadWarp = 16, kMmaWarp = 17;
constexpr int kBwdThreads = 32 * 20;
constexpr int kMaxSlots = 4;         // of each ring
constexpr int kRowSlots = 2;         // of the row values
constexpr int kSmemMax = 227 * 1024;
constexpr int kSharedFixed = 3 * 1024;      // BwdShared and what aligns the tiles behind it
constexpr float kLog2e = 1.4426950408889634f;

// Per query row and head, negated: the log-sum-exp as an exponent of 2, and delta.  A row that sees
// no key (lse -inf) has -inf here, so that its probabilities are 0.
struct alignas(8) RowValue {
  float nlse2, ndelta;
};

// Read past L1, for a kernel that has not waited for the row values' kernel itself: that one has ended,
// and its writes are in L2, before the kernel in between lets its successor start (it does so behind its own
// wait); but an L1 may still hold what this workspace held in the call before.
__device__ __forceinline__ RowValue row_value_l2(const RowValue* p) {
  const float2 v = __ldcg(reinterpret_cast<const float2*>(p));
  return RowValue{v.x, v.y};
}

// Memory bound: out and dout once.  Eight sequences of 256 to 5184, 16 heads of 80, in bf16 (92 MB):
// 24 us, of which the bytes need 14; a fortieth of the whole.
template <typename T>
__global__ void __launch_bounds__(256) attn_rows_kernel(const AttnArgs a) {
  grid_dep_trigger();
  if (a.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0) {   // a wait that runs out overrides it later
    a.status[0] = kOk;
    a.status[1] = -1;
  }
  // 16 lanes per (row, head), 8 elements a lane
  const int d = a.s.head_dim, sub = threadIdx.x & 15;
  const int64_t n = a.s.rows_q * a.s.heads_q, step = (int64_t)gridDim.x * 16;
  RowValue* rows = static_cast<RowValue*>(a.workspace);
  for (int64_t i0 = (int64_t)blockIdx.x * 16; i0 < n; i0 += step) {
    const int64_t i = i0 + (threadIdx.x >> 4);
    float s = 0.f;
    if (i < n && sub * 8 < d) {
      const int64_t r = i / a.s.heads_q;
      const int h = (int)(i - r * a.s.heads_q);
      const Vec<T, 8> o = *reinterpret_cast<const Vec<T, 8>*>(static_cast<const T*>(a.out) + r * a.out_stride + h * d + sub * 8);
      const Vec<T, 8> g = *reinterpret_cast<const Vec<T, 8>*>(static_cast<const T*>(a.dout) + r * a.dout_stride + h * d + sub * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(to_f32(o.v[e]), to_f32(g.v[e]), s);
    }
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (i < n && sub == 0) {
      const float lse = a.lse[i];
      rows[i] = RowValue{lse == -INFINITY ? -INFINITY : -(lse * kLog2e), -s};
    }
  }
}

// The slots of the two rings.  Ring A holds the tiles that a step's last product still reads (Q for
// dK, K for dQ): its next tile is wanted a step early, so it is the deeper one.
struct RingSizes {
  uint32_t a, b;
};

struct BwdShared {
  uint64_t kv_full, kv_empty;                         // the resident pair of tiles
  uint64_t a_full[kMaxSlots], a_empty[kMaxSlots], b_full[kMaxSlots], b_empty[kMaxSlots];
  uint64_t a_landed[kMaxSlots], b_landed[kMaxSlots];  // of tiles that are cleaned before they are full
  uint64_t row_full[kRowSlots], row_empty[kRowSlots];
  uint64_t s_full[2], s_empty[2], dp_full, dp_read, p_full, ds_full[2], acc_full, drain[2];
  uint32_t tmem;
  int abort;
  uint32_t loads;                                     // tiles asked for so far (query pass)
  alignas(16) float nlse2[kRowSlots][kAttnRows], ndelta[kRowSlots][kAttnRows];   // of a query tile's rows
};
// With two column blocks to a tile, seven tiles and this fill an SM's shared memory to the byte.
static_assert(sizeof(BwdShared) <= kSharedFixed, "");

__device__ __forceinline__ int deal(int round) {
  return round * (int)gridDim.x + ((round & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
}
__device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((unsigned)a + (unsigned)b - 1u) / (unsigned)b); }

// The counts of matrix warps that read the resident tiles and ring B, and that finish an item.
__device__ __forceinline__ void bwd_init(BwdShared& sh, uint32_t kv_users, uint32_t b_users, uint32_t acc_users) {
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sh.kv_full), 1);
    mbar_init(smem_u32(&sh.kv_empty), kv_users);
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(smem_u32(&sh.a_full[i]), 1);
      mbar_init(smem_u32(&sh.a_empty[i]), 1);
      mbar_init(smem_u32(&sh.b_full[i]), 1);
      mbar_init(smem_u32(&sh.b_empty[i]), b_users);
      mbar_init(smem_u32(&sh.a_landed[i]), 1);
      mbar_init(smem_u32(&sh.b_landed[i]), 1);
    }
    for (int i = 0; i < kRowSlots; ++i) {
      mbar_init(smem_u32(&sh.row_full[i]), 1);
      mbar_init(smem_u32(&sh.row_empty[i]), kScoreWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.s_empty[i]), 1);
      mbar_init(smem_u32(&sh.ds_full[i]), kScoreWarps);
      mbar_init(smem_u32(&sh.drain[i]), 1);
    }
    mbar_init(smem_u32(&sh.dp_full), 1);
    mbar_init(smem_u32(&sh.p_full), kScoreWarps);
    mbar_init(smem_u32(&sh.dp_read), kScoreWarps);
    mbar_init(smem_u32(&sh.acc_full), acc_users);
    sh.abort = 0;
    sh.loads = 0;
    fence_mbar_init();
  }
  if ((threadIdx.x >> 5) == kMmaWarp) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
    tc_fence_before();
  }
}

__device__ __forceinline__ void bwd_end(BwdShared& sh, uint32_t tmem, int32_t* status) {
  tc_fence_before();
  __syncthreads();
  if ((threadIdx.x >> 5) == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && sh.abort && status != nullptr) {
    status[0] = kTimeout;
    status[1] = -1;
  }
}

// After an abort: the loads of one ring, or of the resident tiles, land on their own; wait for the last
// `n` uses of the slots at `full` before the CTA ends (2 ms: a tile to be cleaned does not get there).
__device__ __forceinline__ void drain_loads(uint64_t* full, uint32_t n, uint32_t slots) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = n - (n < slots ? n : slots); i < n; ++i)
    while (!mbar_try_wait(smem_u32(&full[i % slots]), (i / slots) & 1u) && global_timer_ns() - t0 < 2000000ull) {
    }
}

// ... and this warp's matrix instructions in flight.
__device__ __forceinline__ void drain_mma(uint64_t* bar) {
  if (elect_one()) umma_commit(smem_u32(bar));
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(smem_u32(bar), 0) && global_timer_ns() - t0 < kAttnDrainNs) {
  }
  __syncwarp();
}

// A wait that may span works whose tiles are none of the waiter's: its bound counts from the last tile that
// the loading warp has asked for (each of whose own waits is bounded).  By a whole warp.
__device__ __forceinline__ bool wait_paced(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns,
                                           const volatile uint32_t* loads) {
  uint64_t t0 = global_timer_ns();
  uint32_t seen = 0;
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_poll<false>(bar, parity))) return true;
    if ((i & 15u) != 0) continue;
    const uint32_t now = (uint32_t)uniform((int)*loads);
    if (now != seen) {
      seen = now;
      t0 = global_timer_ns();
    }
    if (__any_sync(0xffffffffu, *abort_flag != 0 || global_timer_ns() - t0 > limit_ns)) {
      *abort_flag = 1;
      return false;
    }
  }
}

// One tile's column blocks from a [rows][heads][head_dim] tensor.
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int nb, int head, int row) {
  for (int b = 0; b < nb; ++b) tma_load_3d(dst + (uint32_t)b * kColBlockBytes, map, bar, b * kColBlock, head, row);
}

__device__ __forceinline__ uint64_t pair_of(const uint32_t* v) { return (uint64_t)v[0] | ((uint64_t)v[1] << 32); }

// 16-bit rows of an accumulator, columns [c0, c1) in steps of 16, times `f`.
template <typename T>
__device__ __forceinline__ void store_rows(uint32_t acc, int c0, int c1, int d, float f, T* out, bool live, bool have) {
  for (int c = c0; c < c1; c += 16) {
    uint32_t o[16] = {};
    if (have) {
      tmem_ld_32x32b_x16(acc + (uint32_t)c, o);
      tmem_wait_ld();
    }
    if (!live) continue;
#pragma unroll
    for (int e = 0; e < 16; e += 8) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = pack2<T>(__uint_as_float(o[e + 2 * i]) * f, __uint_as_float(o[e + 2 * i + 1]) * f);
      if (c + e < d) *reinterpret_cast<uint4*>(out + c + e) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

// Query tiles [first token, tiles) that see any key of a key item.
struct TileRange {
  int t0, n;
};
__device__ __forceinline__ TileRange query_tiles(const AttnKeyItem& it, int tok) {
  const int from = max(0, -it.off);
  if (from >= it.qn) return TileRange{0, 0};
  const int t0 = from / tok * tok;
  return TileRange{t0, ceil_div(it.qn - t0, tok)};
}

// ---------------------------------------------------------------------------
// dk, dv.  Resident: the tiles of K and V.  Rings: Q tiles and dO tiles.  Scores are transposed (lane =
// key), so that P^T and dS^T are A operands in tensor memory and Q and dO are read with their rows as the
// contraction.  Tensor memory: S^T (P^T over it), dP^T (dS^T over it), dV, dK: 128 columns each.
// One matrix warp runs dV += P^T dO and the next S^T, the other dK += dS^T Q and the next dP^T.
// Heads of 80: the score warps' way from S^T to dS^T bounds it (1,280 of a step's 2,260 cycles are
// products; with nearly all of them left out, both kernels together still took 86% of their time); of
// 128: the products (2,050 of 2,850 cycles).
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attn_keys_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
                     const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const RingSizes ring) {
  extern __shared__ __align__(1024) uint8_t raw[];
  __shared__ BwdShared sh;
  const uint32_t tiles = smem_u32(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = a.s.heads_kv, g = a.l.group, d = a.s.head_dim, tok = a.l.tok;
  const int nb = (d + kColBlock - 1) / kColBlock;
  const uint32_t tile_bytes = (uint32_t)nb * kColBlockBytes;
  const uint32_t ring_a = tiles + 2 * tile_bytes, ring_b = ring_a + ring.a * tile_bytes;
  volatile int* abort_flag = &sh.abort;
  bwd_init(sh, 2, 2, 2);
  // ring rows that no load writes (a group that does not divide 128)
  if (tok * g < kAttnRows && warp < (int)(ring.a + ring.b)) zero_tile_rows(ring_a + (uint32_t)warp * tile_bytes, nb, tok * g);
  __syncthreads();
  // The row values are there; and with them the next kernel of this call may start, on the SMs that this
  // one leaves.
  grid_dep_wait();
  grid_dep_trigger();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t st_col = tmem, dpt_col = tmem + 128u, dv_col = tmem + 256u, dk_col = tmem + 384u;
  const AttnPlanHdr* hdr = reinterpret_cast<const AttnPlanHdr*>(a.plan);
  const AttnKeyItem* items = reinterpret_cast<const AttnKeyItem*>(a.plan + a.l.at_keys);
  const int works = hdr->n_keys * hk;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {      // by a whole warp
    ok = ok && mbar_wait_warp<false>(smem_u32(bar), parity, abort_flag, a.wait_ns);
    return ok;
  };

  if (warp < kScoreWarps) {
    const int part = warp >> 2;                      // columns [32 part, 32 part + 32)
    const int key = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t c0 = lanes + 32u * part;
    const float scale2 = a.scale * kLog2e;
    const uint64_t sc = f32x2(scale2, scale2);
    uint32_t i = 0, acc = 0;                         // tiles so far, finished items (phases)
    RingPos pos;
    for (int r = 0, w = deal(0); ok && w < works; w = deal(++r)) {
      const AttnKeyItem it = items[w / hk];
      const int kh = w % hk;
      const TileRange tr = query_tiles(it, tok);
      for (int q = 0; q < tr.n; ++q, ++i) {
        const uint32_t stg = pos.i;
        if (!wait(&sh.row_full[stg], pos.parity) || !wait(&sh.s_full[0], i & 1u)) break;
        pos = pos.next(kRowSlots);
        tc_fence_after();
        uint32_t s[32], pk[16];
        tmem_ld_32x32b_x32(st_col + c0, s);
        tmem_wait_ld();
        const int t = tr.t0 + q * tok;
        // every row of the tile is there and sees every key; else this key is seen by the columns
        // [from, to) of its part: token t + column / g sees it when key <= token + off
        const bool whole = t + tok <= it.qn && it.off >= it.kn - 1 - t;
        const int from = max(0, key - it.off - t) * g - 32 * part, to = min(tok, it.qn - t) * g - 32 * part;
        // the row vectors are the same for every lane: shared memory serves four floats to the warp at once
        const ulonglong2* nl = reinterpret_cast<const ulonglong2*>(sh.nlse2[stg] + 32 * part);
        const ulonglong2* nd = reinterpret_cast<const ulonglong2*>(sh.ndelta[stg] + 32 * part);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const ulonglong2 v = nl[e >> 2];
          const uint64_t x = fma_f32x2(pair_of(s + e), sc, v.x), y = fma_f32x2(pair_of(s + e + 2), sc, v.y);
          s[e] = __float_as_uint(exp2_approx(lo_f32(x)));
          s[e + 1] = __float_as_uint(exp2_approx(hi_f32(x)));
          s[e + 2] = __float_as_uint(exp2_approx(lo_f32(y)));
          s[e + 3] = __float_as_uint(exp2_approx(hi_f32(y)));
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 32; ++e) s[e] = e < from || e >= to ? 0u : s[e];
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) pk[e >> 1] = pack2<T>(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        tmem_st_32x32b_x16(st_col + c0, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full));
        if (!wait(&sh.dp_full, i & 1u)) break;
        tc_fence_after();
        uint32_t dp[32];
        tmem_ld_32x32b_x32(dpt_col + c0, dp);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const ulonglong2 v = nd[e >> 2];
          const uint64_t x = mul_f32x2(pair_of(s + e), add_f32x2(pair_of(dp + e), v.x));
          const uint64_t y = mul_f32x2(pair_of(s + e + 2), add_f32x2(pair_of(dp + e + 2), v.y));
          dp[e] = (uint32_t)x;
          dp[e + 1] = (uint32_t)(x >> 32);
          dp[e + 2] = (uint32_t)y;
          dp[e + 3] = (uint32_t)(y >> 32);
        }
        if (!whole) {      // a hidden pair counts nothing, whatever dP holds there
#pragma unroll
          for (int e = 0; e < 32; ++e) dp[e] = e < from || e >= to ? 0u : dp[e];
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) pk[e >> 1] = pack2<T>(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1]));
        tmem_st_32x32b_x16(dpt_col + c0, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh.ds_full[0]));
          mbar_arrive(smem_u32(&sh.row_empty[stg]));
        }
      }
      if (!ok || (tr.n > 0 && !wait(&sh.acc_full, acc++ & 1u))) break;
      tc_fence_after();
      // parts 0, 1: the halves of dV's columns; 2, 3: of dK's
      const int64_t krow = (int64_t)it.k0 + key;
      const bool is_v = part < 2;
      const int mid = (d / 2 + 15) / 16 * 16;
      T* out = is_v ? static_cast<T*>(a.dv) + krow * a.dv_stride : static_cast<T*>(a.dk) + krow * a.dk_stride;
      store_rows<T>((is_v ? dv_col : dk_col) + lanes, part & 1 ? mid : 0, part & 1 ? d : mid, d, is_v ? 1.f : a.scale,
                    out + kh * d, key < it.kn, tr.n > 0);
      tc_fence_before();
    }
  } else if (warp == kLoadWarp) {
    if (lane == 0 && !a.stall) {
      uint32_t la = 0, lb = 0, np = 0;      // loads into the rings and the resident tiles
      RingPos pa, pb;
      const uint32_t q_bytes = (uint32_t)(nb * tok * g) * 128u;
      auto load = [&](const CUtensorMap* map, uint64_t* full, uint64_t* empty, uint32_t base, RingPos& p, uint32_t slots,
                      uint32_t& count, int head, int row) {
        if (!mbar_wait(smem_u32(&empty[p.i]), p.parity ^ 1u, abort_flag, a.wait_ns)) return false;
        mbar_arrive_expect_tx(smem_u32(&full[p.i]), q_bytes);
        load_tile(base + p.i * tile_bytes, map, smem_u32(&full[p.i]), nb, head, row);
        p = p.next(slots);
        ++count;
        return true;
      };
      for (int r = 0, w = deal(0); ok && w < works; w = deal(++r)) {
        const AttnKeyItem it = items[w / hk];
        const int kh = w % hk;
        const TileRange tr = query_tiles(it, tok);
        if (tr.n == 0) continue;
        if (!mbar_wait(smem_u32(&sh.kv_empty), (np & 1u) ^ 1u, abort_flag, a.wait_ns)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(smem_u32(&sh.kv_full), 2 * tile_bytes);
        load_tile(tiles, &map_k, smem_u32(&sh.kv_full), nb, kh, it.k0);
        load_tile(tiles + tile_bytes, &map_v, smem_u32(&sh.kv_full), nb, kh, it.k0);
        ++np;
        for (int q = 0; ok && q < tr.n; ++q) {
          const int t = tr.t0 + q * tok;
          const bool clean = it.qn - t < tok;
          ok = load(&map_q, clean ? sh.a_landed : sh.a_full, sh.a_empty, ring_a, pa, ring.a, la, kh * g, it.q0 + t) &&
               load(&map_do, clean ? sh.b_landed : sh.b_full, sh.b_empty, ring_b, pb, ring.b, lb, kh * g, it.q0 + t);
        }
      }
      if (*abort_flag) {
        drain_loads(&sh.kv_full, np, 1);
        drain_loads(sh.a_full, la, ring.a);
        drain_loads(sh.b_full, lb, ring.b);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    const bool first = warp == kMmaWarp;             // S^T and dV; the other: dP^T and dK
    const uint32_t id_s = idesc_16<T>(128, 128, false), id_acc = idesc_16<T>(128, (d + 15) / 16 * 16, true);
    const int ksteps = (d + 15) / 16;
    const uint64_t tile_step = (uint64_t)(tile_bytes >> 4);
    const uint64_t k_desc = sw128_desc(tiles), v_desc = k_desc + tile_step;
    const uint64_t q_cols = sw128_desc(ring_a), do_cols = sw128_desc(ring_b);             // contraction: columns
    const uint64_t q_rows = sw128_desc_rows(ring_a), do_rows = sw128_desc_rows(ring_b);   // contraction: rows
    uint32_t i = 0, np = 0;
    RingPos pa, pb;
    for (int r = 0, w = deal(0); ok && w < works; w = deal(++r)) {
      const AttnKeyItem it = items[w / hk];
      const int n = uniform(query_tiles(it, tok).n);
      if (n == 0) continue;
      if (!wait(&sh.kv_full, np++ & 1u)) break;
      if (first) {
        if (!wait(&sh.a_full[pa.i], pa.parity)) break;
        if (elect_one()) {
          issue_scores(st_col, k_desc, q_cols + pa.i * tile_step, id_s, ksteps);
          umma_commit(smem_u32(&sh.s_full[0]));
        }
      } else {
        if (!wait(&sh.b_full[pb.i], pb.parity)) break;
        if (elect_one()) {
          issue_scores(dpt_col, v_desc, do_cols + pb.i * tile_step, id_s, ksteps);
          umma_commit(smem_u32(&sh.dp_full));
          umma_commit(smem_u32(&sh.b_empty[pb.i]));
        }
      }
      __syncwarp();
      for (int q = 0; q < n; ++q, ++i) {
        const bool more = q + 1 < n;
        const RingPos na = pa.next(ring.a), nbp = pb.next(ring.b);
        if (first) {
          if (!wait(&sh.b_full[pb.i], pb.parity) || (more && !wait(&sh.a_full[na.i], na.parity)) ||
              !wait(&sh.p_full, i & 1u))
            break;
          tc_fence_after();
          if (elect_one()) {
            issue_sum<32>(dv_col, st_col, do_rows + pb.i * tile_step, id_acc, q > 0);
            umma_commit(smem_u32(&sh.b_empty[pb.i]));
            if (more) {
              issue_scores(st_col, k_desc, q_cols + na.i * tile_step, id_s, ksteps);
              umma_commit(smem_u32(&sh.s_full[0]));
            }
          }
        } else {
          if (!wait(&sh.a_full[pa.i], pa.parity) || (more && !wait(&sh.b_full[nbp.i], nbp.parity)) ||
              !wait(&sh.ds_full[0], i & 1u))
            break;
          tc_fence_after();
          if (elect_one()) {
            issue_sum<32>(dk_col, dpt_col, q_rows + pa.i * tile_step, id_acc, q > 0);
            umma_commit(smem_u32(&sh.a_empty[pa.i]));      // (S^T of this tile was done before its dS^T)
            if (more) {
              issue_scores(dpt_col, v_desc, do_cols + nbp.i * tile_step, id_s, ksteps);
              umma_commit(smem_u32(&sh.dp_full));
              umma_commit(smem_u32(&sh.b_empty[nbp.i]));
            }
          }
        }
        __syncwarp();
        if (!more && elect_one()) {
          umma_commit(smem_u32(&sh.acc_full));
          umma_commit(smem_u32(&sh.kv_empty));
        }
        __syncwarp();
        pa = na;
        pb = nbp;
      }
    }
    if (!ok) drain_mma(&sh.drain[first ? 0 : 1]);
  } else {
    // each query tile's row values beside it; and tiles that reach past their sequence: rows of others
    // are zeroed (their P and dS are 0, but 0 * NaN is NaN)
    const RowValue* rows = static_cast<const RowValue*>(a.workspace);
    RingPos pos;
    uint32_t seen = 0, pa = 0, pb = 0;             // tiles so far; a parity bit for each slot's cleaned uses
    for (int r = 0, w = deal(0); ok && w < works; w = deal(++r)) {
      const AttnKeyItem it = items[w / hk];
      const int kh = w % hk;
      const TileRange tr = query_tiles(it, tok);
      for (int q = 0; q < tr.n; ++q) {
        const uint32_t stg = pos.i;
        const int t = tr.t0 + q * tok;
        RowValue v[kAttnRows / 32];
#pragma unroll
        for (int c = 0; c < kAttnRows / 32; ++c) {
          const int x = 32 * c + lane, tt = t + x / g;
          v[c] = RowValue{-INFINITY, 0.f};
          if (x < tok * g && tt < it.qn) v[c] = rows[((int64_t)it.q0 + tt) * a.s.heads_q + kh * g + x % g];
        }
        if (!wait(&sh.row_empty[stg], pos.parity ^ 1u)) break;
        pos = pos.next(kRowSlots);
#pragma unroll
        for (int c = 0; c < kAttnRows / 32; ++c) {
          sh.nlse2[stg][32 * c + lane] = v[c].nlse2;
          sh.ndelta[stg][32 * c + lane] = v[c].ndelta;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.row_full[stg]));
      }
      if (!ok || tr.n == 0) continue;
      seen += (uint32_t)tr.n;
      const int have = it.qn - tr.t0 - (tr.n - 1) * tok;
      if (have >= tok) continue;
      const uint32_t sa = (seen - 1u) % ring.a, sb = (seen - 1u) % ring.b;
      if (!wait(&sh.a_landed[sa], (pa >> sa) & 1u)) break;
      pa ^= 1u << sa;
      zero_tile_rows(ring_a + sa * tile_bytes, nb, have * g);
      if (lane == 0) mbar_arrive(smem_u32(&sh.a_full[sa]));
      if (!wait(&sh.b_landed[sb], (pb >> sb) & 1u)) break;
      pb ^= 1u << sb;
      zero_tile_rows(ring_b + sb * tile_bytes, nb, have * g);
      if (lane == 0) mbar_arrive(smem_u32(&sh.b_full[sb]));
    }
  }
  bwd_end(sh, tmem, a.status);
  for (int r = 0, w = deal(0); sh.abort && w < works; w = deal(++r)) {
    const AttnKeyItem it = items[w / hk];
    fill_nan(static_cast<T*>(a.dk) + (int64_t)it.k0 * a.dk_stride + w % hk * d, it.kn, a.dk_stride, d);
    fill_nan(static_cast<T*>(a.dv) + (int64_t)it.k0 * a.dv_stride + w % hk * d, it.kn, a.dv_stride, d);
  }
}

// ---------------------------------------------------------------------------
// dq.  Resident: the tiles of Q and dO.  Rings: K blocks and V blocks.  Lane = query row; four threads to
// a row, 32 keys each.  Tensor memory: S (two buffers; dS over the one it came from), dP, dQ.
// One matrix warp runs S and dP, the other dQ += dS K.  dP's place is free as soon as all score warps
// have it in their registers, so the next block's dP is not kept waiting for this one's dS (three per
// cent of the gradients).  dS has two barriers in turn, as the score warps may be a block ahead.
// Bounded as the kernel above.
// ---------------------------------------------------------------------------
// Key blocks that tile t of an item reads, over the item's whole range (of a cut item the first
// piece takes all of it: enough rows to fill the GPU are the rule in training).
__device__ __forceinline__ int key_blocks(const AttnItem& it, int t, int tok, bool causal) {
  const int have = min(tok, it.qn - t * tok);
  if (have <= 0 || it.kb > 0) return 0;
  const int last = causal ? min(it.kn, max(0, it.off + t * tok + have)) : it.kn;
  return ceil_div(last, kAttnKeys);
}

template <typename T>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attn_queries_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
                        const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const RingSizes ring) {
  extern __shared__ __align__(1024) uint8_t raw[];
  __shared__ BwdShared sh;
  const uint32_t tiles = smem_u32(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = a.s.heads_kv, g = a.l.group, d = a.s.head_dim, tok = a.l.tok;
  const bool causal = a.s.causal != 0;
  const int nb = (d + kColBlock - 1) / kColBlock;
  const uint32_t tile_bytes = (uint32_t)nb * kColBlockBytes;
  const uint32_t ring_a = tiles + 2 * tile_bytes, ring_b = ring_a + ring.a * tile_bytes;
  volatile int* abort_flag = &sh.abort;
  bwd_init(sh, 1, 1, 1);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t dp_col = tmem + 256u, dq_col = tmem + 384u;    // S buffers: tmem, tmem + 128
  const AttnPlanHdr* hdr = reinterpret_cast<const AttnPlanHdr*>(a.plan);
  const AttnItem* items = reinterpret_cast<const AttnItem*>(a.plan + a.l.at_items);
  const int per = hdr->tiles;                                   // score tiles of an item
  const int works = hdr->n_items * hk * per;                    // (item, key head, tile)
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {             // by a whole warp
    ok = ok && mbar_wait_warp<false>(smem_u32(bar), parity, abort_flag, a.wait_ns);
    return ok;
  };

  if (warp < kScoreWarps) {
    const int part = warp >> 2;                                 // keys [32 part, 32 part + 32) of a block
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float scale2 = a.scale * kLog2e;
    const uint64_t sc = f32x2(scale2, scale2);
    const RowValue* rows = static_cast<const RowValue*>(a.workspace);
    uint32_t i = 0, acc = 0;
    for (int r = 0, w = deal(0); ok && w < works; w = deal(++r)) {
      const AttnItem it = items[w / (per * hk)];
      const int t = w % per, kh = w / per % hk;
      if (it.kb > 0 || it.qn <= t * tok) continue;
      const int n = key_blocks(it, t, tok, causal);
      const int my_tok = t * tok + row / g, head = kh * g + row % g;
      const bool live = row < tok * g && my_tok < it.qn;
      int lim = causal ? min(it.kn, it.off + my_tok + 1) : it.kn;
      RowValue v{-INFINITY, 0.f};
      if (live) v = row_value_l2(rows + ((int64_t)it.q0 + my_tok) * a.s.heads_q + head);
      else lim = 0;
      const uint64_t nl = f32x2(v.nlse2, v.nlse2), nd = f32x2(v.ndelta, v.ndelta);
      for (int j = 0; j < n; ++j, ++i) {
        const uint32_t s_col = tmem + lanes + (i & 1u) * 128u + 32u * part;
        if (!wait(&sh.s_full[i & 1u], (i >> 1) & 1u)) break;
        tc_fence_after();
        uint32_t s[32], dp[32], pk[16];
        tmem_ld_32x32b_x32(s_col, s);
        tmem_wait_ld();
        const int left = lim - j * kAttnKeys - 32 * part;
        const bool whole = __all_sync(0xffffffffu, left >= 32);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t x = fma_f32x2(pair_of(s + e), sc, nl);
          s[e] = __float_as_uint(exp2_approx(lo_f32(x)));
          s[e + 1] = __float_as_uint(exp2_approx(hi_f32(x)));
        }
        if (!wait(&sh.dp_full, i & 1u)) break;
        tc_fence_after();
        tmem_ld_32x32b_x32(dp_col + lanes + 32u * part, dp);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.dp_read));
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t x = mul_f32x2(pair_of(s + e), add_f32x2(pair_of(dp + e), nd));
          dp[e] = (uint32_t)x;
          dp[e + 1] = (uint32_t)(x >> 32);
        }
        if (!whole) {      // a hidden key counts nothing, whatever dP holds there
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e >= left) dp[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) pk[e >> 1] = pack2<T>(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1]));
        tmem_st_32x32b_x16(s_col, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.ds_full[i & 1u]));
      }
      if (!ok || (n > 0 && !wait(&sh.acc_full, acc++ & 1u))) break;
      tc_fence_after();
      // each part of the warps stores a quarter of the columns, in steps of 16
      const int each = (d + 63) / 64 * 16, c0 = min(d, each * part), c1 = min(d, each * (part + 1));
      T* out = static_cast<T*>(a.dq) + ((int64_t)it.q0 + my_tok) * a.dq_stride + head * d;
      store_rows<T>(dq_col + lanes, c0, c1, d, a.scale, out, live, n > 0);
      tc_fence_before();
    }
  } else if (warp == kLoadWarp) {
    if (lane == 0 && !a.stall) {
      uint32_t la = 0, lb = 0, np = 0;      // loads into the rings and the resident tiles
      RingPos pa, pb;
      const uint32_t q_bytes = (uint32_t)(nb * tok * g) * 128u;
      auto load = [&](const CUtensorMap* map, uint64_t* full, uint64_t* empty, uint32_t base, RingPos& p, uint32_t slots,
                      uint32_t& count, int head, int key) {
        if (!mbar_wait(smem_u32(&empty[p.i]), p.parity ^ 1u, abort_flag, a.wait_ns)) return false;
        mbar_arrive_expect_tx(smem_u32(&full[p.i]), tile_bytes);
        load_tile(base + p.i * tile_bytes, map, smem_u32(&full[p.i]), nb, head, key);
        p = p.next(slots);
        ++count;
        *const_cast<volatile uint32_t*>(&sh.loads) = la + lb;
        return true;
      };
      for (int r = 0, w = deal(0); ok && w < works; w = deal(++r)) {
        const AttnItem it = items[w / (per * hk)];
        const int t = w % per, kh = w / per % hk;
        const int nk = key_blocks(it, t, tok, causal);
        if (nk == 0) continue;
        if (!mbar_wait(smem_u32(&sh.kv_empty), (np & 1u) ^ 1u, abort_flag, a.wait_ns)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(smem_u32(&sh.kv_full), 2 * q_bytes);
        load_tile(tiles, &map_q, smem_u32(&sh.kv_full), nb, kh * g, it.q0 + t * tok);
        load_tile(tiles + tile_bytes, &map_do, smem_u32(&sh.kv_full), nb, kh * g, it.q0 + t * tok);
        ++np;
        for (int j = 0; ok && j < nk; ++j) {
          const int key = it.k0 + j * kAttnKeys;
          const bool clean = it.kn - j * kAttnKeys < kAttnKeys;
          ok = load(&map_k, clean ? sh.a_landed : sh.a_full, sh.a_empty, ring_a, pa, ring.a, la, kh, key) &&
               load(&map_v, sh.b_full, sh.b_empty, ring_b, pb, ring.b, lb, kh, key);
        }
      }
      if (*abort_flag) {
        drain_loads(&sh.kv_full, np, 1);
        drain_loads(sh.a_full, la, ring.a);
        drain_loads(sh.b_full, lb, ring.b);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    const bool first = warp == kMmaWarp;             // S and dP; the other: dQ
    const uint32_t id_s = idesc_16<T>(128, 128, false), id_acc = idesc_16<T>(128, (d + 15) / 16 * 16, true);
    const int ksteps = (d + 15) / 16;
    const uint64_t tile_step = (uint64_t)(tile_bytes >> 4);
    const uint64_t q_desc = sw128_desc(tiles), do_desc = q_desc + tile_step;
    const uint64_t k_cols = sw128_desc(ring_a), v_cols = sw128_desc(ring_b), k_rows = sw128_desc_rows(ring_a);
    uint32_t i = 0, np = 0;
    RingPos pa, pb;
    // S of block x into its buffer, when dQ has taken the dS that was there
    auto s_of = [&](const RingPos& p, uint32_t x) {
      if (!wait(&sh.a_full[p.i], p.parity) || !wait(&sh.s_empty[x & 1u], ((x >> 1) & 1u) ^ 1u)) return false;
      tc_fence_after();
      if (elect_one()) {
        issue_scores(tmem + (x & 1u) * 128u, q_desc, k_cols + p.i * tile_step, id_s, ksteps);
        umma_commit(smem_u32(&sh.s_full[x & 1u]));
      }
      __syncwarp();
      return true;
    };
    auto dp_of = [&](const RingPos& p) {
      if (elect_one()) {
        issue_scores(dp_col, do_desc, v_cols + p.i * tile_step, id_s, ksteps);
        umma_commit(smem_u32(&sh.dp_full));
        umma_commit(smem_u32(&sh.b_empty[p.i]));
      }
      __syncwarp();
    };
    for (int r = 0, w = deal(0); ok && w < works; w = deal(++r)) {
      const AttnItem it = items[w / (per * hk)];
      const int n = uniform(key_blocks(it, w % per, tok, causal));
      if (n == 0) continue;
      if (first) {
        if (!wait(&sh.kv_full, np++ & 1u) || !s_of(pa, i) || !wait(&sh.b_full[pb.i], pb.parity)) break;
        dp_of(pb);
      }
      for (int j = 0; j < n; ++j, ++i) {
        const bool more = j + 1 < n;
        const RingPos na = pa.next(ring.a), nbp = pb.next(ring.b);
        if (first) {
          if (more) {
            if (!s_of(na, i + 1) || !wait(&sh.b_full[nbp.i], nbp.parity) || !wait(&sh.dp_read, i & 1u)) break;
            tc_fence_after();
            dp_of(nbp);
          } else {
            // the next item's first dP waits for the scores of this one's last block, as any other
            if (elect_one()) umma_commit(smem_u32(&sh.kv_empty));
            __syncwarp();
            if (!wait(&sh.dp_read, i & 1u)) break;
            tc_fence_after();
          }
        } else {
          if (!wait(&sh.a_full[pa.i], pa.parity) || !wait(&sh.ds_full[i & 1u], (i >> 1) & 1u)) break;
          tc_fence_after();
          if (elect_one()) {
            issue_sum<32>(dq_col, tmem + (i & 1u) * 128u, k_rows + pa.i * tile_step, id_acc, j > 0);
            umma_commit(smem_u32(&sh.a_empty[pa.i]));      // (S of this block was done before its dS)
            umma_commit(smem_u32(&sh.s_empty[i & 1u]));
            if (!more) umma_commit(smem_u32(&sh.acc_full));
          }
          __syncwarp();
        }
        pa = na;
        pb = nbp;
      }
    }
    if (!ok) drain_mma(&sh.drain[first ? 0 : 1]);
  } else {
    // K blocks that reach past their sequence: rows of others are zeroed for dQ (their dS is 0, but
    // 0 * NaN is NaN).  Works that end with a whole block are passed over, so the wait for the next tile
    // to clean may last as long as they do.
    uint32_t na = 0, pa = 0;                         // blocks so far; a parity bit for each slot's cleaned uses
    for (int r = 0, w = deal(0); ok && w < works; w = deal(++r)) {
      const AttnItem it = items[w / (per * hk)];
      const int n = key_blocks(it, w % per, tok, causal);
      if (n == 0) continue;
      na += (uint32_t)n;
      const int have = it.kn - (n - 1) * kAttnKeys;
      if (have >= kAttnKeys) continue;
      const uint32_t sa = (na - 1u) % ring.a;
      if (!wait_paced(smem_u32(&sh.a_landed[sa]), (pa >> sa) & 1u, abort_flag, a.wait_ns, &sh.loads)) break;
      pa ^= 1u << sa;
      zero_tile_rows(ring_a + sa * tile_bytes, nb, have);
      if (lane == 0) mbar_arrive(smem_u32(&sh.a_full[sa]));
    }
  }
  // It may have started beside the kernel before it (which had seen the row values), but ends after it, so
  // that what follows on the stream finds both done.
  grid_dep_wait();
  bwd_end(sh, tmem, a.status);
  for (int r = 0, w = deal(0); sh.abort && w < works; w = deal(++r)) {
    const AttnItem it = items[w / (per * hk)];
    const int first = w % per * tok, n = it.kb > 0 ? 0 : min(tok, it.qn - first), head = w / per % hk * g;
    fill_nan(static_cast<T*>(a.dq) + ((int64_t)it.q0 + first) * a.dq_stride + head * d, n, a.dq_stride, g * d);
  }
}

template <typename T>
cudaError_t launch_typed(const AttnArgs& a, cudaStream_t st) {
  const vitfe_attention_shape& s = a.s;
  static std::atomic<uint64_t> allowed_keys{0}, allowed_queries{0};
  int sms = 0;
  cudaError_t e = current_sms(&sms);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (s.rows_q * s.heads_q + 15) / 16;
  attn_rows_kernel<T><<<(unsigned)(blocks < 1 ? 1 : blocks < 8 * sms ? blocks : 8 * sms), 256, 0, st>>>(a);
  const int tile = (s.head_dim + kColBlock - 1) / kColBlock * kColBlockBytes;
  const uint32_t slots = (uint32_t)((kSmemMax - kSharedFixed) / tile - 2);
  RingSizes ring;
  ring.a = slots / 2 + (slots & 1u) < (uint32_t)kMaxSlots ? slots / 2 + (slots & 1u) : (uint32_t)kMaxSlots;
  ring.b = slots - ring.a < (uint32_t)kMaxSlots ? slots - ring.a : (uint32_t)kMaxSlots;
  const int smem = (2 + (int)(ring.a + ring.b)) * tile;
  CUtensorMap mq, md, mk, mv;
  if (s.rows_q > 0 && s.rows_k > 0) {
    if (!make_head_map(&mq, a.q, s.dtype, s.head_dim, s.heads_q, s.rows_q, a.q_stride, a.l.group, a.l.tok) ||
        !make_head_map(&md, a.dout, s.dtype, s.head_dim, s.heads_q, s.rows_q, a.dout_stride, a.l.group, a.l.tok) ||
        !make_head_map(&mk, a.k, s.dtype, s.head_dim, s.heads_kv, s.rows_k, a.k_stride, 1, kAttnKeys) ||
        !make_head_map(&mv, a.v, s.dtype, s.head_dim, s.heads_kv, s.rows_k, a.v_stride, 1, kAttnKeys))
      return cudaErrorInvalidValue;
  } else if (s.rows_q > 0 || s.rows_k > 0) {
    // one side is empty: every item stores zeros and nothing is loaded, so any valid map will do
    const void* p = s.rows_q > 0 ? a.q : a.k;
    const int64_t rows = s.rows_q > 0 ? s.rows_q : s.rows_k, stride = s.rows_q > 0 ? a.q_stride : a.k_stride;
    if (!make_head_map(&mq, p, s.dtype, s.head_dim, 1, rows, stride, 1, kAttnKeys)) return cudaErrorInvalidValue;
    md = mk = mv = mq;
  }
  const int64_t wk = a.l.cap_keys * s.heads_kv, wq = a.l.cap_items * s.heads_kv * 2;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kBwdThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (s.rows_k > 0) {
    e = allow_smem(reinterpret_cast<const void*>(attn_keys_kernel<T>), kSmemMax - kSharedFixed, allowed_keys);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(wk < sms ? wk : sms));
    e = cudaLaunchKernelEx(&cfg, attn_keys_kernel<T>, a, mq, md, mk, mv, ring);
    if (e != cudaSuccess) return e;
  } else {
    cfg.numAttrs = 0;      // right behind the row values: it waits for them in full
  }
  if (s.rows_q > 0) {
    e = allow_smem(reinterpret_cast<const void*>(attn_queries_kernel<T>), kSmemMax - kSharedFixed, allowed_queries);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(wq < sms ? wq : sms));
    e = cudaLaunchKernelEx(&cfg, attn_queries_kernel<T>, a, mq, md, mk, mv, ring);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_backward(const AttnArgs& a, cudaStream_t st) {
  return a.s.dtype == VITFE_F16 ? launch_typed<__half>(a, st) : launch_typed<__nv_bfloat16>(a, st);
}

}  // namespace vitfe
