// Attention over packed sequences: the plan's layout and the launchers.
#pragma once

#include "vitfe_block.cuh"

namespace vitfe {

template <typename T>
struct T_is_bf16 {
  static constexpr bool value = false;
};
template <>
struct T_is_bf16<__nv_bfloat16> {
  static constexpr bool value = true;
};

constexpr int kAttnRows = 128;      // rows of one score tile: tokens x the query heads of a key head
constexpr int kAttnKeys = 128;      // keys of one block
constexpr int kAttnSMs = 152;       // GB300; the plan's balance and the capacities derived from it
constexpr int kAttnMinBlocks = 4;   // key blocks below which a range is not cut
constexpr int kAttnFewRows = 32;    // score rows up to which pieces are cheap to join,
constexpr int kAttnFewCuts = 4;     // and then made a fourth of an SM's even share

// A query item: the tokens of one or two score tiles of one sequence over the key blocks
// [kb, ke) of it, for one key head at a time.  Rows are token-major: row = token * group + head.
struct alignas(16) AttnItem {
  int q0;      // first query row
  int qn;      // tokens
  int k0;      // the sequence's first key row
  int kn;      // its keys (0: rows of no sequence)
  int off;     // causal: token i sees keys below min(kn, off + i + 1); full: off = kn
  int kb, ke;
  int slot;    // partial-result slot of this piece, or -1 when the item is whole
};
static_assert(sizeof(AttnItem) == 32, "");

// A key item of the backward pass: up to 128 keys of one sequence against its query tokens.
struct alignas(16) AttnKeyItem {
  int k0;      // first key row
  int kn;      // keys of this tile
  int q0;      // the sequence's first query row
  int qn;      // its tokens (0: rows of no sequence)
  int off;     // causal: token i sees local key j when j <= i + off; full: off = 128
  int pad[3];
};
static_assert(sizeof(AttnKeyItem) == 32, "");

// An item cut into pieces: their slots are slot, slot + 1, ...
struct alignas(16) AttnJoin {
  int q0, qn, slot, pieces;
};

struct alignas(16) AttnPlanHdr {
  int n_items;
  int n_keys;
  int n_joins;
  int tiles;      // score tiles of an item: 2, or 1 where sequences are short
};

// Capacities and offsets of a plan, from the shape alone.
struct AttnLayout {
  int group;              // query heads to a key head
  int tok;                // tokens of one score tile: 128 / group
  bool may_single;        // items may turn out to be of one score tile (attn_plan_kernel)
  int64_t cap_items, cap_keys, cap_joins;
  int64_t cap_many, cap_few;   // slots of partial results of items of many and of few rows
  int64_t at_items, at_keys, at_joins, at_scan_q, at_scan_k, bytes;
  bool may_split;         // some sequence may hold more than kAttnMinBlocks key blocks
};

inline AttnLayout attn_layout(const vitfe_attention_shape& s) {
  AttnLayout l;
  l.group = s.heads_q / s.heads_kv;
  l.tok = kAttnRows / l.group;
  l.may_single = s.max_seqs > 0 && s.rows_q <= (int64_t)s.max_seqs * l.tok;
  l.may_split = (s.rows_k + kAttnKeys - 1) / kAttnKeys > kAttnMinBlocks;
  const int64_t seqs = (int64_t)s.max_seqs + 1;
  // Pieces of items of many rows are as long as an SM's even share of the W blocks of all items and key
  // heads, of few rows a fourth of it (attn_plan_kernel): at most `n` SM shares make n x SMs / heads
  // pieces beyond the first of each item, and twice that number of pieces in all.
  const int64_t many = l.may_split ? kAttnSMs / s.heads_kv + 1 : 0;
  const int64_t few = l.may_split ? kAttnFewCuts * kAttnSMs / s.heads_kv + 1 : 0;
  l.cap_many = 2 * many;
  l.cap_few = 2 * few;
  auto lesser = [](int64_t a, int64_t b) { return a < b ? a : b; };
  l.cap_items = s.rows_q / ((l.may_single ? 1 : 2) * l.tok) + lesser(seqs, s.rows_q) + many + few;
  l.cap_keys = s.rows_k / kAttnKeys + lesser(seqs, s.rows_k);
  l.cap_joins = many + few;
  int64_t at = sizeof(AttnPlanHdr);
  auto take = [&](int64_t n) {
    const int64_t r = at;
    at += (n + 15) / 16 * 16;
    return r;
  };
  l.at_items = take(l.cap_items * (int64_t)sizeof(AttnItem));
  l.at_keys = take(l.cap_keys * (int64_t)sizeof(AttnKeyItem));
  l.at_joins = take(l.cap_joins * (int64_t)sizeof(AttnJoin));
  l.at_scan_q = take((seqs + 1) * 4);
  l.at_scan_k = take((seqs + 1) * 4);
  l.bytes = at;
  return l;
}

// Rows of a slot of an item of many rows.
__host__ __device__ inline int64_t attn_slot_rows(const vitfe_attention_shape& s, const AttnLayout& l) {
  return (s.rows_q < 2 * l.tok ? s.rows_q : 2 * l.tok) * l.group;
}
// First row of a slot of one key head, in the workspace's [rows] of (maximum, sum) and of outputs; the
// slots of an item's pieces follow each other heads_kv slots on.
struct AttnSlots {
  int64_t rows_many, base_few;
  int cap_many, hk;
  __host__ __device__ AttnSlots(const vitfe_attention_shape& s, const AttnLayout& l)
      : rows_many(attn_slot_rows(s, l)), cap_many((int)l.cap_many), hk(s.heads_kv) {
    base_few = l.cap_many * hk * rows_many;
  }
  __host__ __device__ int64_t rows(const AttnLayout& l) const { return base_few + l.cap_few * hk * kAttnFewRows; }
  __host__ __device__ int64_t step(int slot) const { return slot < cap_many ? hk * rows_many : (int64_t)hk * kAttnFewRows; }
  __host__ __device__ int64_t at(int slot, int kh) const {
    return slot < cap_many ? ((int64_t)slot * hk + kh) * rows_many
                           : base_few + ((int64_t)(slot - cap_many) * hk + kh) * kAttnFewRows;
  }
};
inline int64_t attn_workspace(const vitfe_attention_shape& s) {
  const AttnLayout l = attn_layout(s);
  return l.may_split ? (AttnSlots(s, l).rows(l) * (s.head_dim + 2) * 4 + 15) / 16 * 16 : 0;
}
inline int64_t attn_backward_workspace(const vitfe_attention_shape& s) {
  return (s.rows_q * s.heads_q * 8 + 15) / 16 * 16;   // two floats a row and head
}

// ---------------------------------------------------------------------------
// tiles and matrix instructions shared by the forward and backward kernels
// ---------------------------------------------------------------------------
constexpr int kColBlock = 64;                             // 16-bit elements in one 128-byte row
constexpr int kColBlockBytes = kAttnRows * 128;           // 128 rows of it
constexpr uint64_t kAttnDrainNs = 1000000000ull;          // bound of the waits for what is in flight after an abort

// Shared-memory descriptor of a tile of 128-byte rows (128-byte swizzle) read with the row index
// as the contraction: 64 columns contiguous, 8 rows 1024 bytes apart, the next 64 columns one
// column block on.  A step of 16 rows is 2048 bytes.
__device__ __forceinline__ uint64_t sw128_desc_rows(uint32_t saddr) {
  return (sw128_desc(saddr) & ~((uint64_t)0x3FFFu << 16)) | ((uint64_t)(kColBlockBytes >> 4) << 16);
}

// kind::f16 instruction descriptor: 16-bit A and B of one type, fp32 D; `b_rows`: B is read with
// its rows as the contraction.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_16(int m, int n, bool b_rows) {
  const uint32_t fmt = T_is_bf16<T>::value ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (b_rows ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

// D (+)= A * B with A in tensor memory: lane i holds row i, column c the pair (2c, 2c + 1) of its
// contraction index; a step of 16 spans 8 columns.
__device__ __forceinline__ void umma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                            int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// 32 lanes x 16 columns into / from registers.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The warpgroup's registers a thread from here on (all four warps; multiples of 8).
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A value that is the same in all lanes, in a form that the compiler takes as such: loop bounds and
// addresses of the issuing warp then stay in uniform registers, where the matrix instructions want
// their operands (moving each one there costs more than the instruction's own issue).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// A position in a ring of `n` slots: index and the parity of its use.
struct RingPos {
  uint32_t i = 0, parity = 0;
  __device__ __forceinline__ RingPos next(uint32_t n) const {
    RingPos r;
    const bool wrap = i + 1 == n;
    r.i = wrap ? 0u : i + 1;
    r.parity = wrap ? parity ^ 1u : parity;
    return r;
  }
};

// S or dP: D = A B^T over the head's columns, both tiles K-major in shared memory.  `ksteps`: steps of
// 16 columns, up to 8.
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc, int ksteps) {
#pragma unroll
  for (int k = 0; k < VITFE_ATTN_MAX_HEAD_DIM / 16; ++k) {
    constexpr uint64_t block = kColBlockBytes >> 4;
    const uint64_t o = (uint64_t)(k >> 2) * block + (uint64_t)(k & 3) * 2;
    if (k < ksteps) umma_bf16(d_tmem, ad + o, bd + o, idesc, k > 0);
  }
}
// O, dV, dK or dQ: D (+)= A B, A (128 x 128, 16-bit) in tensor memory, B read by rows.  A was written
// over fp32 scores by warps of `kPart` columns each, packed at the start of their own columns.
template <int kPart>
__device__ __forceinline__ void issue_sum(uint32_t d_tmem, uint32_t a_tmem, uint64_t bd, uint32_t idesc,
                                          uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < kAttnKeys / 16; ++k)
    umma_ta(d_tmem, a_tmem + (uint32_t)(k * 16 / kPart * kPart + k * 16 % kPart / 2), bd + (uint64_t)(128 * k), idesc,
            k > 0 ? 1u : accumulate);
}

// mbar_wait_warp<false> all inline: a kernel that shares out its registers anew can hold no call.
__device__ __forceinline__ bool wait_inline(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  const uint32_t b = smem_u32(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
    if ((i & 15u) == 0 && __any_sync(0xffffffffu, *abort_flag != 0 || global_timer_ns() - t0 > limit_ns)) {
      *abort_flag = 1;
      return false;
    }
  }
}

// Zero rows [first, 128) of a tile of `blocks` column blocks (whole warp; the swizzle moves
// 16-byte chunks inside a row only), visible to the tensor core that reads the tile next.
__device__ __forceinline__ void zero_tile_rows(uint32_t tile, int blocks, int first) {
  const int lane = threadIdx.x & 31;
  for (int b = 0; b < blocks; ++b)
    for (uint32_t o = (uint32_t)first * 128u + (uint32_t)lane * 16u; o < (uint32_t)kColBlockBytes; o += 512u)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + (uint32_t)b * kColBlockBytes + o), "r"(0)
                   : "memory");
  fence_proxy_async_smem();
  __syncwarp();
}

// After a wait that ran out, by the whole block: NaN over `n` rows of `len` elements (an item's: at
// most 2^15), so that what is missing shows without the status as well.
template <typename T>
__device__ __forceinline__ void fill_nan(T* rows, int n, int64_t stride, int len) {
  for (int i = threadIdx.x; i < n * len; i += blockDim.x) rows[i / len * stride + i % len] = from_f32<T>(NAN);
}

// Tensor map of a [rows][heads][head_dim] tensor; a box is 64 columns x box_heads x box_rows with
// 128-byte swizzle, and what lies outside the tensor reads as zero.
bool make_head_map(CUtensorMap* map, const void* p, vitfe_dtype dtype, int head_dim, int heads, int64_t rows,
                   int64_t row_stride, int box_heads, int box_rows);

struct AttnArgs {
  vitfe_attention_shape s;
  AttnLayout l;
  const char* plan;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  void* out;               // forward: written; backward: the forward pass's
  int64_t out_stride;
  float* lse;
  void* workspace;
  int32_t* status;
  uint64_t wait_ns;        // bound of every wait in the kernels
  bool stall;              // tests: load nothing, so that the waits run out
  // backward
  const void* dout;
  void *dq, *dk, *dv;
  int64_t dout_stride, dq_stride, dk_stride, dv_stride;
};
cudaError_t launch_attention_plan(const vitfe_attention_shape& s, const int32_t* cu_q, const int32_t* cu_k,
                                  void* plan, int32_t* status, cudaStream_t st);
cudaError_t launch_attention(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attention_backward(const AttnArgs& a, cudaStream_t st);

}  // namespace vitfe
