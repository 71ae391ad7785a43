// C ABI of the encoder-block operators: argument validation, launches.
#include <cmath>
#include <cstdlib>

#include "vitfe_attn.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxRows = 0x7fffffffLL - 1024;

vitfe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? VITFE_OK : VITFE_ECUDA; }

bool dtype_ok(vitfe_dtype d) { return d == VITFE_BF16 || d == VITFE_F16 || d == VITFE_F32; }

// A [rows][width] matrix of `dtype` with a row stride.
bool matrix_ok(const void* p, int64_t stride, int64_t rows, int64_t width, vitfe_dtype d) {
  if (rows == 0) return true;
  return p != nullptr && aligned(p, vitfe::dtype_bytes(d)) && stride >= width;
}

vitfe_status norm_check(int64_t rows, int32_t width, vitfe_dtype d, const void* weight, const void* bias,
                        vitfe_dtype pd) {
  if (rows < 0 || rows > kMaxRows || width < 1 || !dtype_ok(d) || !dtype_ok(pd)) return VITFE_EINVAL;
  if (!aligned(weight, vitfe::dtype_bytes(pd)) || !aligned(bias, vitfe::dtype_bytes(pd))) return VITFE_EINVAL;
  return width > VITFE_NORM_MAX_WIDTH ? VITFE_EUNSUPPORTED : VITFE_OK;
}

vitfe_status shape_check(const vitfe_attention_shape* s) {
  if (s == nullptr || s->rows_q < 0 || s->rows_q > kMaxRows || s->rows_k < 0 || s->rows_k > kMaxRows) return VITFE_EINVAL;
  if (s->max_seqs < 0 || s->heads_q < 1 || s->heads_kv < 1 || s->heads_q % s->heads_kv != 0) return VITFE_EINVAL;
  if (s->head_dim < 8 || s->head_dim % 8 != 0 || !dtype_ok(s->dtype)) return VITFE_EINVAL;
  if (s->head_dim > VITFE_ATTN_MAX_HEAD_DIM || s->heads_q / s->heads_kv > VITFE_ATTN_MAX_GROUP ||
      s->heads_q > 4096 || s->dtype == VITFE_F32 || s->max_seqs > (1 << 24))
    return VITFE_EUNSUPPORTED;
  const vitfe::AttnLayout l = vitfe::attn_layout(*s);
  // works are counted in 32 bits, query tiles two to an item
  if (l.cap_items * s->heads_kv > kMaxRows / 4 || l.cap_keys * s->heads_kv > kMaxRows / 4) return VITFE_EUNSUPPORTED;
  return VITFE_OK;
}

// [rows][heads][head_dim] with a row stride, in the attention calls' alignment.
bool heads_ok(const void* p, int64_t stride, int64_t rows, int heads, int head_dim) {
  if (rows == 0) return true;
  return p != nullptr && aligned(p, 16) && stride % 8 == 0 && stride >= (int64_t)heads * head_dim;
}

}  // namespace

extern "C" {

vitfe_status vitfe_layer_norm(const void* x, int64_t x_row_stride, vitfe_dtype dtype, int64_t rows, int32_t width,
                              const void* weight, const void* bias, vitfe_dtype param_dtype, float eps, void* out,
                              int64_t out_row_stride, float* mean, float* rstd, cudaStream_t stream) {
  const vitfe_status st = norm_check(rows, width, dtype, weight, bias, param_dtype);
  if (st != VITFE_OK) return st;
  if (!std::isfinite(eps) || eps < 0.0f) return VITFE_EINVAL;
  if (!matrix_ok(x, x_row_stride, rows, width, dtype) || !matrix_ok(out, out_row_stride, rows, width, dtype))
    return VITFE_EINVAL;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return VITFE_EINVAL;
  vitfe::NormArgs a{};
  a.x = x;
  a.x_stride = x_row_stride;
  a.dtype = dtype;
  a.rows = rows;
  a.width = width;
  a.weight = weight;
  a.bias = bias;
  a.param_dtype = param_dtype;
  a.eps = eps;
  a.out = out;
  a.out_stride = out_row_stride;
  a.mean = mean;
  a.rstd = rstd;
  return from_cuda(vitfe::launch_layer_norm(a, stream));
}

int64_t vitfe_layer_norm_workspace(int64_t rows, int32_t width) {
  if (rows < 0 || width < 1) return 0;
  return vitfe::layer_norm_workspace(rows, width);
}

vitfe_status vitfe_layer_norm_backward(const void* dout, int64_t dout_row_stride, const void* x,
                                       int64_t x_row_stride, vitfe_dtype dtype, int64_t rows, int32_t width,
                                       const void* weight, vitfe_dtype param_dtype, const float* mean,
                                       const float* rstd, void* dx, int64_t dx_row_stride, float* dweight,
                                       float* dbias, void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  const vitfe_status st = norm_check(rows, width, dtype, weight, nullptr, param_dtype);
  if (st != VITFE_OK) return st;
  if (!matrix_ok(x, x_row_stride, rows, width, dtype) || !matrix_ok(dout, dout_row_stride, rows, width, dtype) ||
      !matrix_ok(dx, dx_row_stride, rows, width, dtype))
    return VITFE_EINVAL;
  if (rows > 0 && (mean == nullptr || rstd == nullptr)) return VITFE_EINVAL;
  if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4)) return VITFE_EINVAL;
  const bool params = dweight != nullptr || dbias != nullptr;
  if (params && (workspace == nullptr || !aligned(workspace, 16) ||
                 workspace_bytes < vitfe::layer_norm_workspace(rows, width)))
    return VITFE_EINVAL;
  vitfe::NormArgs a{};
  a.x = x;
  a.x_stride = x_row_stride;
  a.dtype = dtype;
  a.rows = rows;
  a.width = width;
  a.weight = weight;
  a.param_dtype = param_dtype;
  a.out = dx;
  a.out_stride = dx_row_stride;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dout = dout;
  a.dout_stride = dout_row_stride;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partial = params ? static_cast<float*>(workspace) : nullptr;
  a.wait_ns = vitfe::wait_limit_ns();
  a.stall = vitfe::stall_loads();
  return from_cuda(vitfe::launch_layer_norm_backward(a, stream));
}

vitfe_status vitfe_mrope_positions(const vitfe_span* spans, const int32_t* n_spans, int32_t max_spans,
                                   const vitfe_item* items, const int32_t* n_items, int32_t max_items, int32_t merge,
                                   int64_t rows, int32_t* pos, int32_t* status, cudaStream_t stream) {
  if (n_spans == nullptr || max_spans < 0 || max_spans > VITFE_MAX_SPANS || (max_spans > 0 && spans == nullptr))
    return VITFE_EINVAL;
  if (max_items < 0 || max_items > VITFE_MAX_ITEMS || (max_items > 0 && (items == nullptr || n_items == nullptr)))
    return VITFE_EINVAL;
  if (merge < 1 || merge > 8 || rows < 0 || rows > kMaxRows || (rows > 0 && pos == nullptr)) return VITFE_EINVAL;
  if (!aligned(spans, 4) || !aligned(n_spans, 4) || !aligned(items, 8) || !aligned(n_items, 4) || !aligned(pos, 4) ||
      !aligned(status, 4))
    return VITFE_EINVAL;
  return from_cuda(vitfe::launch_mrope_positions(spans, n_spans, max_spans, items, n_items, max_items, merge, rows,
                                                 pos, status, stream));
}

vitfe_status vitfe_mrope_apply(const int32_t* pos, int32_t axes, const uint8_t* axis_of_pair, int32_t rotary_dim,
                               float theta, int32_t inverse, int64_t rows, int32_t head_dim, vitfe_dtype dtype,
                               const void* q, int32_t heads_q, int64_t q_row_stride, void* q_out,
                               int64_t q_out_row_stride, const void* k, int32_t heads_k, int64_t k_row_stride,
                               void* k_out, int64_t k_out_row_stride, cudaStream_t stream) {
  if (rows < 0 || rows > kMaxRows || !dtype_ok(dtype)) return VITFE_EINVAL;
  if (head_dim < 8 || head_dim > VITFE_ROPE_MAX_HEAD_DIM || head_dim % 8 != 0) return VITFE_EINVAL;
  if (rotary_dim < 8 || rotary_dim > head_dim || rotary_dim % 8 != 0) return VITFE_EINVAL;
  if (axes < 1 || axes > VITFE_MAX_AXES || axis_of_pair == nullptr) return VITFE_EINVAL;
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (axis_of_pair[i] >= axes) return VITFE_EINVAL;
  if (!std::isfinite(theta) || !(theta > 0.0f)) return VITFE_EINVAL;
  if (heads_q < 0 || heads_k < 0 || heads_q > 4096 || heads_k > 4096) return VITFE_EINVAL;
  if (rows > 0 && (pos == nullptr || !aligned(pos, 4))) return VITFE_EINVAL;
  const size_t base = dtype == VITFE_F32 ? 16 : 8;
  auto ok = [&](const void* p, int64_t stride, int heads) {
    return p != nullptr && aligned(p, base) && stride % 4 == 0 && stride >= (int64_t)heads * head_dim;
  };
  if (rows > 0 && heads_q > 0 && !(ok(q, q_row_stride, heads_q) && ok(q_out, q_out_row_stride, heads_q)))
    return VITFE_EINVAL;
  if (rows > 0 && heads_k > 0 && !(ok(k, k_row_stride, heads_k) && ok(k_out, k_out_row_stride, heads_k)))
    return VITFE_EINVAL;
  vitfe::MropeArgs a{};
  a.pos = pos;
  a.axes = axes;
  a.axis_of_pair = axis_of_pair;
  a.rotary_dim = rotary_dim;
  a.theta = theta;
  a.inverse = inverse != 0;
  a.rows = rows;
  a.head_dim = head_dim;
  a.dtype = dtype;
  a.x[0] = q;
  a.y[0] = q_out;
  a.heads[0] = heads_q;
  a.x_stride[0] = q_row_stride;
  a.y_stride[0] = q_out_row_stride;
  a.x[1] = k;
  a.y[1] = k_out;
  a.heads[1] = heads_k;
  a.x_stride[1] = k_row_stride;
  a.y_stride[1] = k_out_row_stride;
  return from_cuda(vitfe::launch_mrope_apply(a, stream));
}

int64_t vitfe_attention_plan_bytes(const vitfe_attention_shape* shape) {
  return shape_check(shape) == VITFE_OK ? vitfe::attn_layout(*shape).bytes : 0;
}

vitfe_status vitfe_attention_plan(const vitfe_attention_shape* shape, const int32_t* cu_q, const int32_t* cu_k,
                                  void* plan, int32_t* status, cudaStream_t stream) {
  const vitfe_status st = shape_check(shape);
  if (st != VITFE_OK) return st;
  if (cu_q == nullptr || cu_k == nullptr || !aligned(cu_q, 4) || !aligned(cu_k, 4)) return VITFE_EINVAL;
  if (plan == nullptr || !aligned(plan, 16) || !aligned(status, 4)) return VITFE_EINVAL;
  return from_cuda(vitfe::launch_attention_plan(*shape, cu_q, cu_k, plan, status, stream));
}

int64_t vitfe_attention_workspace(const vitfe_attention_shape* shape) {
  return shape_check(shape) == VITFE_OK ? vitfe::attn_workspace(*shape) : 0;
}

int64_t vitfe_attention_backward_workspace(const vitfe_attention_shape* shape) {
  return shape_check(shape) == VITFE_OK ? vitfe::attn_backward_workspace(*shape) : 0;
}

vitfe_status vitfe_attention(const vitfe_attention_shape* shape, const void* plan, const void* q,
                             int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                             int64_t v_row_stride, float scale, void* out, int64_t out_row_stride, float* lse,
                             void* workspace, int32_t* status, cudaStream_t stream) {
  const vitfe_status st = shape_check(shape);
  if (st != VITFE_OK) return st;
  if (plan == nullptr || !aligned(plan, 16) || !std::isfinite(scale) || !(scale > 0.0f)) return VITFE_EINVAL;
  const vitfe_attention_shape& s = *shape;
  if (!heads_ok(q, q_row_stride, s.rows_q, s.heads_q, s.head_dim) ||
      !heads_ok(k, k_row_stride, s.rows_k, s.heads_kv, s.head_dim) ||
      !heads_ok(v, v_row_stride, s.rows_k, s.heads_kv, s.head_dim) ||
      !heads_ok(out, out_row_stride, s.rows_q, s.heads_q, s.head_dim))
    return VITFE_EINVAL;
  if (!aligned(lse, 4) || !aligned(workspace, 16) || !aligned(status, 4)) return VITFE_EINVAL;
  if (vitfe::attn_workspace(s) > 0 && workspace == nullptr) return VITFE_EINVAL;
  vitfe::AttnArgs a{};
  a.s = s;
  a.l = vitfe::attn_layout(s);
  a.plan = static_cast<const char*>(plan);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.scale = scale;
  a.out = out;
  a.out_stride = out_row_stride;
  a.lse = lse;
  a.workspace = workspace;
  a.status = status;
  a.wait_ns = vitfe::wait_limit_ns();
  a.stall = vitfe::stall_loads();
  return from_cuda(vitfe::launch_attention(a, stream));
}

vitfe_status vitfe_attention_backward(const vitfe_attention_shape* shape, const void* plan, const void* dout,
                                      int64_t dout_row_stride, const void* q, int64_t q_row_stride, const void* k,
                                      int64_t k_row_stride, const void* v, int64_t v_row_stride, const void* out,
                                      int64_t out_row_stride, const float* lse, float scale, void* dq,
                                      int64_t dq_row_stride, void* dk, int64_t dk_row_stride, void* dv,
                                      int64_t dv_row_stride, void* workspace, int32_t* status,
                                      cudaStream_t stream) {
  const vitfe_status st = shape_check(shape);
  if (st != VITFE_OK) return st;
  if (plan == nullptr || !aligned(plan, 16) || !std::isfinite(scale) || !(scale > 0.0f)) return VITFE_EINVAL;
  const vitfe_attention_shape& s = *shape;
  if (!heads_ok(q, q_row_stride, s.rows_q, s.heads_q, s.head_dim) ||
      !heads_ok(dout, dout_row_stride, s.rows_q, s.heads_q, s.head_dim) ||
      !heads_ok(out, out_row_stride, s.rows_q, s.heads_q, s.head_dim) ||
      !heads_ok(dq, dq_row_stride, s.rows_q, s.heads_q, s.head_dim) ||
      !heads_ok(k, k_row_stride, s.rows_k, s.heads_kv, s.head_dim) ||
      !heads_ok(v, v_row_stride, s.rows_k, s.heads_kv, s.head_dim) ||
      !heads_ok(dk, dk_row_stride, s.rows_k, s.heads_kv, s.head_dim) ||
      !heads_ok(dv, dv_row_stride, s.rows_k, s.heads_kv, s.head_dim))
    return VITFE_EINVAL;
  if (s.rows_q > 0 && (lse == nullptr || workspace == nullptr)) return VITFE_EINVAL;
  if (!aligned(lse, 4) || !aligned(workspace, 16) || !aligned(status, 4)) return VITFE_EINVAL;
  vitfe::AttnArgs a{};
  a.s = s;
  a.l = vitfe::attn_layout(s);
  a.plan = static_cast<const char*>(plan);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.scale = scale;
  a.out = const_cast<void*>(out);
  a.out_stride = out_row_stride;
  a.lse = const_cast<float*>(lse);
  a.workspace = workspace;
  a.status = status;
  a.wait_ns = vitfe::wait_limit_ns();
  a.stall = vitfe::stall_loads();
  a.dout = dout;
  a.dout_stride = dout_row_stride;
  a.dq = dq;
  a.dq_stride = dq_row_stride;
  a.dk = dk;
  a.dk_stride = dk_row_stride;
  a.dv = dv;
  a.dv_stride = dv_row_stride;
  return from_cuda(vitfe::launch_attention_backward(a, stream));
}

}  // extern "C"

namespace vitfe {

bool stall_loads() {
  const char* env = std::getenv("VITFE_TEST_STALL_BLOCK_LOADS");
  return env != nullptr && env[0] == '1';
}

cudaError_t current_sms(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

cudaError_t allow_smem(const void* kernel, int smem, std::atomic<uint64_t>& done, int regs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  if (regs > 0) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != regs) return cudaErrorInvalidDeviceFunction;
  }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

bool make_head_map(CUtensorMap* map, const void* p, vitfe_dtype dtype, int head_dim, int heads, int64_t rows,
                   int64_t row_stride, int box_heads, int box_rows) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t stride[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)row_stride * 2};
  const cuuint32_t box[3] = {(cuuint32_t)kColBlock, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(map, dtype == VITFE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace vitfe
