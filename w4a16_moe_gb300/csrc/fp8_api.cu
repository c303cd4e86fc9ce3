// extern "C" entry points of the FP8 operators (b4_fp8_* and b4_fused_moe_fp8 in
// b4moe.h): argument validation, workspace carve-up and launches.  Every launch goes to
// the caller's stream; nothing here allocates or synchronises.

#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "b4moe.h"
#include "fp4_ptx.cuh"
#include "fp8.cuh"

namespace b4 {
void set_last_error(const char* fmt, ...);
b4_status require_device(int* sms);
cudaError_t launch_fp8_quantize(const Fp8QuantParams& p, int dtype, int block_rows, int num_sms, cudaStream_t stream);
cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, int rows, int grid, int splits, cudaStream_t stream);
cudaError_t launch_fp8_gemm_direct(const Fp8GemmParams& p, int grid, int splits, cudaStream_t stream);
cudaError_t launch_fp8_gemm_pair(const Fp8GemmParams& p, int pairs, cudaStream_t stream);
cudaError_t launch_fp8_gemm_h(const Fp8GemmParams& p, bool gated, int pairs, cudaStream_t stream);
cudaError_t launch_fp4_combine(const Fp4CombineParams& p, cudaStream_t stream);
}  // namespace b4

using namespace b4;

namespace {

#define FP8_FAIL(st, ...)        \
  do {                           \
    set_last_error(__VA_ARGS__); \
    return st;                   \
  } while (0)
#define FP8_INVALID(...) FP8_FAIL(B4_ERR_INVALID_ARGUMENT, __VA_ARGS__)

b4_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return B4_OK;
  set_last_error("%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return B4_ERR_CUDA;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int dtype_bytes(int dtype) { return dtype == B4_DTYPE_F32 ? 4 : 2; }
bool is_gated(const b4_fp8_config* c) {
  return c->activation == B4_ACT_SILU_SWIGLU || c->activation == B4_ACT_SWIGLU_OAI;
}
int64_t width_of(const b4_fp8_config* c) { return is_gated(c) ? 2 * (int64_t)c->k : c->k; }
int64_t operand_rows(const b4_fp8_config* c, bool ragged) { return ragged ? c->m : (int64_t)c->m * c->num_groups; }

b4_status check(const b4_fp8_config* c) {
  if (!c) FP8_INVALID("cfg is NULL");
  if (c->m < 0 || c->m > (1 << 25)) FP8_INVALID("m = %d not in [0, 2^25]", c->m);
  if (c->num_groups < 1 || c->num_groups > B4_MAX_LOCAL_EXPERTS)
    FP8_INVALID("num_groups = %d not in [1, %d]", c->num_groups, B4_MAX_LOCAL_EXPERTS);
  if (c->k < 16 || c->k % 16 || c->k > (1 << 16)) FP8_INVALID("k = %d must be a positive multiple of 16 (<= 65536)", c->k);
  if (c->x_dtype < B4_DTYPE_BF16 || c->x_dtype > B4_DTYPE_F32) FP8_INVALID("x_dtype = %d unknown", c->x_dtype);
  if (c->out_dtype < B4_DTYPE_BF16 || c->out_dtype > B4_DTYPE_F32) FP8_INVALID("out_dtype = %d unknown", c->out_dtype);
  if (c->activation < -1 || c->activation > B4_ACT_SWIGLU_OAI) FP8_INVALID("activation = %d unknown", c->activation);
  if (c->activation == B4_ACT_SWIGLU_OAI &&
      (!std::isfinite(c->swiglu_alpha) || !std::isfinite(c->swiglu_beta) || !(c->swiglu_limit > 0.0f)))
    FP8_INVALID("swiglu_alpha = %g and swiglu_beta = %g must be finite and swiglu_limit = %g positive",
                (double)c->swiglu_alpha, (double)c->swiglu_beta, (double)c->swiglu_limit);
  if (c->scale_mode != B4_FP8_SCALE_F32 && c->scale_mode != B4_FP8_SCALE_POW2) FP8_INVALID("scale_mode = %d unknown", c->scale_mode);
  if (c->block_rows != 1 && c->block_rows != kFp8Block) FP8_INVALID("block_rows = %d is neither 1 nor 128", c->block_rows);
  if (c->row_div < 1) FP8_INVALID("row_div = %d must be positive", c->row_div);
  if (c->x_rows < 0) FP8_INVALID("x_rows = %d negative", c->x_rows);
  if (c->x_stride != 0 && c->x_stride < width_of(c))
    FP8_INVALID("x_stride = %lld below the row's %lld elements", (long long)c->x_stride, (long long)width_of(c));
  return B4_OK;
}

b4_status check_n(const b4_fp8_config* c) {
  if (c->n < 1 || c->n > (1 << 20)) FP8_INVALID("n = %d not in [1, 2^20]", c->n);
  if (c->out_stride != 0 && c->out_stride < c->n)
    FP8_INVALID("out_stride = %lld below n = %d", (long long)c->out_stride, c->n);
  if (c->block_rows != 1) FP8_INVALID("a product takes activations with a scale per row (block_rows = 1)");
  return B4_OK;
}

b4_status check_rows(const b4_fp8_config* c, bool ragged) {
  if (operand_rows(c, ragged) > INT_MAX - 256)
    FP8_INVALID("%lld rows exceed the row index", (long long)operand_rows(c, ragged));
  return B4_OK;
}

Fp8QuantParams quant_params(const b4_fp8_config* c, const void* x, const int32_t* rows, const int32_t* offsets,
                            uint8_t* codes, float* scales, void* values) {
  Fp8QuantParams p{};
  Fp4QuantParams& q = p.q;
  q.x = x;
  q.x_stride = c->x_stride ? c->x_stride : width_of(c);
  q.rows = rows;
  q.row_div = c->row_div;
  q.x_rows = c->x_rows;
  q.offsets = offsets;
  q.groups = c->num_groups;
  q.m = c->m;
  q.k = c->k;
  q.act = c->activation < 0 ? -1 : is_gated(c) ? 0 : 1;
  q.glu = c->activation == B4_ACT_SWIGLU_OAI ? GluParams{c->swiglu_alpha, c->swiglu_beta, c->swiglu_limit}
                                             : GluParams{1.0f, 0.0f, INFINITY};
  q.codes = codes;
  q.ld = c->k;
  q.values = values;
  q.values_vec = aligned(values, 32) && c->k * dtype_bytes(c->x_dtype) % 32 == 0 ? 2 : 1;
  const int64_t pitch = q.x_stride * dtype_bytes(c->x_dtype);
  q.vec = aligned(x, 32) && pitch % 32 == 0 ? 2 : aligned(x, 16) && pitch % 16 == 0 ? 1 : 0;
  // (the gated prologue's second half starts k elements on: a multiple of 32 bytes, k being one of 16)
  p.scales = scales;
  p.kb = cdiv(c->k, kFp8Block);
  p.pow2 = c->scale_mode == B4_FP8_SCALE_POW2;
  return p;
}

// Activation rows of a unit: 32 or 128 (fp8_gemm.cuh, one SM a unit of 128 outputs), 256
// (fp8_gemm_pair.cu, a pair of SMs, 256 outputs).  By the rows, of ragged groups their mean.
// Measured in us at 32 / 128 / 256: N = K = 4096, m = 64 9.5 / 13.4 / 18.0, 128 12.7 / 13.9 / 19.0, 256 21.3 / 14.1 /
// 19.1, 512 38.8 / 14.5 / 19.5, 1024 66 / 25.5 / 19.9; 64 groups, N = 2816, K = 2048, mean 6 61.4 / 64.4 / -, 16 62.3 / 65.1 /
// -, 96 168 / 69.4 / 73.8, 128 214 / 91.5 / 83.9, 192 - / 123 / 99.5, with popularities spread by e^N(0, 1) 64 124 / 71.1 /
// 69.1, 96 164 / 83.4 / 76.7, 192 - / 123 / 99.6; 28 groups, N = K = 2880, mean 32 54.7 / 47.3 / 50.9, 64 80.0 / 48.2 / 52.3,
// 96 - / 49.5 / 54.0, 128 - / 62.9 / 61.6.
int unit_rows(const b4_fp8_config* c, bool ragged) {
  if (ragged) {
    const int64_t per = c->m / c->num_groups;
    return per <= 16 ? 32 : per <= 104 ? 128 : 256;
  }
  return c->m <= 128 ? 32 : c->m <= 512 ? 128 : 256;
}

// Most units a call can have: a group ends at most one unit early, and holds at least one
// row.
int64_t most_units(const b4_fp8_config* c, bool ragged, int rows) {
  int64_t tok = (int64_t)cdiv(c->m, rows) * c->num_groups;
  if (ragged) tok = c->m / rows + c->num_groups < c->m ? c->m / rows + c->num_groups : c->m;
  return tok * cdiv(c->n, rows == 256 ? 256 : 128);
}

// CTAs that share a unit along K where the units are fewer than the SMs: each keeps three stages
// (of 128 K) or more, and the first has room for the others' partial sums.
int k_splits(const b4_fp8_config* c, int64_t units, int sms) {
  const int stages = cdiv(c->k, kFp8Block);
  const int rows = c->m < 32 ? c->m : 32;
  int splits = 8;
  while (splits > 1 && (splits * units > sms || stages < 3 * splits || (splits - 1) * rows * 512 > kFp8PartBytes)) splits /= 2;
  return splits;
}

// 16-bit outputs as boxes of 64 columns x 32 rows, 128-byte swizzle.
bool make_tmap_out16(CUtensorMap* tm, void* out, uint64_t rows, uint64_t cols, uint64_t stride) {
  TmapEncodeFn fn = tmap_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {stride * 2};
  const cuuint32_t box[2] = {64, 32};
  const cuuint32_t estr[2] = {1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The fields of a product that do not depend on where its activations come from.
Fp8GemmParams product_params(const b4_fp8_config* c, const float* w_scales, const int32_t* offsets, const int32_t* out_rows,
                             void* out, uint32_t* status) {
  Fp8GemmParams p{};
  Fp4GemmParams& g = p.g;
  g.groups = c->num_groups;
  g.m = c->m;
  g.n = c->n;
  g.k = c->k;
  g.offsets = offsets;
  g.out_rows = out_rows;
  g.out_rows_end = (int)operand_rows(c, offsets);
  g.out = out;
  g.out_stride = c->out_stride ? c->out_stride : c->n;
  g.out_dtype = c->out_dtype;
  const int per16 = 16 / dtype_bytes(c->out_dtype);
  g.vec = aligned(out, 16) && g.out_stride % per16 == 0 && c->n % per16 == 0;
  g.halves_from = INT_MAX;
  g.status = status;
  p.w_scales = w_scales;
  p.kb = cdiv(c->k, kFp8Block);
  p.w_vec = aligned(w_scales, 16) && p.kb % 4 == 0;
  return p;
}

// K splits of a direct product (0: the call takes the two launches): few rows, every unit has a
// CTA or a cluster of its own, and a CTA's part of the quantised rows fits in shared memory.
int direct_splits(const b4_fp8_config* c, bool ragged, int sms) {
  if (c->m > kFp8DirectRows) return 0;
  const int64_t units = most_units(c, ragged, 32);
  if (units > sms) return 0;
  const int splits = k_splits(c, units, sms);
  return cdiv(cdiv(c->k, kFp8Block), splits) <= (splits > 1 ? kFp8DirectSplitStages : kFp8DirectStages) ? splits : 0;
}

b4_status launch_direct(const b4_fp8_config* c, const Fp8QuantParams& q, const uint8_t* w_codes, const float* w_scales,
                        const int32_t* out_rows, void* out, uint32_t* clear, uint32_t* status, int splits,
                        cudaStream_t stream) {
  Fp8GemmParams p = product_params(c, w_scales, q.q.offsets, out_rows, out, status);
  if (!make_tmap_bytes_2d(&p.tmap_w, w_codes, (uint64_t)c->n * c->num_groups, c->k, c->k, 128))
    FP8_FAIL(B4_ERR_CUDA, "cuTensorMapEncodeTiled rejected an operand map");
  p.q = q;
  p.x_dtype = c->x_dtype;
  p.g.clear_status = clear != nullptr;
  return cuda_status(launch_fp8_gemm_direct(p, (int)most_units(c, q.q.offsets, 32), splits, stream), "fp8 product");
}

b4_status launch_product(const b4_fp8_config* c, const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes,
                         const float* w_scales, const int32_t* offsets, const int32_t* out_rows, void* out,
                         uint32_t* status, bool a_is_new, int sms, cudaStream_t stream) {
  Fp8GemmParams p = product_params(c, w_scales, offsets, out_rows, out, status);
  const int rows = unit_rows(c, offsets);
  if (!make_tmap_bytes_2d(&p.tmap_w, w_codes, (uint64_t)c->n * c->num_groups, c->k, c->k, 128) ||
      !make_tmap_bytes_2d(&p.tmap_a, a_codes, (uint64_t)operand_rows(c, offsets), c->k, c->k, rows == 256 ? 64 : 32))
    FP8_FAIL(B4_ERR_CUDA, "cuTensorMapEncodeTiled rejected an operand map");
  p.out_boxes = rows == 256 && !out_rows && p.g.vec && c->out_dtype != B4_DTYPE_F32;
  if (p.out_boxes && !make_tmap_out16(&p.tmap_out, out, (uint64_t)operand_rows(c, offsets), c->n, p.g.out_stride))
    FP8_FAIL(B4_ERR_CUDA, "cuTensorMapEncodeTiled rejected an output map");
  p.a_scales = a_scales;
  p.a_vec = aligned(a_scales, 16) && p.kb % 4 == 0;
  p.g.a_is_new = a_is_new;
  const int64_t units = most_units(c, offsets, rows);
  if (units > (1 << 30)) FP8_INVALID("too many units of work: m, n and num_groups too large together");
  if (rows == 256)
    return cuda_status(launch_fp8_gemm_pair(p, (int)(units < sms / 2 ? units : sms / 2), stream), "fp8 product");
  const int splits = rows == 32 ? k_splits(c, units, sms) : 1;
  return cuda_status(launch_fp8_gemm(p, rows, (int)(splits > 1 || units < sms ? units : sms), splits, stream), "fp8 product");
}

// Workspace of b4_fp8_linear: the quantised activation operand of m rows.
struct LinearWs {
  size_t status, codes, scales, total;
};

LinearWs linear_ws(const b4_fp8_config* c) {
  LinearWs L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  L.status = take(256);
  L.codes = take((size_t)c->m * c->k);
  L.scales = take(sizeof(float) * (size_t)c->m * cdiv(c->k, kFp8Block));
  L.total = off;
  return L;
}

b4_status quantize_and_multiply(const b4_fp8_config* c, const void* x, const int32_t* rows, const int32_t* offsets,
                                const uint8_t* w_codes, const float* w_scales, const int32_t* out_rows, void* out,
                                uint8_t* ws, uint32_t* clear, uint32_t* status, int sms, cudaStream_t stream) {
  const LinearWs L = linear_ws(c);
  uint8_t* codes = ws + L.codes;
  float* scales = reinterpret_cast<float*>(ws + L.scales);
  Fp8QuantParams q = quant_params(c, x, rows, offsets, codes, scales, nullptr);
  if (const int splits = direct_splits(c, offsets, sms))
    return launch_direct(c, q, w_codes, w_scales, out_rows, out, clear, status, splits, stream);
  q.q.status = clear;
  const cudaError_t e = launch_fp8_quantize(q, c->x_dtype, 1, sms, stream);
  if (e != cudaSuccess) return cuda_status(e, "fp8 quantise");
  return launch_product(c, codes, scales, w_codes, w_scales, offsets, out_rows, out, status, true, sms, stream);
}

b4_status check_weights(const uint8_t* w_codes, const float* w_scales) {
  if (!w_codes || !w_scales) FP8_INVALID("null weight pointer");
  if (!aligned(w_codes, 16)) FP8_INVALID("weight codes must be 16-byte aligned");
  if (!aligned(w_scales, 4)) FP8_INVALID("misaligned weight scales");
  return B4_OK;
}

// The layer's FC1 for many rows: x quantised into `ws` (linear_ws of c), the product, and h = act(x W13^T)
// quantised into h_codes and h_scales by the product's own kernel.
b4_status quantize_and_make_h(const b4_fp8_config* c, const b4_fp8_config* act, const void* x, const int32_t* rows,
                              const int32_t* offsets, const uint8_t* w_codes, const float* w_scales, uint8_t* ws,
                              uint8_t* h_codes, float* h_scales, uint32_t* status, int sms, cudaStream_t stream) {
  const LinearWs L = linear_ws(c);
  uint8_t* codes = ws + L.codes;
  float* scales = reinterpret_cast<float*>(ws + L.scales);
  Fp8QuantParams q = quant_params(c, x, rows, offsets, codes, scales, nullptr);
  q.q.status = status;
  const cudaError_t e = launch_fp8_quantize(q, c->x_dtype, 1, sms, stream);
  if (e != cudaSuccess) return cuda_status(e, "fp8 quantise");
  Fp8GemmParams p = product_params(c, w_scales, offsets, nullptr, nullptr, status);
  const bool gated = is_gated(act);
  if (!make_tmap_bytes_2d(&p.tmap_w, w_codes, (uint64_t)c->n * c->num_groups, c->k, c->k, gated ? 64 : 128) ||
      !make_tmap_bytes_2d(&p.tmap_a, codes, (uint64_t)c->m, c->k, c->k, 64))
    FP8_FAIL(B4_ERR_CUDA, "cuTensorMapEncodeTiled rejected an operand map");
  p.a_scales = scales;
  p.a_vec = aligned(scales, 16) && p.kb % 4 == 0;
  p.g.a_is_new = 1;
  p.q = quant_params(act, nullptr, nullptr, offsets, h_codes, h_scales, nullptr);
  const int64_t units = most_units(c, true, 256);
  if (units > (1 << 30)) FP8_INVALID("too many units of work: m, n and num_groups too large together");
  return cuda_status(launch_fp8_gemm_h(p, gated, (int)(units < sms / 2 ? units : sms / 2), stream), "fp8 product");
}

// The layer: the shapes of its two products and its workspace.
struct MoeFp8 {
  b4_fp8_config c1, c2;
  size_t status, counts, offsets, sorted, quant, fc1, y, total;
};

b4_status moe_plan(const b4_moe_config* cfg, int32_t activation, MoeFp8* M) {
  if (!cfg) FP8_INVALID("cfg is NULL");
  b4_moe_config shared = *cfg;  // the shared checks (the reason is set); format and path are not read
  shared.format = B4_NVFP4_E4M3_K16;
  shared.path = B4_PATH_AUTO;
  if (b4_workspace_bytes(&shared, activation) == 0) return B4_ERR_INVALID_ARGUMENT;
  const int r_cap = b4_route_capacity_tokens(cfg->m) * cfg->top_k;
  const int n1 = activation == B4_ACT_RELU2 ? cfg->inter : 2 * cfg->inter;
  b4_fp8_config c{};
  c.m = cfg->m * cfg->top_k;
  c.num_groups = cfg->num_local_experts;
  c.x_dtype = c.out_dtype = B4_DTYPE_BF16;
  c.scale_mode = B4_FP8_SCALE_F32;
  c.block_rows = 1;
  c.row_div = 1;
  c.activation = -1;
  M->c1 = M->c2 = c;
  M->c1.n = n1;
  M->c1.k = cfg->hidden;
  M->c1.row_div = cfg->top_k;
  M->c1.x_rows = cfg->m;
  M->c1.out_dtype = B4_DTYPE_F32;
  M->c2.x_dtype = B4_DTYPE_F32;
  M->c2.n = cfg->hidden;
  M->c2.k = cfg->inter;
  M->c2.activation = activation;
  M->c2.swiglu_alpha = cfg->swiglu_alpha;
  M->c2.swiglu_beta = cfg->swiglu_beta;
  M->c2.swiglu_limit = cfg->swiglu_limit;
  b4_fp8_config cap1 = M->c1, cap2 = M->c2;  // sizes depend on m only through its capacity
  cap1.m = cap2.m = r_cap;
  const LinearWs L1 = linear_ws(&cap1), L2 = linear_ws(&cap2);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  M->status = take(256);
  M->counts = take(sizeof(int32_t) * cfg->num_local_experts);
  M->offsets = take(sizeof(int32_t) * (cfg->num_local_experts + 1));
  M->sorted = take(sizeof(int32_t) * (size_t)r_cap);
  M->quant = take(L1.total > L2.total ? L1.total : L2.total);  // x's rows, then h's
  M->fc1 = take(sizeof(float) * (size_t)r_cap * n1);
  // FC2's output of a route, rounded to bf16 before the weighted sum: 2^-9 of it, where each code of its operands
  // is rounded by 2^-4; in 32 bits the rows that pass through memory here would be twice as many bytes
  M->y = take(sizeof(uint16_t) * (size_t)r_cap * cfg->hidden);
  M->total = off;
  return B4_OK;
}

b4_status combine(const b4_moe_config* cfg, const uint16_t* y, const int32_t* topk_ids, const float* topk_weights,
                  uint16_t* out, cudaStream_t s) {
  Fp4CombineParams cp{};
  cp.y = y;
  cp.topk_ids = topk_ids;
  cp.topk_weights = topk_weights;
  cp.expert_map = cfg->expert_map;
  cp.m = cfg->m;
  cp.top_k = cfg->top_k;
  cp.num_global_experts = cfg->num_global_experts;
  cp.num_local_experts = cfg->num_local_experts;
  cp.hidden = cfg->hidden;
  cp.out = out;
  return cuda_status(launch_fp4_combine(cp, s), "fp8 combine");
}

}  // namespace

extern "C" {

b4_status b4_fp8_quantize(const b4_fp8_config* cfg, const void* x, const int32_t* rows, const int32_t* offsets,
                          uint8_t* codes, float* scales, void* values, b4_stream_t stream) {
  b4_status st = check(cfg);
  if (st != B4_OK) return st;
  if ((st = check_rows(cfg, offsets)) != B4_OK) return st;
  if (cfg->block_rows != 1 && (rows || offsets)) FP8_INVALID("blocks of 128 rows take neither rows nor offsets");
  if (cfg->m == 0) return B4_OK;
  if (!x || !codes || !scales) FP8_INVALID("null pointer argument");
  if (!aligned(codes, 16) || !aligned(values, 16)) FP8_INVALID("codes and values must be 16-byte aligned");
  if (!aligned(x, dtype_bytes(cfg->x_dtype)) || !aligned(scales, 4) || !aligned(rows, 4) || !aligned(offsets, 4))
    FP8_INVALID("misaligned x, scales, rows or offsets");
  const int64_t most = cfg->block_rows == 1 ? operand_rows(cfg, offsets) : (int64_t)cdiv(cfg->m, kFp8Block) * cfg->num_groups;
  if (most * cdiv(cfg->k, kFp8Block) > (int64_t)INT_MAX * (cfg->block_rows == 1 ? 16 : 1))
    FP8_INVALID("too many blocks: m, k and num_groups too large together");
  int sms = 0;
  if ((st = require_device(&sms)) != B4_OK) return st;
  const Fp8QuantParams p = quant_params(cfg, x, rows, offsets, codes, scales, values);
  return cuda_status(launch_fp8_quantize(p, cfg->x_dtype, cfg->block_rows, sms, reinterpret_cast<cudaStream_t>(stream)),
                     "fp8 quantise");
}

b4_status b4_fp8_matmul(const b4_fp8_config* cfg, const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes,
                        const float* w_scales, const int32_t* offsets, const int32_t* out_rows, void* out,
                        uint32_t* device_status, b4_stream_t stream) {
  b4_status st = check(cfg);
  if (st != B4_OK) return st;
  if ((st = check_n(cfg)) != B4_OK || (st = check_rows(cfg, offsets)) != B4_OK) return st;
  if (cfg->m == 0) return B4_OK;
  if (!a_codes || !a_scales || !out) FP8_INVALID("null pointer argument");
  if ((st = check_weights(w_codes, w_scales)) != B4_OK) return st;
  if (!aligned(a_codes, 16)) FP8_INVALID("a_codes must be 16-byte aligned");
  if (!aligned(a_scales, 4) || !aligned(out, dtype_bytes(cfg->out_dtype)) || !aligned(offsets, 4) ||
      !aligned(out_rows, 4) || !aligned(device_status, 4))
    FP8_INVALID("misaligned a_scales, out, offsets, out_rows or device_status");
  int sms = 0;
  if ((st = require_device(&sms)) != B4_OK) return st;
  return launch_product(cfg, a_codes, a_scales, w_codes, w_scales, offsets, out_rows, out, device_status, false, sms,
                        reinterpret_cast<cudaStream_t>(stream));
}

size_t b4_fp8_linear_workspace_bytes(const b4_fp8_config* cfg) {
  if (check(cfg) != B4_OK || check_n(cfg) != B4_OK) return 0;
  return linear_ws(cfg).total;
}

b4_status b4_fp8_linear(const b4_fp8_config* cfg, const void* x, const int32_t* rows, const int32_t* offsets,
                        const uint8_t* w_codes, const float* w_scales, const int32_t* out_rows, void* out,
                        void* workspace, size_t workspace_bytes, b4_stream_t stream) {
  b4_status st = check(cfg);
  if (st != B4_OK) return st;
  if ((st = check_n(cfg)) != B4_OK) return st;
  if (!offsets && cfg->num_groups != 1) FP8_INVALID("num_groups = %d without offsets", cfg->num_groups);
  if (cfg->m == 0) return B4_OK;
  if (!x || !out || !workspace) FP8_INVALID("null pointer argument");
  if ((st = check_weights(w_codes, w_scales)) != B4_OK) return st;
  if (!aligned(workspace, 256)) FP8_INVALID("workspace must be 256-byte aligned");
  if (!aligned(x, dtype_bytes(cfg->x_dtype)) || !aligned(out, dtype_bytes(cfg->out_dtype)) || !aligned(rows, 4) ||
      !aligned(offsets, 4) || !aligned(out_rows, 4))
    FP8_INVALID("misaligned x, out, rows, offsets or out_rows");
  const LinearWs L = linear_ws(cfg);
  if (workspace_bytes < L.total)
    FP8_FAIL(B4_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", workspace_bytes, L.total);
  int sms = 0;
  if ((st = require_device(&sms)) != B4_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* status = reinterpret_cast<uint32_t*>(ws + L.status);
  return quantize_and_multiply(cfg, x, rows, offsets, w_codes, w_scales, out_rows, out, ws, status, status, sms,
                               reinterpret_cast<cudaStream_t>(stream));
}

size_t b4_fused_moe_fp8_workspace_bytes(const b4_moe_config* cfg, int32_t activation) {
  MoeFp8 M{};
  return moe_plan(cfg, activation, &M) == B4_OK ? M.total : 0;
}

b4_status b4_fused_moe_fp8(const b4_moe_config* cfg, const uint16_t* x, const uint8_t* w13, const float* s13,
                           const uint8_t* w2, const float* s2, const int32_t* topk_ids, const float* topk_weights,
                           int32_t activation, uint16_t* out, void* workspace, size_t workspace_bytes,
                           b4_stream_t stream) {
  MoeFp8 M{};
  b4_status st = moe_plan(cfg, activation, &M);
  if (st != B4_OK) return st;
  if ((st = check(&M.c2)) != B4_OK || (st = check_n(&M.c1)) != B4_OK || (st = check_n(&M.c2)) != B4_OK) return st;
  if (cfg->m == 0) return B4_OK;
  if (!x || !topk_ids || !topk_weights || !out || !workspace) FP8_INVALID("null pointer argument");
  if ((st = check_weights(w13, s13)) != B4_OK || (st = check_weights(w2, s2)) != B4_OK) return st;
  if (!aligned(x, 16) || !aligned(out, 16)) FP8_INVALID("x and out must be 16-byte aligned");
  if (!aligned(topk_ids, 4) || !aligned(topk_weights, 4)) FP8_INVALID("misaligned topk_ids or topk_weights");
  if (!aligned(workspace, 256)) FP8_INVALID("workspace must be 256-byte aligned");
  if (workspace_bytes < M.total)
    FP8_FAIL(B4_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", workspace_bytes, M.total);
  int sms = 0;
  if ((st = require_device(&sms)) != B4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* status = reinterpret_cast<uint32_t*>(ws + M.status);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + M.offsets);
  int32_t* sorted = reinterpret_cast<int32_t*>(ws + M.sorted);
  float* fc1 = reinterpret_cast<float*>(ws + M.fc1);
  uint16_t* y = reinterpret_cast<uint16_t*>(ws + M.y);
  b4_moe_config pack = *cfg;
  pack.format = B4_NVFP4_E4M3_K16;
  pack.path = B4_PATH_AUTO;
  if ((st = b4_route_pack(&pack, topk_ids, reinterpret_cast<int32_t*>(ws + M.counts), offsets, sorted, stream)) != B4_OK)
    return st;
  // many rows and whole blocks of h: FC1 leaves h quantised (in the room of its sums), then FC2
  if (unit_rows(&M.c1, true) == 256 && unit_rows(&M.c2, true) == 256 && cfg->inter % kFp8Block == 0) {
    uint8_t* h_codes = ws + M.fc1;
    float* h_scales = reinterpret_cast<float*>(h_codes + align_up((size_t)M.c2.m * cfg->inter, 256));
    if ((st = quantize_and_make_h(&M.c1, &M.c2, x, sorted, offsets, w13, s13, ws + M.quant, h_codes, h_scales, status, sms,
                                  s)) != B4_OK ||
        (st = launch_product(&M.c2, h_codes, h_scales, w2, s2, offsets, sorted, y, status, true, sms, s)) != B4_OK)
      return st;
    return combine(cfg, y, topk_ids, topk_weights, out, s);
  }
  // FC1: gather x rows of the packed routes, quantise, multiply by W13
  if ((st = quantize_and_multiply(&M.c1, x, sorted, offsets, w13, s13, nullptr, fc1, ws + M.quant, status, status, sms,
                                  s)) != B4_OK)
    return st;
  // FC2: activation and quantisation of the FC1 rows, product stored in route order
  if ((st = quantize_and_multiply(&M.c2, fc1, nullptr, offsets, w2, s2, sorted, y, ws + M.quant, nullptr, status, sms,
                                  s)) != B4_OK)
    return st;
  return combine(cfg, y, topk_ids, topk_weights, out, s);
}

}  // extern "C"
