// extern "C" entry points of the FP4 x FP4 operators (b4_fp4_* and
// b4_fused_moe_a4 in b4moe.h): argument validation, workspace carve-up and
// launches.  Every launch goes to the caller's stream; nothing here allocates
// or synchronises.

#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "b4moe.h"
#include "fp4.cuh"
#include "fp4_ptx.cuh"

namespace b4 {
void set_last_error(const char* fmt, ...);
b4_status require_device(int* sms);
cudaError_t launch_fp4_quantize(const Fp4QuantParams& p, int dtype, int num_sms, bool pdl, cudaStream_t stream);
cudaError_t launch_fp4_tile_scales(const uint8_t* src, uint8_t* dst, int groups, int m, int blocks, int k_tiles,
                                   int num_sms, cudaStream_t stream);
cudaError_t launch_fp4_combine(const Fp4CombineParams& p, cudaStream_t stream);
cudaError_t launch_fp4_gemm(const Fp4GemmParams& p, int fmt, int grid, int splits, bool pdl, cudaStream_t stream);
cudaError_t launch_fp4_gemm_direct(const Fp4GemmParams& p, int fmt, int grid, int splits, bool pdl, cudaStream_t stream);
cudaError_t launch_fp4_gemm_pair(const Fp4GemmParams& p, int fmt, int nr, int pairs, int rounds, bool pdl,
                                 cudaStream_t stream);
}  // namespace b4

using namespace b4;

namespace {

#define FP4_FAIL(st, ...)        \
  do {                           \
    set_last_error(__VA_ARGS__); \
    return st;                   \
  } while (0)
#define FP4_INVALID(...) FP4_FAIL(B4_ERR_INVALID_ARGUMENT, __VA_ARGS__)

b4_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return B4_OK;
  set_last_error("%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return B4_ERR_CUDA;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

int dtype_bytes(int dtype) { return dtype == B4_DTYPE_F32 ? 4 : 2; }

b4_status check(const b4_fp4_config* c) {
  if (!c) FP4_INVALID("cfg is NULL");
  if (c->m < 0 || c->m > (1 << 25)) FP4_INVALID("m = %d not in [0, 2^25]", c->m);
  if (c->num_groups < 1 || c->num_groups > B4_MAX_LOCAL_EXPERTS)
    FP4_INVALID("num_groups = %d not in [1, %d]", c->num_groups, B4_MAX_LOCAL_EXPERTS);
  if (c->format != B4_NVFP4_E4M3_K16 && c->format != B4_MXFP4_E8M0_K32) FP4_INVALID("format = %d unknown", c->format);
  const int g = fp4_group(c->format);
  if (c->k < g || c->k % g || c->k > (1 << 16))
    FP4_INVALID("k = %d must be a positive multiple of %d (<= 65536)", c->k, g);
  if (c->x_dtype < B4_DTYPE_BF16 || c->x_dtype > B4_DTYPE_F32) FP4_INVALID("x_dtype = %d unknown", c->x_dtype);
  if (c->out_dtype < B4_DTYPE_BF16 || c->out_dtype > B4_DTYPE_F32) FP4_INVALID("out_dtype = %d unknown", c->out_dtype);
  if (c->activation < -1 || c->activation > B4_ACT_SWIGLU_OAI) FP4_INVALID("activation = %d unknown", c->activation);
  if (c->activation == B4_ACT_SWIGLU_OAI &&
      (!std::isfinite(c->swiglu_alpha) || !std::isfinite(c->swiglu_beta) || !(c->swiglu_limit > 0.0f)))
    FP4_INVALID("swiglu_alpha = %g and swiglu_beta = %g must be finite and swiglu_limit = %g positive",
                (double)c->swiglu_alpha, (double)c->swiglu_beta, (double)c->swiglu_limit);
  if (c->gs_mode < B4_FP4_GS_NONE || c->gs_mode > B4_FP4_GS_TENSOR) FP4_INVALID("gs_mode = %d unknown", c->gs_mode);
  if ((c->format == B4_MXFP4_E8M0_K32) != (c->gs_mode == B4_FP4_GS_NONE))
    FP4_INVALID("gs_mode = %d: MXFP4 takes no global scale (B4_FP4_GS_NONE) and NVFP4 needs one", c->gs_mode);
  if (c->scale_layout != B4_FP4_SCALES_TILED && c->scale_layout != B4_FP4_SCALES_ROWS)
    FP4_INVALID("scale_layout = %d unknown", c->scale_layout);
  if (c->row_div < 1) FP4_INVALID("row_div = %d must be positive", c->row_div);
  const bool gated = c->activation == B4_ACT_SILU_SWIGLU || c->activation == B4_ACT_SWIGLU_OAI;
  const int64_t cols = gated ? 2 * (int64_t)c->k : c->k;
  if (c->x_stride != 0 && c->x_stride < cols) FP4_INVALID("x_stride = %lld below the row's %lld elements",
                                                          (long long)c->x_stride, (long long)cols);
  if (c->x_rows < 0) FP4_INVALID("x_rows = %d negative", c->x_rows);
  return B4_OK;
}

b4_status check_n(const b4_fp4_config* c) {
  if (c->n < 1 || c->n > (1 << 20)) FP4_INVALID("n = %d not in [1, 2^20]", c->n);
  if ((int64_t)c->n * c->num_groups > INT_MAX - 128) FP4_INVALID("n x num_groups = %lld exceeds the row index",
                                                                 (long long)c->n * c->num_groups);
  if (c->out_stride != 0 && c->out_stride < c->n) FP4_INVALID("out_stride = %lld below n = %d",
                                                              (long long)c->out_stride, c->n);
  return B4_OK;
}

// Rows of the activation operand and its scale tiles.  Ragged operands need
// m / 128 + E row tiles, stacks E ceil(m / 128); a workspace serves either.
int64_t operand_rows(const b4_fp4_config* c, bool ragged) { return ragged ? c->m : (int64_t)c->m * c->num_groups; }
int64_t operand_tiles(const b4_fp4_config* c, bool ragged) {
  return ragged ? c->m / 128 + c->num_groups : (int64_t)cdiv(c->m, 128) * c->num_groups;
}

b4_status check_rows(const b4_fp4_config* c, bool ragged) {
  if (operand_rows(c, ragged) > INT_MAX - 256) FP4_INVALID("%lld rows exceed the row index",
                                                           (long long)operand_rows(c, ragged));
  return B4_OK;
}

GluParams glu_of(const b4_fp4_config* c) {
  return c->activation == B4_ACT_SWIGLU_OAI ? GluParams{c->swiglu_alpha, c->swiglu_beta, c->swiglu_limit}
                                            : GluParams{1.0f, 0.0f, INFINITY};
}

Fp4QuantParams quant_params(const b4_fp4_config* c, const void* x, const int32_t* rows, const int32_t* offsets,
                            float* gs, uint8_t* codes, uint8_t* scales) {
  Fp4QuantParams p{};
  const bool gated = c->activation == B4_ACT_SILU_SWIGLU || c->activation == B4_ACT_SWIGLU_OAI;
  p.x = x;
  p.x_stride = c->x_stride ? c->x_stride : (gated ? 2 * (int64_t)c->k : c->k);
  p.rows = rows;
  p.row_div = c->row_div;
  p.x_rows = c->x_rows;
  p.offsets = offsets;
  p.groups = c->num_groups;
  p.m = c->m;
  p.k = c->k;
  p.fmt = c->format;
  p.act = c->activation < 0 ? -1 : gated ? 0 : 1;
  p.glu = glu_of(c);
  p.gs_mode = c->gs_mode;
  p.gs = gs;
  p.codes = codes;
  p.ld = fp4_ld(c->k);
  p.scales = scales;
  p.rowmajor_scales = c->scale_layout == B4_FP4_SCALES_ROWS;
  p.k_tiles = fp4_k_tiles(c->k, c->format);
  const int64_t pitch = p.x_stride * dtype_bytes(c->x_dtype);
  p.vec = aligned(x, 32) && pitch % 32 == 0 ? 2 : aligned(x, 16) && pitch % 16 == 0 ? 1 : 0;
  return p;
}

// Activation rows of a unit: 64 (fp4_gemm.cuh, one SM a unit), 128 or 256
// (fp4_gemm_pair.cu, a pair of SMs).  Dense: 64 where that makes one round of the SMs,
// else by the rounds of the pairs, one with 128 rows taken as 0.7 of one with 256.
// Measured in us at 64 / 128 / 256: N = K = 4096 m = 256 8.1 / 8.7 / 10.5, m = 512 13.3 / 9.0 / 10.7,
// m = 1024 23 / 13.3 / 11.3; N = 2048 K = 1408 m = 512 5.1 / 6.3 / 7.8, m = 1024 7.4 / 6.5 / 7.9;
// N = 11264 K = 4096 m = 384 - / 14.2 / 18.0, m = 512 - / 17.7 / 17.1.  Ragged groups take the
// unit by their mean, which popular experts exceed (64 groups N = 2816 K = 2048, popularities
// spread by e^N(0, 1/2), or e^N(0, 1) up to a mean of 24): mean 8 36.4 / 36.1, 24 39.8 / 38.5, 40 41.4 /
// 40.1 / 42.0, 64 50.1 / 41.1 / 44.1, 96 65 / 45.7 / 44.8, 112 71 / 47.5 / 45.5, 144 87 / 52.2 / 48.3; without
// the spread 64 49.8 / 42.0 / 43.1, 96 65 / 43.6 / 45.0, 112 68 / 44.4 / 45.8; 28 MXFP4 groups N = K =
// 2880 mean 16 23.4 / 26.0, 32 26.3 / 27.4, 64 33.7 / 28.1 / 30.5, 112 44 / 31.3 / 31.6, 128 48 / 34.8 / 33.1.
// The mean alone decides, for every N, K and format: of these series it is 4 % off the best at
// MXFP4 mean 32 and 3 % at NVFP4 mean 112 without the spread.
int unit_rows(const b4_fp4_config* c, bool ragged, int sms) {
  const int64_t groups = c->num_groups;
  if (ragged) {  // the rows of a group are known on the device: their mean
    const int64_t per = c->m / groups;
    return per <= 16 ? 64 : per <= 104 ? 128 : 256;
  }
  if (c->m <= 64 || groups * cdiv(c->m, 64) * cdiv(c->n, 128) <= sms) return 64;
  auto rounds = [&](int nt) { return (groups * cdiv(c->m, nt) * cdiv(c->n, 256) + sms / 2 - 1) / (sms / 2); };
  return 7 * rounds(128) < 10 * rounds(256) ? 128 : 256;
}

// CTAs that share a unit along K where the units are fewer than the SMs.  A CTA
// keeps at least three stages (of 256 K), more where its partial sums are larger
// (16 rows a part): N = K = 4096 in us at 1 / 2 / 4 / 8 CTAs a unit, m = 1: 9.2 / 7.7 /
// 7.0 / 7.1, m = 32: 9.3 / 8.4 / 8.0 / 8.0, m = 64: 9.7 / 9.4 / 10.6; K = 2048, N = 8192,
// m = 64: 7.5 / 8.3.
int k_splits(const b4_fp4_config* c, int64_t units, int sms) {
  const int stages = cdiv(c->k, 256);
  const int parts = cdiv(c->m < 64 ? c->m : 64, 16);
  const int least = 2 * parts - 1 > 3 ? 2 * parts - 1 : 3;
  int splits = 8;
  while (splits > 1 && (splits * units > sms || stages < least * splits ||
                        (splits - 1) * parts * 8 * 1024 > kSplitPartBytes))
    splits /= 2;
  return splits;
}

// Most units a call can have: a group ends at most one unit early, and holds at
// least one row.
int64_t most_units(const b4_fp4_config* c, bool ragged, int nt) {
  int64_t tok = (int64_t)cdiv(c->m, nt) * c->num_groups;
  if (ragged) tok = c->m / nt + c->num_groups < c->m ? c->m / nt + c->num_groups : c->m;
  return tok * cdiv(c->n, nt == 64 ? 128 : 256);
}

// The fields of a product that do not depend on where its activations come from.
Fp4GemmParams product_params(const b4_fp4_config* c, const uint8_t* w_scales, const float* w_gs, const int32_t* offsets,
                             const int32_t* out_rows, void* out, uint32_t* status) {
  Fp4GemmParams p{};
  p.w_scales = w_scales;
  p.w_gs = w_gs;
  p.groups = c->num_groups;
  p.m = c->m;
  p.n = c->n;
  p.k = c->k;
  p.offsets = offsets;
  p.out_rows = out_rows;
  p.out_rows_end = (int)operand_rows(c, offsets);
  p.out = out;
  p.out_stride = c->out_stride ? c->out_stride : c->n;
  p.out_dtype = c->out_dtype;
  const int per16 = 16 / dtype_bytes(c->out_dtype);
  p.vec = aligned(out, 16) && p.out_stride % per16 == 0 && c->n % per16 == 0;
  p.status = status;
  return p;
}

// K splits of a direct product (0: the call takes the two launches): few rows, every
// unit has a CTA or a cluster of its own, and a CTA's part of the quantised rows fits
// in shared memory.  One launch saves 2 us of the caller's time; on the GPU alone
// (N = K = 4096) it takes 6.6 / 6.9 / 7.3 / 8.6 us for 1 / 2 / 4 / 8 rows of a unit where
// two launches take 7.0.  A ragged call of 8 rows has them in a unit only if all chose
// the same expert; 8 rows in 8 groups take 10.4 (two launches 10.7, 128 experts, N 1408, K 2048).
int direct_splits(const b4_fp4_config* c, bool ragged, int sms) {
  if (c->m > (ragged ? kDirectRows : kDirectDenseRows)) return 0;
  const int64_t units = most_units(c, ragged, 64);
  if (units > sms) return 0;
  const int splits = k_splits(c, units, sms);
  return cdiv(cdiv(c->k, 256), splits) <= fp4_direct_stages(splits > 1) ? splits : 0;
}

b4_status launch_direct(const b4_fp4_config* c, const Fp4QuantParams& q, const uint8_t* w_codes, const uint8_t* w_scales,
                        const float* w_gs, const int32_t* out_rows, void* out, uint32_t* clear, uint32_t* status,
                        int splits, cudaStream_t stream) {
  Fp4GemmParams p = product_params(c, w_scales, w_gs, q.offsets, out_rows, out, status);
  if (!make_tmap_bytes_2d(&p.tmap_w, w_codes, (uint64_t)c->n * c->num_groups, c->k / 2, (uint64_t)fp4_ld(c->k), 128))
    FP4_FAIL(B4_ERR_CUDA, "cuTensorMapEncodeTiled rejected an operand map");
  p.q = q;
  p.x_dtype = c->x_dtype;
  p.clear_status = clear != nullptr;
  return cuda_status(launch_fp4_gemm_direct(p, c->format, (int)most_units(c, q.offsets, 64), splits, true, stream),
                     "fp4 product");
}

b4_status launch_product(const b4_fp4_config* c, const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gs,
                         const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs, const int32_t* offsets,
                         const int32_t* out_rows, void* out, uint32_t* status, bool a_is_new, int sms,
                         cudaStream_t stream) {
  const bool ragged = offsets != nullptr;
  Fp4GemmParams p = product_params(c, w_scales, w_gs, offsets, out_rows, out, status);
  const int nt = unit_rows(c, ragged, sms);
  const uint64_t ld = (uint64_t)fp4_ld(c->k);
  if (!make_tmap_bytes_2d(&p.tmap_w, w_codes, (uint64_t)c->n * c->num_groups, c->k / 2, ld, 128) ||
      !make_tmap_bytes_2d(&p.tmap_a, a_codes, (uint64_t)operand_rows(c, ragged), c->k / 2, ld,
                          nt == 64 ? 32 : nt / 4))
    FP4_FAIL(B4_ERR_CUDA, "cuTensorMapEncodeTiled rejected an operand map");
  p.a_scales = a_scales;
  p.a_gs = a_gs;
  p.a_gs_per_row = c->gs_mode == B4_FP4_GS_ROW;
  p.a_is_new = a_is_new;
  const int64_t units = most_units(c, ragged, nt);
  if (units > (1 << 30)) FP4_INVALID("too many units of work: m, n and num_groups too large together");
  if (nt == 64) {
    const int splits = k_splits(c, units, sms);
    const int grid = (int)(splits > 1 || units < sms ? units : sms);
    return cuda_status(launch_fp4_gemm(p, c->format, grid, splits, a_is_new, stream), "fp4 product");
  }
  const uint64_t k_tiles = (uint64_t)fp4_k_tiles(c->k, c->format);
  const uint32_t box = (uint32_t)(c->format == B4_NVFP4_E4M3_K16 ? 4 : 2);
  if (!make_tmap_tiles(&p.tmap_ws, w_scales, (uint64_t)cdiv(c->n, 128) * c->num_groups * k_tiles, box) ||
      !make_tmap_tiles(&p.tmap_as, a_scales, (uint64_t)operand_tiles(c, ragged) * k_tiles, box))
    FP4_FAIL(B4_ERR_CUDA, "cuTensorMapEncodeTiled rejected a scale map");
  const int pairs = (int)(units < sms / 2 ? units : sms / 2);
  // the last round's units in halves, where a round holds them: N = K = 4096, 4096 rows 28.7 us
  // for 30.6, 5120 rows 34.7 for 36.4; N = 2048, K = 1408, 2560 rows 9.4 for 10.8
  const int64_t left = units % pairs;
  const bool even = (c->m + 127) / 128 % 2 == 0;  // every unit has a second half
  p.halves_from = (int)(2 * left <= pairs && even ? units - left : units);
  return cuda_status(
      launch_fp4_gemm_pair(p, c->format, nt, pairs, cdiv((int)units, pairs), a_is_new, stream), "fp4 product");
}

// Workspace of b4_fp4_linear: the quantised activation operand (m rows, dense or
// ragged).
struct LinearWs {
  size_t status, codes, scales, gs, total;
};

LinearWs linear_ws(const b4_fp4_config* c) {
  LinearWs L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  L.status = take(256);
  L.codes = take((size_t)c->m * fp4_ld(c->k));
  L.scales = take((size_t)operand_tiles(c, true) * fp4_k_tiles(c->k, c->format) * kSfTile);
  L.gs = take(sizeof(float) * (size_t)c->m);
  L.total = off;
  return L;
}

// Quantise and multiply: one launch for a few rows, else one into `ws` and one that
// is a programmatic dependent of it.
b4_status quantize_and_multiply(const b4_fp4_config* c, const void* x, const float* x_gs, const int32_t* rows,
                                const int32_t* offsets, const uint8_t* w_codes, const uint8_t* w_scales,
                                const float* w_gs, const int32_t* out_rows, void* out, uint8_t* ws, uint32_t* clear,
                                uint32_t* status, int sms, cudaStream_t stream) {
  const LinearWs L = linear_ws(c);
  uint8_t* codes = ws + L.codes;
  uint8_t* scales = ws + L.scales;
  float* gs = c->gs_mode == B4_FP4_GS_ROW ? reinterpret_cast<float*>(ws + L.gs) : const_cast<float*>(x_gs);
  Fp4QuantParams q = quant_params(c, x, rows, offsets, gs, codes, scales);
  if (const int splits = direct_splits(c, offsets, sms))
    return launch_direct(c, q, w_codes, w_scales, w_gs, out_rows, out, clear, status, splits, stream);
  q.status = clear;
  cudaError_t e = launch_fp4_quantize(q, c->x_dtype, sms, true, stream);
  if (e != cudaSuccess) return cuda_status(e, "fp4 quantise");
  return launch_product(c, codes, scales, gs, w_codes, w_scales, w_gs, offsets, out_rows, out, status, true, sms,
                        stream);
}

b4_status check_weights(const b4_fp4_config* c, const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs) {
  if (!w_codes || !w_scales) FP4_INVALID("null weight pointer");
  const bool nv = c->format == B4_NVFP4_E4M3_K16;
  if (nv && !w_gs) FP4_INVALID("NVFP4 weights need their global scales");
  if (!nv && w_gs) FP4_INVALID("MXFP4 takes no global scale (pass NULL)");
  if (!aligned(w_codes, 16) || !aligned(w_scales, 16) || (w_gs && !aligned(w_gs, 4)))
    FP4_INVALID("weight codes and scales must be 16-byte aligned");
  return B4_OK;
}

// W4A4 layer: the shapes of its two products and its workspace.
struct MoeA4 {
  b4_fp4_config c1, c2;
  int r_cap, t_cap, n1;
  size_t status, counts, offsets, sorted, quant, fc1, y, total;
};

b4_status moe_a4_plan(const b4_moe_config* cfg, int32_t activation, MoeA4* M) {
  if (b4_workspace_bytes(cfg, activation) == 0) return B4_ERR_INVALID_ARGUMENT;  // the shared checks; the reason is set
  const bool gated = activation != B4_ACT_RELU2;
  M->t_cap = b4_route_capacity_tokens(cfg->m);
  M->r_cap = M->t_cap * cfg->top_k;
  M->n1 = gated ? 2 * cfg->inter : cfg->inter;
  b4_fp4_config c{};
  c.m = cfg->m * cfg->top_k;
  c.num_groups = cfg->num_local_experts;
  c.format = cfg->format;
  c.x_dtype = c.out_dtype = B4_DTYPE_BF16;
  c.gs_mode = cfg->format == B4_NVFP4_E4M3_K16 ? B4_FP4_GS_ROW : B4_FP4_GS_NONE;
  c.row_div = 1;
  c.activation = -1;
  M->c1 = M->c2 = c;
  M->c1.n = M->n1;
  M->c1.k = cfg->hidden;
  M->c1.row_div = cfg->top_k;
  M->c1.x_rows = cfg->m;
  M->c2.n = cfg->hidden;
  M->c2.k = cfg->inter;
  M->c2.activation = activation;
  M->c2.swiglu_alpha = cfg->swiglu_alpha;
  M->c2.swiglu_beta = cfg->swiglu_beta;
  M->c2.swiglu_limit = cfg->swiglu_limit;
  b4_fp4_config cap1 = M->c1, cap2 = M->c2;  // sizes depend on m only through its capacity
  cap1.m = cap2.m = M->r_cap;
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
  M->sorted = take(sizeof(int32_t) * (size_t)M->r_cap);
  M->quant = take(L1.total > L2.total ? L1.total : L2.total);  // x's rows, then h's
  M->fc1 = take(sizeof(uint16_t) * (size_t)M->r_cap * M->n1);
  M->y = take(sizeof(uint16_t) * (size_t)M->r_cap * cfg->hidden);
  M->total = off;
  return B4_OK;
}

}  // namespace

extern "C" {

size_t b4_fp4_codes_bytes(const b4_fp4_config* cfg, int32_t ragged) {
  if (check(cfg) != B4_OK) return 0;
  return (size_t)operand_rows(cfg, ragged) * fp4_ld(cfg->k);
}

size_t b4_fp4_scale_bytes(const b4_fp4_config* cfg, int32_t ragged) {
  if (check(cfg) != B4_OK) return 0;
  if (cfg->scale_layout == B4_FP4_SCALES_ROWS)
    return (size_t)operand_rows(cfg, ragged) * (cfg->k / fp4_group(cfg->format));
  return (size_t)operand_tiles(cfg, ragged) * fp4_k_tiles(cfg->k, cfg->format) * kSfTile;
}

b4_status b4_fp4_quantize(const b4_fp4_config* cfg, const void* x, const int32_t* rows, const int32_t* offsets,
                          float* gs, uint8_t* codes, uint8_t* scales, void* values, b4_stream_t stream) {
  b4_status st = check(cfg);
  if (st != B4_OK) return st;
  if ((st = check_rows(cfg, offsets)) != B4_OK) return st;
  if (cfg->gs_mode == B4_FP4_GS_TENSOR && (rows || offsets))
    FP4_INVALID("one global scale per matrix (B4_FP4_GS_TENSOR) takes neither rows nor offsets");
  if (cfg->m == 0) return B4_OK;
  if ((cfg->gs_mode == B4_FP4_GS_NONE) != (gs == nullptr))
    FP4_INVALID("gs must be given for NVFP4 and NULL for MXFP4");
  if (!x || !codes || !scales) FP4_INVALID("null pointer argument");
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(values, 16))
    FP4_INVALID("codes, scales and values must be 16-byte aligned");
  if (!aligned(x, dtype_bytes(cfg->x_dtype)) || !aligned(gs, 4) || !aligned(rows, 4) || !aligned(offsets, 4))
    FP4_INVALID("misaligned x, gs, rows or offsets");
  int sms = 0;
  if ((st = require_device(&sms)) != B4_OK) return st;
  Fp4QuantParams p = quant_params(cfg, x, rows, offsets, gs, codes, scales);
  p.values = values;
  p.values_vec = aligned(values, 32) ? 2 : 1;
  p.pad_rows = !offsets && !p.rowmajor_scales;
  return cuda_status(launch_fp4_quantize(p, cfg->x_dtype, sms, true, reinterpret_cast<cudaStream_t>(stream)),
                     "fp4 quantise");
}

b4_status b4_fp4_tile_scales(const b4_fp4_config* cfg, const uint8_t* src, uint8_t* dst, b4_stream_t stream) {
  b4_status st = check(cfg);
  if (st != B4_OK) return st;
  if (cfg->scale_layout != B4_FP4_SCALES_TILED) FP4_INVALID("b4_fp4_tile_scales writes tiled scales");
  if (cfg->m == 0) return B4_OK;
  if (!src || !dst) FP4_INVALID("null pointer argument");
  if (!aligned(dst, 16)) FP4_INVALID("dst must be 16-byte aligned");
  int sms = 0;
  if ((st = require_device(&sms)) != B4_OK) return st;
  return cuda_status(launch_fp4_tile_scales(src, dst, cfg->num_groups, cfg->m, cfg->k / fp4_group(cfg->format),
                                            fp4_k_tiles(cfg->k, cfg->format), sms,
                                            reinterpret_cast<cudaStream_t>(stream)),
                     "fp4 scale tiles");
}

b4_status b4_fp4_matmul(const b4_fp4_config* cfg, const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gs,
                        const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs, const int32_t* offsets,
                        const int32_t* out_rows, void* out, uint32_t* device_status, b4_stream_t stream) {
  b4_status st = check(cfg);
  if (st != B4_OK) return st;
  if ((st = check_n(cfg)) != B4_OK) return st;
  if ((st = check_rows(cfg, offsets)) != B4_OK) return st;
  if (cfg->scale_layout != B4_FP4_SCALES_TILED) FP4_INVALID("b4_fp4_matmul takes tiled scales");
  if (cfg->m == 0) return B4_OK;
  if (!a_codes || !a_scales || !out) FP4_INVALID("null pointer argument");
  if ((cfg->gs_mode == B4_FP4_GS_NONE) != (a_gs == nullptr))
    FP4_INVALID("a_gs must be given for NVFP4 and NULL for MXFP4");
  if ((st = check_weights(cfg, w_codes, w_scales, w_gs)) != B4_OK) return st;
  if (!aligned(a_codes, 16) || !aligned(a_scales, 16)) FP4_INVALID("a_codes and a_scales must be 16-byte aligned");
  if (!aligned(out, dtype_bytes(cfg->out_dtype)) || !aligned(a_gs, 4) || !aligned(offsets, 4) ||
      !aligned(out_rows, 4) || !aligned(device_status, 4))
    FP4_INVALID("misaligned out, a_gs, offsets, out_rows or device_status");
  int sms = 0;
  if ((st = require_device(&sms)) != B4_OK) return st;
  return launch_product(cfg, a_codes, a_scales, a_gs, w_codes, w_scales, w_gs, offsets, out_rows, out, device_status,
                        false, sms, reinterpret_cast<cudaStream_t>(stream));
}

size_t b4_fp4_linear_workspace_bytes(const b4_fp4_config* cfg) {
  if (check(cfg) != B4_OK || check_n(cfg) != B4_OK) return 0;
  return linear_ws(cfg).total;
}

b4_status b4_fp4_linear(const b4_fp4_config* cfg, const void* x, const float* x_gs, const int32_t* rows,
                        const int32_t* offsets, const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs,
                        const int32_t* out_rows, void* out, void* workspace, size_t workspace_bytes,
                        b4_stream_t stream) {
  b4_status st = check(cfg);
  if (st != B4_OK) return st;
  if ((st = check_n(cfg)) != B4_OK) return st;
  if (!offsets && cfg->num_groups != 1) FP4_INVALID("num_groups = %d without offsets", cfg->num_groups);
  if (cfg->gs_mode == B4_FP4_GS_TENSOR) FP4_INVALID("b4_fp4_linear takes per-row or given global scales");
  if (cfg->scale_layout != B4_FP4_SCALES_TILED) FP4_INVALID("b4_fp4_linear takes tiled scales");
  if ((cfg->gs_mode == B4_FP4_GS_GIVEN) != (x_gs != nullptr)) FP4_INVALID("x_gs goes with B4_FP4_GS_GIVEN");
  if (cfg->m == 0) return B4_OK;
  if (!x || !out || !workspace) FP4_INVALID("null pointer argument");
  if ((st = check_weights(cfg, w_codes, w_scales, w_gs)) != B4_OK) return st;
  if (!aligned(workspace, 256)) FP4_INVALID("workspace must be 256-byte aligned");
  if (!aligned(x, dtype_bytes(cfg->x_dtype)) || !aligned(out, dtype_bytes(cfg->out_dtype)) || !aligned(x_gs, 4) ||
      !aligned(rows, 4) || !aligned(offsets, 4) || !aligned(out_rows, 4))
    FP4_INVALID("misaligned x, out, x_gs, rows, offsets or out_rows");
  const LinearWs L = linear_ws(cfg);
  if (workspace_bytes < L.total)
    FP4_FAIL(B4_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", workspace_bytes, L.total);
  int sms = 0;
  if ((st = require_device(&sms)) != B4_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* status = reinterpret_cast<uint32_t*>(ws + L.status);
  return quantize_and_multiply(cfg, x, x_gs, rows, offsets, w_codes, w_scales, w_gs, out_rows, out, ws, status, status,
                               sms, reinterpret_cast<cudaStream_t>(stream));
}

size_t b4_fused_moe_a4_workspace_bytes(const b4_moe_config* cfg, int32_t activation) {
  MoeA4 M{};
  return moe_a4_plan(cfg, activation, &M) == B4_OK ? M.total : 0;
}

b4_status b4_fused_moe_a4(const b4_moe_config* cfg, const uint16_t* x, const uint8_t* w13, const uint8_t* s13,
                          const float* gs13, const uint8_t* w2, const uint8_t* s2, const float* gs2,
                          const int32_t* topk_ids, const float* topk_weights, int32_t activation, uint16_t* out,
                          void* workspace, size_t workspace_bytes, b4_stream_t stream) {
  MoeA4 M{};
  b4_status st = moe_a4_plan(cfg, activation, &M);
  if (st != B4_OK) return st;
  if (cfg->hidden % 8) FP4_INVALID("hidden = %d must be a multiple of 8", cfg->hidden);
  if ((st = check(&M.c2)) != B4_OK || (st = check_n(&M.c1)) != B4_OK || (st = check_n(&M.c2)) != B4_OK) return st;
  if (cfg->m == 0) return B4_OK;
  if (!x || !topk_ids || !topk_weights || !out || !workspace) FP4_INVALID("null pointer argument");
  if ((st = check_weights(&M.c1, w13, s13, gs13)) != B4_OK || (st = check_weights(&M.c2, w2, s2, gs2)) != B4_OK)
    return st;
  if (!aligned(x, 16) || !aligned(out, 16)) FP4_INVALID("x and out must be 16-byte aligned");
  if (!aligned(topk_ids, 4) || !aligned(topk_weights, 4)) FP4_INVALID("misaligned topk_ids or topk_weights");
  if (!aligned(workspace, 256)) FP4_INVALID("workspace must be 256-byte aligned");
  if (workspace_bytes < M.total)
    FP4_FAIL(B4_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", workspace_bytes, M.total);
  int sms = 0;
  if ((st = require_device(&sms)) != B4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* status = reinterpret_cast<uint32_t*>(ws + M.status);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + M.offsets);
  int32_t* sorted = reinterpret_cast<int32_t*>(ws + M.sorted);
  uint16_t* fc1 = reinterpret_cast<uint16_t*>(ws + M.fc1);
  uint16_t* y = reinterpret_cast<uint16_t*>(ws + M.y);
  if ((st = b4_route_pack(cfg, topk_ids, reinterpret_cast<int32_t*>(ws + M.counts), offsets, sorted, stream)) != B4_OK)
    return st;
  // FC1: gather x rows of the packed routes, quantise, multiply by W13
  if ((st = quantize_and_multiply(&M.c1, x, nullptr, sorted, offsets, w13, s13, gs13, nullptr, fc1, ws + M.quant,
                                  status, status, sms, s)) != B4_OK)
    return st;
  // FC2: activation and quantisation of the FC1 rows, product stored in route order
  if ((st = quantize_and_multiply(&M.c2, fc1, nullptr, nullptr, offsets, w2, s2, gs2, sorted, y, ws + M.quant,
                                  nullptr, status, sms, s)) != B4_OK)
    return st;
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
  return cuda_status(launch_fp4_combine(cp, s), "fp4 combine");
}

}  // extern "C"
