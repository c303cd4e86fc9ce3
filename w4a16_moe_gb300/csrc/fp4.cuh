// Parameter blocks and layout of the FP4 x FP4 (W4A4) operators: block-scaled
// quantisation, the product of two quantised operands, and its form grouped
// by expert with ragged sizes (b4_fp4_* in b4moe.h).
//
// A quantised operand of R rows and K columns is
//   codes   [R][ld] bytes, two E2M1 codes a byte, ld = K/2 rounded up to 16;
//   scales  tiles of 512 bytes, one per 128 rows x 4 scale blocks along K:
//           [row tile][ceil(K / 4g)][row % 32][row / 32 % 4][block % 4], the
//           order in which tcgen05.cp spreads a tile over tensor memory, so the
//           product kernel moves whole tiles and never shuffles scales;
//   gs      fp32 per row or per group (NVFP4 only).
// Group e of a stack of matrices of m rows starts at row tile e ceil(m / 128).
// Group e of a ragged operand (rows offsets[e] .. offsets[e + 1]) starts at row
// tile offsets[e] / 128 + e: the tiles of groups 0 .. e - 1 number at most that
// many (each adds at most one tile to the floor of its rows), so no prefix sum
// over the groups is needed to find them, and m / 128 + E tiles hold any split.
#pragma once

#include <cuda.h>

#include <cstddef>
#include <cstdint>

#include "kernels.cuh"

namespace b4 {

enum Fp4Gs : int { kGsNone = 0, kGsGiven = 1, kGsRow = 2, kGsTensor = 3 };

constexpr int kSfTile = 512;  // bytes of a scale tile: 128 rows x 4 scales

__host__ __device__ constexpr int fp4_group(int fmt) { return fmt == 0 ? 16 : 32; }
__host__ __device__ inline int64_t fp4_ld(int k) { return ((int64_t)k / 2 + 15) / 16 * 16; }
__host__ __device__ inline int fp4_k_tiles(int k, int fmt) { return cdiv(k, 4 * fp4_group(fmt)); }

// Shared memory for the partial sums of a unit that a cluster splits along K: 8 KB
// for every other CTA and 16 activation rows.
constexpr int kSplitPartBytes = 96 * 1024;

// Direct products: rows of a call that the kernel quantises for itself (a ragged call's
// groups share them), rows of its operand in shared memory (the instruction's least N),
// and stages of 256 K of them that a CTA keeps.
constexpr int kDirectRows = 8, kDirectDenseRows = 4, kDirectTile = 16;
__host__ __device__ constexpr int fp4_direct_stages(bool split) { return split ? 6 : 16; }

struct Fp4QuantParams {
  const void* x;
  int64_t x_stride;          // elements between rows
  const int32_t* rows;       // gather: x row = rows[i] / row_div, or null
  int row_div, x_rows;       // x_rows > 0: gathered rows outside [0, x_rows) read as zero
  const int32_t* offsets;    // ragged groups [groups + 1], or null: a stack of m-row matrices
  int groups, m, k;
  int fmt, act;              // act: -1 none, 0 gated, 1 ReLU^2
  GluParams glu;
  int gs_mode;
  float* gs;
  uint8_t* codes;
  int64_t ld;
  uint8_t* scales;
  int rowmajor_scales;       // 1: scales [row][K / g], 0: tiles
  int k_tiles;
  void* values;              // dequantised rows in x's type, [row][K], or null
  int pad_rows;              // also clear the scales of each last row tile's missing rows
  int vec;                   // alignment of x's rows: 2 32 bytes, 1 16 bytes, 0 less
  int values_vec;            // of values: 2 or 1
  uint32_t* status;          // cleared (first kernel of a composite call), or null
};

struct Fp4GemmParams {
  CUtensorMap tmap_w;        // weight codes [E N][K/2] bytes, box 128 x 128 rows
  CUtensorMap tmap_a;        // activation codes [rows][K/2] bytes, box 128 x 32 or 64 rows
  CUtensorMap tmap_ws, tmap_as;  // scale tiles of both (pair kernel)
  const uint8_t* w_scales;
  const uint8_t* a_scales;
  const float* w_gs;         // [E] or null
  const float* a_gs;         // [row] or [E] or null
  int a_gs_per_row;
  int groups, m, n, k;       // m: rows per group (stack) or row capacity (ragged)
  const int32_t* offsets;    // ragged, or null
  const int32_t* out_rows;   // output row of each activation row, or null
  int out_rows_end;          // rows of the operand: entries of out_rows outside [0, this) are dropped
  void* out;
  int64_t out_stride;        // elements
  int out_dtype;             // 0 bf16, 1 f16, 2 f32
  int vec;                   // rows of out are 16-byte aligned and n fills them
  Fp4QuantParams q;          // direct: the rows the kernel quantises for itself
  int x_dtype, clear_status;
  int halves_from;           // dense units of 256 rows from here on are taken as two halves
  int a_is_new;              // the activation operand comes from the kernel before (programmatic launch)
  uint32_t* status;          // or null
};

struct Fp4CombineParams {
  const uint16_t* y;         // [m top_k][H] bf16 in route order
  const int32_t* topk_ids;
  const float* topk_weights;
  const int32_t* expert_map;
  int m, top_k, num_global_experts, num_local_experts, hidden;
  uint16_t* out;             // [m][H] bf16
};

}  // namespace b4
