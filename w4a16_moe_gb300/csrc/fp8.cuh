// Parameter blocks of the FP8 operators (b4_fp8_* and b4_fused_moe_fp8 in b4moe.h):
// E4M3 operands with an fp32 scale per block of 128 along K.
//
// A quantised operand of R rows and K columns is
//   codes   [R][K] bytes of E4M3 (K a multiple of 16, so rows are 16-byte pieces);
//   scales  [R][ceil(K / 128)] fp32 for activation rows, [ceil(R / 128)][ceil(K / 128)]
//           for each weight matrix: the layout in which checkpoints hold them.
#pragma once

#include "fp4.cuh"

namespace b4 {

constexpr int kFp8Block = 128;

struct Fp8QuantParams {
  Fp4QuantParams q;  // source rows, gathering, activation, codes, values, status (scales and gs unused)
  float* scales;
  int kb;            // blocks along K
  int pow2;          // scales are powers of two
};

// Shared memory for the partial sums of a unit that a cluster splits along K: 512 bytes for
// every other CTA and activation row.
constexpr int kFp8PartBytes = 56 * 1024;

// Direct products: rows of a call that the kernel quantises for itself, rows of its operand in
// shared memory, and stages of 128 K of them that a CTA keeps.
constexpr int kFp8DirectRows = 8, kFp8DirectTile = 8;
constexpr int kFp8DirectStages = 64, kFp8DirectSplitStages = 24;

struct Fp8GemmParams {
  CUtensorMap tmap_w;     // weight codes [E N][K], box 128 bytes x 128 rows
  CUtensorMap tmap_a;     // activation codes [rows][K], box 128 bytes x the kernel's rows
  CUtensorMap tmap_out;   // 16-bit outputs [rows][n], box 64 x 32 rows (pair kernel, where out_boxes)
  int out_boxes;
  Fp4GemmParams g;        // groups, sizes, offsets, output, status (operands and scales unused)
  const float* w_scales;  // [E][ceil(N / 128)][kb]
  const float* a_scales;  // [rows][kb]
  int kb;
  int a_vec, w_vec;       // rows of a_scales, of w_scales are 16-byte aligned
  Fp8QuantParams q;       // direct: the rows the kernel quantises for itself
  int x_dtype;
};

}  // namespace b4
