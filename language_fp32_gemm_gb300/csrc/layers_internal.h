// Launch interface between the C ABI of the layer operators (layers.cu) and
// their kernels.  Not installed; not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/phobos_layers.h"

namespace phobos {

// Lets `kernel` use `bytes` of dynamic shared memory on the current device; asked
// of the CUDA runtime once per kernel and device.  The library's lock is held.
cudaError_t allow_shared_memory(const void *kernel, int bytes);

// One operand of a product: `rows` vectors along the contraction.  kmajor:
// element (row, k) at row * ld + k, otherwise at k * ld + row.
struct Operand {
  const void *ptr;
  int64_t ld;
  int kmajor;
};

// What follows the sum s_ij of a product: z = s * scales + bias_j; out =
// act(z) + residual.  All pointers are row-major M x N with unit column stride.
struct Epilogue {
  int type;  // of bias, residual, preact and out
  int act;
  int vec;   // groups of four columns of every matrix here are aligned for vector access
  const void *bias;
  const void *residual;
  void *preact, *out;
  int64_t residual_ld, preact_ld, out_ld;
  const float *row_scale, *col_scale;  // both or neither
  const int *row_exp, *col_exp;        // powers of two, both or neither
};

// C[M][N] = epilogue(sum_k a_ik b_jk)
struct LinearArgs {
  int M, N, K;
  int type;  // of a and b
  Operand a, b;
  Epilogue e;
};

// CUDA-core product: any strides and alignment.  kslices (1..8) CTAs of one
// cluster share the contraction of a tile.
struct SimtArgs {
  LinearArgs l;
  int vec_a, vec_b;  // groups of four elements along the operand's unit stride are aligned
  int kslices;
};
cudaError_t launch_linear_simt(const SimtArgs &a, cudaStream_t stream);
cudaError_t launch_linear_ffma(const SimtArgs &a, cudaStream_t stream);  // F32 only
// F32, at most 16 rows of x, both operands aligned (vec_a, vec_b), x along the
// contraction; chooses its own kslices.
cudaError_t launch_linear_gemv(const SimtArgs &a, int sm_count, cudaStream_t stream);
// 16-bit or 8-bit, at most 16 rows of x, both operands along the contraction with
// rows aligned to 16 bytes.
cudaError_t launch_linear_token(const LinearArgs &l, int sm_count, cudaStream_t stream);

// Tensor-core product.  Operand vectors along the tile's rows (tensor memory
// lanes) and columns; the output is row-major with the rows of `row` as its rows,
// or transposed (`swap`): the rows of `col` as its rows.
struct TcLinearArgs {
  CUtensorMap row[2], col[2];  // with two passes' second terms in [1]
  // Boxes of the epilogue (see kEpilogueBox), where every matrix of it can be
  // reached by TMA (`tma`).
  CUtensorMap residual, preact, out;
  int tma;
  int type;                    // F16, BF16 or E4M3
  int row_kmajor, col_kmajor;
  int tiles_r, tiles_c, group;  // tiles along rows and columns; rows per raster group
  int k_blocks;                 // 128 bytes of the contraction each
  int promote_blocks;           // blocks per partial sum in tensor memory
  // Tiles [0, full_tiles) are whole work items; each later tile is cut along the
  // contraction into `pieces` items.
  int full_tiles, items, pieces;
  float *partials;
  unsigned *counters;  // zero between launches
  int M, N;  // of the output
  Epilogue e;
  int *err;
  int withhold_first_load;  // testing only: the first load is skipped
};
// One kernel: bn columns a tile; pair: 256 rows on a CTA pair (bn 256), else 128;
// split: both operands are sums of two fp16 terms.
struct TcShapeId {
  int bn;
  bool pair, split, swap;
};
// Epilogue blocks in shared memory: 2048 bytes.  As computed (a lane per output
// row): 32 rows of 64 bytes, 64-byte swizzle.  Transposed (a lane per output
// column): 32 columns, 32 rows of a 16-bit or 16 of a 32-bit type.
constexpr int kEpilogueBox = 2048;
cudaError_t launch_linear_tc(const TcLinearArgs &a, const TcShapeId &id, int units, cudaStream_t stream);
// Partial-sum floats and counters of one piece of a tile.
inline int64_t tc_partial_floats(const TcShapeId &id) { return (id.pair ? 256 : 128) * static_cast<int64_t>(id.bn); }
inline int tc_counters(const TcShapeId &id) { return !id.pair ? 4 : id.split ? 16 : 32; }

// Prepares an operand for the tensor-core kernel: a copy with aligned rows, or
// (split) its rows scaled by 2^-exp as sums of two fp16 terms.  The layout stays.
struct PrepArgs {
  Operand in;
  int rows, k;
  int type;
  int vec;      // groups of four input elements are aligned
  void *hi, *lo;  // lo: split only
  int64_t ld;     // of hi and lo, elements, a multiple of 16 bytes
  int *exp;       // split only: [rows]
};
cudaError_t launch_copy(const PrepArgs &a, int sm_count, cudaStream_t stream);
// One launch: both operands (`second` may be null) lie along the contraction, or neither.
cudaError_t launch_split(const PrepArgs &first, const PrepArgs *second, int sm_count, cudaStream_t stream);

// dz = dout * act'(z), and sums of dz over strips of rows.
struct DzArgs {
  int M, N;
  int type, act;
  const void *dout;
  int64_t dout_ld;
  const void *z;  // null: act is the identity
  int64_t z_ld;
  void *dz;       // [M][dz_ld], null: not stored
  int64_t dz_ld;
  float *partial;  // [strips][N], null: no sums
  int strips, strip_rows;
  int vec;
};
cudaError_t launch_dz(const DzArgs &a, cudaStream_t stream);
// out_j (+)= sum_s partial[s][j], s ascending.
cudaError_t launch_column_sums(const float *partial, int strips, int N, void *out, int type,
                               int accumulate, cudaStream_t stream);

struct NormArgs {
  int rows, cols;
  int type;
  int q8;
  float eps;
  const void *x, *residual, *weight;
  int64_t x_ld, residual_ld;
  void *sum, *out;
  int64_t sum_ld, out_ld;
  float *scale;
  int vec, vec_out;  // 16-byte groups of the inputs, of the outputs are aligned
};
cudaError_t launch_rmsnorm(const NormArgs &a, int sm_count, cudaStream_t stream);

struct NormBackwardArgs {
  int rows, cols;
  int type;
  float eps;
  const void *dy, *h, *weight, *dsum;
  int64_t dy_ld, h_ld, dsum_ld;
  void *dx;
  int64_t dx_ld;
  float *partial;  // [strips][cols] sums of dy n, null: not wanted
  int strips;
  int vec, vec_out;  // 16-byte groups of the inputs, of dx are aligned
};
// CTAs per SM that run at once.
int rmsnorm_backward_ctas(const NormBackwardArgs &a);
cudaError_t launch_rmsnorm_backward(const NormBackwardArgs &a, cudaStream_t stream);

}  // namespace phobos
