// The parts of the backward pass of a linear layer that are not products:
//   dz = dout * act'(z), rounded to the operands' type, and
//   dbias_j = sum_i dz_ij of the unrounded values.
//
// The tensor cores take dz as 16-bit operands beside 16-bit x and w, so it is rounded once
// before the two products.  bf16 gradients are then off by 0.0023 of their norm, without
// that rounding 0.0017 (their own); dz as two 16-bit terms would keep it, for two passes
// of both products (354 of the 420 us at 4096 x 8192 x 4096) and twice dz's traffic.
//
// One pass over dout and z does both: a CTA of 256 threads takes 32 groups of
// columns (16 bytes of each matrix a group; single elements where rows are not
// aligned) of a strip of rows, eight rows at a time, sums its columns in registers
// and leaves one fp32 row of sums per strip; a second kernel adds the strips in
// order.  Bound by memory: 2 reads and 1 write of the matrix (bf16 4096 x 8192: 37 us,
// 5.4 TB/s, and 4 for the strips).
#include "epilogue.cuh"
#include "launch.cuh"

namespace phobos {

namespace {

constexpr int kColThreads = 32, kRowThreads = 8;
constexpr int kRowsAhead = 2;  // rows a thread loads before it works on the first

template <int TYPE, int ACT, int V>
__global__ void __launch_bounds__(kColThreads *kRowThreads, 4) dz_kernel(const __grid_constant__ DzArgs a) {
  grid_begin();
  using G = Group<TYPE, V>;
  const int tx = threadIdx.x % kColThreads, ty = threadIdx.x / kColThreads;
  const int col = (blockIdx.x * kColThreads + tx) * V, n = a.N - col;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * a.strip_rows;
  const int64_t r1 = min(static_cast<int64_t>(a.M), r0 + a.strip_rows);
  float sum[V] = {};
  for (int64_t r = r0 + ty; r < r1 && n > 0; r += kRowThreads * kRowsAhead) {
    G d[kRowsAhead], z[kRowsAhead];
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      const int64_t row = r + i * kRowThreads;
      d[i].load(a.dout, row * a.dout_ld + col, row < r1 ? n : 0);
      if (ACT != PHOBOS_ACT_NONE) z[i].load(a.z, row * a.z_ld + col, row < r1 ? n : 0);
    }
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      const int64_t row = r + i * kRowThreads;
      G o;
      float dv[V], zv[V];  // zero outside
      d[i].unpack(dv);
      if (ACT != PHOBOS_ACT_NONE) z[i].unpack(zv);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (ACT != PHOBOS_ACT_NONE) dv[j] *= activate_slope<ACT>(zv[j]);
        sum[j] += dv[j];
      }
      o.pack(dv);
      if (a.dz && row < r1) o.store(a.dz, row * a.dz_ld + col, n);
    }
  }
  if (!a.partial) return;
  __shared__ float sums[kRowThreads][kColThreads * V];
#pragma unroll
  for (int j = 0; j < V; ++j) sums[ty][j * kColThreads + tx] = sum[j];
  __syncthreads();
  // all threads: one or more columns each
  for (int c = threadIdx.x; c < kColThreads * V; c += kColThreads * kRowThreads) {
    float s = sums[0][c];
#pragma unroll
    for (int i = 1; i < kRowThreads; ++i) s += sums[i][c];
    const int64_t at = (blockIdx.x * static_cast<int64_t>(kColThreads) + c % kColThreads) * V + c / kColThreads;
    if (at < a.N) a.partial[static_cast<int64_t>(blockIdx.y) * a.N + at] = s;
  }
}

template <int TYPE>
__global__ void __launch_bounds__(1024) column_sums_kernel(const float *partial, int strips,
                                                           int N, void *out, int accumulate) {
  grid_begin();
  using E = Elem<TYPE>;
  // 32 columns a CTA, 32 interleaved groups of strips
  __shared__ float sums[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t col = blockIdx.x * 32ll + tx;
  float s = 0.f;
  if (col < N) {
#pragma unroll 8
    for (int i = ty; i < strips; i += 32) s += partial[static_cast<int64_t>(i) * N + col];
  }
  sums[ty][tx] = s;
  __syncthreads();
  if (ty != 0 || col >= N) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) s += sums[i][tx];
  typename E::T *p = static_cast<typename E::T *>(out) + col;
  if (accumulate) s += E::load(*p);
  *p = E::store(s);
}

}  // namespace

namespace {

template <int TYPE, int V>
cudaError_t launch_dz_type(const DzArgs &a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.N + kColThreads * V - 1ll) / (kColThreads * V)), a.strips);
  const int threads = kColThreads * kRowThreads;
  switch (a.act) {
    case PHOBOS_ACT_NONE: return launch_kernel(dz_kernel<TYPE, PHOBOS_ACT_NONE, V>, 1, grid, threads, 0, stream, a);
    case PHOBOS_ACT_RELU: return launch_kernel(dz_kernel<TYPE, PHOBOS_ACT_RELU, V>, 1, grid, threads, 0, stream, a);
    case PHOBOS_ACT_GELU: return launch_kernel(dz_kernel<TYPE, PHOBOS_ACT_GELU, V>, 1, grid, threads, 0, stream, a);
    case PHOBOS_ACT_GELU_TANH: return launch_kernel(dz_kernel<TYPE, PHOBOS_ACT_GELU_TANH, V>, 1, grid, threads, 0, stream, a);
    case PHOBOS_ACT_SILU: return launch_kernel(dz_kernel<TYPE, PHOBOS_ACT_SILU, V>, 1, grid, threads, 0, stream, a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_dz(const DzArgs &a, cudaStream_t stream) {
  switch (a.type) {
    case PHOBOS_TYPE_F32:
      return a.vec ? launch_dz_type<PHOBOS_TYPE_F32, 4>(a, stream) : launch_dz_type<PHOBOS_TYPE_F32, 1>(a, stream);
    case PHOBOS_TYPE_F16:
      return a.vec ? launch_dz_type<PHOBOS_TYPE_F16, 8>(a, stream) : launch_dz_type<PHOBOS_TYPE_F16, 1>(a, stream);
    case PHOBOS_TYPE_BF16:
      return a.vec ? launch_dz_type<PHOBOS_TYPE_BF16, 8>(a, stream) : launch_dz_type<PHOBOS_TYPE_BF16, 1>(a, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_column_sums(const float *partial, int strips, int N, void *out, int type,
                               int accumulate, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((N + 31ll) / 32);
  switch (type) {
    case PHOBOS_TYPE_F32:
      return launch_kernel(column_sums_kernel<PHOBOS_TYPE_F32>, 1, grid, 1024, 0, stream, partial, strips, N, out, accumulate);
    case PHOBOS_TYPE_F16:
      return launch_kernel(column_sums_kernel<PHOBOS_TYPE_F16>, 1, grid, 1024, 0, stream, partial, strips, N, out, accumulate);
    case PHOBOS_TYPE_BF16:
      return launch_kernel(column_sums_kernel<PHOBOS_TYPE_BF16>, 1, grid, 1024, 0, stream, partial, strips, N, out, accumulate);
  }
  return cudaErrorInvalidValue;
}

}  // namespace phobos
