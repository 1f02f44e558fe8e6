// Root-mean-square norm of rows, with the residual's addition and an optional
// 8-bit output, and its backward pass:
//   h = x + residual,  y = h rstd w,  rstd = 1 / sqrt(mean(h^2) + eps),
//   q = e4m3(y / s),   s = max|y| / 448;
//   dx = rstd (g - n mean(g n)) + dsum,  n = h rstd,  g = dy w,
//   dweight_j = sum_i dy_ij n_ij.
//
// Bound by memory: a row is read once, in 16-byte groups where the rows allow it,
// and its elements stay in the registers of the 32 .. 1024 threads that share it
// (longer rows are read again).  One round of reduction suffices in every case:
// max|y| = rstd max|h w| needs no second pass after rstd, and the two sums of the
// backward pass, of h^2 and of g h, go together (mean(g n) = rstd mean(g h)).
// Statistics are fp32 sums over threads, lanes and warps in a fixed order.
//
// With many aligned rows a CTA stays and walks its rows: every thread copies its
// own groups of the next one or two rows to shared memory in the background (cp.async)
// while it works on this one, so the bytes in flight do not cost registers.
// (With the loads in registers the 8-bit norm of 8192 x 8192 took 182 us, 2.6 TB/s; in
// the ring 71 with the residual read and the sum written, 6.6 TB/s, the rate of a
// plain copy.  Backward, bf16 8192 x 4096: 47 us, 5.7 TB/s; fp32 3001 x 5003, whose rows
// are not aligned: 49, 4.9 TB/s.  One row of 4096: 2.5 us, its launch and one reduction.)
#include <algorithm>

#include "epilogue.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace phobos {

namespace {

template <int V>
__device__ __forceinline__ void store_q(void *base, int64_t i, int n, bool aligned, const float (&v)[V]) {
  struct alignas(V) Bytes { __nv_fp8_storage_t x[V]; } q;
  if constexpr (V == 1) {
    q.x[0] = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 2)
      reinterpret_cast<__nv_fp8x2_storage_t *>(q.x)[j / 2] =
          __nv_cvt_float2_to_fp8x2(make_float2(v[j], v[j + 1]), __NV_SATFINITE, __NV_E4M3);
  }
  __nv_fp8_storage_t *p = static_cast<__nv_fp8_storage_t *>(base) + i;
  if (n >= V && aligned) {
    *reinterpret_cast<Bytes *>(p) = q;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) p[j] = q.x[j];
  }
}

// Over the THREADS threads of a row (whole warps): the sum of a and the sum (or,
// with MAX, the maximum) of b, to every thread.  scratch: one float2 per warp; a
// caller that comes again alternates between two.
template <int THREADS, bool MAX>
__device__ __forceinline__ void row_reduce(float &a, float &b, int t, float2 *scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    const float w = __shfl_xor_sync(0xffffffffu, b, o);
    b = MAX ? fmaxf(b, w) : b + w;
  }
  if (THREADS == 32) return;
  if ((t & 31) == 0) scratch[t >> 5] = make_float2(a, b);
  __syncthreads();
  float2 s = scratch[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) {
    const float2 x = scratch[w];
    s.x += x.x;
    s.y = MAX ? fmaxf(s.y, x.y) : s.y + x.y;
  }
  a = s.x;
  b = s.y;
}

// y = h rstd w, q = y inv_scale.  Two factors: of a row of small numbers, rstd may be
// 1 / sqrt(eps) and inv_scale 2^126, whose product is not finite.
struct RowFactors {
  float rstd, inv_scale;
};

// From the row's sum of h^2 and largest |h w|; `first` stores the scale.
__device__ __forceinline__ RowFactors row_factors(const NormArgs &a, float ss, float top, int64_t row, bool first) {
  RowFactors f;
  f.rstd = rsqrtf(ss / static_cast<float>(a.cols) + a.eps);
  f.inv_scale = 1.f;
  if (!a.q8) return f;
  const float amax = top * f.rstd;
  // not below the smallest normal number, whose reciprocal is finite
  const float s = amax == 0.f ? 1.f : fmaxf(amax / 448.f, 1.17549435e-38f);
  if (first) a.scale[row] = isnan(ss) ? ss : s;
  f.inv_scale = 1.f / s;
  return f;
}

// Outputs whose rows are not aligned are stored element by element.
template <typename G>
__device__ __forceinline__ void put_group(const G &g, void *base, int64_t i, int n, bool aligned) {
  if (aligned) g.store(base, i, n);
  else g.store_any(base, i, n);
}

template <typename G>
__device__ __forceinline__ void put_normed(const NormArgs &a, int64_t row, int col, const G &h, const G &w,
                                           const RowFactors &f) {
  constexpr int V = G::kSize;
  float v[V], wv[V];
  h.unpack(v);
  w.unpack(wv);
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = v[j] * f.rstd * wv[j];
  if (a.q8) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= f.inv_scale;
    store_q<V>(a.out, row * a.out_ld + col, a.cols - col, a.vec_out, v);
  } else {
    G y;
    y.pack(v);
    put_group(y, a.out, row * a.out_ld + col, a.cols - col, a.vec_out);
  }
}

// h = x + r, rounded to the type it is stored in, so that the norm is that of the
// stored values.
template <typename G>
__device__ __forceinline__ void add_residual(G &h, const G &r) {
  constexpr int V = G::kSize;
  float hv[V], rv[V];
  h.unpack(hv);
  r.unpack(rv);
#pragma unroll
  for (int j = 0; j < V; ++j) hv[j] += rv[j];
  h.pack(hv);
}

// Adds a group to the sum of h^2 and the largest |h w|.
template <typename G>
__device__ __forceinline__ void add_statistics(const G &h, const G &w, float &ss, float &top) {
  constexpr int V = G::kSize;
  float hv[V], wv[V];
  h.unpack(hv);
  w.unpack(wv);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    ss = fmaf(hv[j], hv[j], ss);
    top = fmaxf(top, fabsf(hv[j] * wv[j]));
  }
}

template <typename G>
__device__ __forceinline__ void load_weight(const void *weight, int col, int n, G &w) {
  if (weight) w.load(weight, col, n);
  else w.fill(1.f);
}

// A thread's next column of a row; a step of up to 8192 from within the longest rows
// (2^31 - 1024) passes 2^31, and stops short of it instead.
__device__ __forceinline__ int next_col(int col, int step) {
  return static_cast<int>(min(static_cast<unsigned>(col) + static_cast<unsigned>(step), 0x7fffffffu));
}

template <int TYPE, int V, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS == 32 ? 256 : THREADS)
    rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  grid_begin();
  using G = Group<TYPE, V>;
  __shared__ float2 scratch[THREADS / 32];
  const int t = threadIdx.x % THREADS;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / THREADS) + threadIdx.x / THREADS;
  if (row >= a.rows) return;  // several rows a CTA only where a row is one warp, which meets no barrier
  const int step = THREADS * V;

  auto load_h = [&](int col, int n, G &h) {
    h.load(a.x, row * a.x_ld + col, n);
    if (a.residual) {
      G r;
      r.load(a.residual, row * a.residual_ld + col, n);
      add_residual(h, r);
    }
  };
  G h[ITEMS], w[ITEMS];
  float ss = 0.f, top = 0.f;  // sum of h^2, largest |h w|
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = i * step + t * V;
    load_h(col, a.cols - col, h[i]);
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = i * step + t * V;
    load_weight(a.weight, col, a.cols - col, w[i]);
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = i * step + t * V;
    if (a.sum) put_group(h[i], a.sum, row * a.sum_ld + col, a.cols - col, a.vec_out);
    add_statistics(h[i], w[i], ss, top);
  }
  for (int col = ITEMS * step + t * V; col < a.cols; col = next_col(col, step)) {  // the rest of a longer row
    G hg, wg;
    load_h(col, a.cols - col, hg);
    load_weight(a.weight, col, a.cols - col, wg);
    if (a.sum) put_group(hg, a.sum, row * a.sum_ld + col, a.cols - col, a.vec_out);
    add_statistics(hg, wg, ss, top);
  }
  row_reduce<THREADS, true>(ss, top, t, scratch);
  const RowFactors factors = row_factors(a, ss, top, row, t == 0);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = i * step + t * V;
    put_normed(a, row, col, h[i], w[i], factors);
  }
  for (int col = ITEMS * step + t * V; col < a.cols; col = next_col(col, step)) {
    G hg, wg;
    // What this thread stored: the sum may lie over x or the residual, which then are gone.
    const int64_t at = row * a.sum_ld + col;
    if (!a.sum) hg.load(a.x, row * a.x_ld + col, a.cols - col);
    else if (a.vec_out) hg.load(a.sum, at, a.cols - col);
    else hg.load_any(a.sum, at, a.cols - col);
    load_weight(a.weight, col, a.cols - col, wg);
    put_normed(a, row, col, hg, wg, factors);
  }
}

// ------------------------------------------------------------ rows in a ring

// Copies 16 bytes to shared memory in the background, the last 16 - bytes of them zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)),
               "r"(bytes)
               : "memory");
}

// This thread's groups of TENSORS matrices' rows in a ring.  Only the thread that
// copied a group reads it, so the ring needs no barrier.
template <int TYPE, int ITEMS, int THREADS, int TENSORS>
struct RowRing {
  static constexpr int V = 16 / sizeof(typename Elem<TYPE>::T);
  using G = Group<TYPE, V>;
  static constexpr int kRowBytes = ITEMS * THREADS * 16;
  // Rows in the ring: the current one and the next one or two.  More bytes in flight
  // than the memory needs cost time again (backward of 8192 x 8192: 98 us with one row
  // ahead, 109 with two; norm, of two matrices: 97 and 94, in 8 bits 80 and 73).
  static constexpr int kRows = TENSORS == 2 && 3 * TENSORS * kRowBytes <= 224 * 1024 ? 3 : 2;
  static constexpr int kBytes = kRows * TENSORS * kRowBytes;
  uint32_t base;

  __device__ __forceinline__ uint32_t at(int slot, int tensor, int i) const {
    return base + static_cast<uint32_t>((slot * TENSORS + tensor) * kRowBytes + (i * THREADS + threadIdx.x) * 16);
  }
  __device__ __forceinline__ void copy(int slot, int tensor, const void *matrix, int64_t offset, int cols) const {
    const typename G::T *row = static_cast<const typename G::T *>(matrix) + offset;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int col = (i * THREADS + static_cast<int>(threadIdx.x)) * V;
      const int n = min(V, cols - col);
      copy16(at(slot, tensor, i), n > 0 ? row + col : row, n > 0 ? n * static_cast<int>(sizeof(typename G::T)) : 0);
    }
  }
  __device__ __forceinline__ G get(int slot, int tensor, int i) const {
    G g;
    *reinterpret_cast<float4 *>(&g) = ld_shared_f4(at(slot, tensor, i));
    return g;
  }
};

template <int TYPE, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS >= 512 ? 1 : 512 / THREADS)
    rmsnorm_ring_kernel(const __grid_constant__ NormArgs a) {
  grid_begin();
  using Ring = RowRing<TYPE, ITEMS, THREADS, 2>;
  using G = typename Ring::G;
  constexpr int V = Ring::V;
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  __shared__ float2 scratch[2][THREADS / 32];
  const Ring ring{smem_u32(ring_bytes)};
  const int t = threadIdx.x;
  G w[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = (i * THREADS + t) * V;
    load_weight(a.weight, col, a.cols - col, w[i]);
  }
  auto fetch = [&](int64_t row, int slot) {
    if (row < a.rows) {
      ring.copy(slot, 0, a.x, row * a.x_ld, a.cols);
      if (a.residual) ring.copy(slot, 1, a.residual, row * a.residual_ld, a.cols);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int r = 0; r < Ring::kRows - 1; ++r) fetch(blockIdx.x + static_cast<int64_t>(r) * gridDim.x, r);
  int slot = 0, turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const int free_slot = slot == 0 ? Ring::kRows - 1 : slot - 1;  // the previous row's
    fetch(row + (Ring::kRows - 1) * static_cast<int64_t>(gridDim.x), free_slot);
    cp_async_wait_group<Ring::kRows - 1>();
    G h[ITEMS];
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int col = (i * THREADS + t) * V;
      h[i] = ring.get(slot, 0, i);
      if (a.residual) {
        add_residual(h[i], ring.get(slot, 1, i));
        put_group(h[i], a.sum, row * a.sum_ld + col, a.cols - col, a.vec_out);
      }
      add_statistics(h[i], w[i], ss, top);
    }
    row_reduce<THREADS, true>(ss, top, t, scratch[turn]);
    const RowFactors factors = row_factors(a, ss, top, row, t == 0);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int col = (i * THREADS + t) * V;
      put_normed(a, row, col, h[i], w[i], factors);
    }
    slot = slot + 1 == Ring::kRows ? 0 : slot + 1;
  }
  cp_async_wait_all();
}

// Adds a group to the sums of h^2 and of g h.
template <typename G>
__device__ __forceinline__ void add_sums(const G &h, const G &dy, const G &w, float &ss, float &gh) {
  constexpr int V = G::kSize;
  float hv[V], dv[V], wv[V];
  h.unpack(hv);
  dy.unpack(dv);
  w.unpack(wv);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    ss = fmaf(hv[j], hv[j], ss);
    gh = fmaf(dv[j] * wv[j], hv[j], gh);
  }
}

// rstd (g - n mean) + dsum of a group; adds dy n to `sum`.
template <typename G>
__device__ __forceinline__ G row_gradient(const G &h, const G &dy, const G &w, const G &ds, bool with_ds, float rstd,
                                          float mean, float (&sum)[G::kSize]) {
  constexpr int V = G::kSize;
  float hv[V], dv[V], wv[V], sv[V];
  h.unpack(hv);
  dy.unpack(dv);
  w.unpack(wv);
  if (with_ds) ds.unpack(sv);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float n = hv[j] * rstd;
    sum[j] = fmaf(dv[j], n, sum[j]);
    hv[j] = fmaf(rstd, fmaf(-n, mean, dv[j] * wv[j]), with_ds ? sv[j] : 0.f);
  }
  G o;
  o.pack(hv);
  return o;
}

// A CTA walks the rows blockIdx.x, blockIdx.x + strips, ...; a thread keeps the
// same columns throughout and sums its part of dweight in registers.  Columns
// beyond the registers are summed in the CTA's own row of `partial` instead, which
// only that thread touches.  Rows of one warp: the CTA's eight warps walk rows of
// their own and add their sums at the end.
template <int TYPE, int V, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS == 32 ? 256 : THREADS, THREADS <= 128 ? 4 : 1024 / THREADS)
    rmsnorm_backward_kernel(const __grid_constant__ NormBackwardArgs a) {
  grid_begin();
  using G = Group<TYPE, V>;
  constexpr int kRowsAtOnce = THREADS == 32 ? 8 : 1;
  __shared__ float2 scratch[2][THREADS / 32];
  const int t = threadIdx.x % THREADS;
  const int step = THREADS * V;
  float *const partial = a.partial ? a.partial + static_cast<int64_t>(blockIdx.x) * a.cols : nullptr;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  float dw[ITEMS][V] = {};
  int turn = 0;
  const int64_t first_row = static_cast<int64_t>(blockIdx.x) * kRowsAtOnce + threadIdx.x / THREADS;
  for (int64_t row = first_row; row < a.rows; row += static_cast<int64_t>(a.strips) * kRowsAtOnce, turn ^= 1) {
    G h[ITEMS], dy[ITEMS], ds[ITEMS];
    float ss = 0.f, gh = 0.f;  // sums of h^2 and of g h
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int col = i * step + t * V;
      h[i].load(a.h, row * a.h_ld + col, a.cols - col);
      dy[i].load(a.dy, row * a.dy_ld + col, a.cols - col);
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int col = i * step + t * V;
      if (a.dsum) ds[i].load(a.dsum, row * a.dsum_ld + col, a.cols - col);
    }
    auto sums = [&](int col, const G &hg, const G &dg) {
      G w;
      load_weight(a.weight, col, a.cols - col, w);
      add_sums(hg, dg, w, ss, gh);
    };
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) sums(i * step + t * V, h[i], dy[i]);
    for (int col = ITEMS * step + t * V; col < a.cols; col = next_col(col, step)) {
      G hg, dg;
      hg.load(a.h, row * a.h_ld + col, a.cols - col);
      dg.load(a.dy, row * a.dy_ld + col, a.cols - col);
      sums(col, hg, dg);
    }
    row_reduce<THREADS, false>(ss, gh, t, scratch[turn]);
    const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
    const float mean = gh * rstd * inv_cols;  // of g n
    auto put = [&](int col, const G &hg, const G &dg, const G &sg, float (&sum)[V]) {
      G w;
      load_weight(a.weight, col, a.cols - col, w);
      put_group(row_gradient(hg, dg, w, sg, a.dsum != nullptr, rstd, mean, sum), a.dx, row * a.dx_ld + col,
                a.cols - col, a.vec_out);
    };
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) put(i * step + t * V, h[i], dy[i], ds[i], dw[i]);
    for (int col = ITEMS * step + t * V; col < a.cols; col = next_col(col, step)) {
      G hg, dg, sg;
      float sum[V] = {};
      hg.load(a.h, row * a.h_ld + col, a.cols - col);
      dg.load(a.dy, row * a.dy_ld + col, a.cols - col);
      if (a.dsum) sg.load(a.dsum, row * a.dsum_ld + col, a.cols - col);
      const bool add = partial && row != first_row;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (add && col + j < a.cols) sum[j] = partial[col + j];
      put(col, hg, dg, sg, sum);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (partial && col + j < a.cols) partial[col + j] = sum[j];
    }
  }
  if (!partial) return;
  if constexpr (kRowsAtOnce > 1) {  // no row is longer than the registers
    constexpr int kCols = 32 * V * ITEMS;
    __shared__ float sums[kRowsAtOnce][kCols];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) sums[threadIdx.x / 32][i * step + t * V + j] = dw[i][j];
    }
    __syncthreads();
    for (int col = threadIdx.x; col < a.cols; col += 256) {
      float s = sums[0][col];
#pragma unroll
      for (int w = 1; w < kRowsAtOnce; ++w) s += sums[w][col];
      partial[col] = s;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = i * step + t * V;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (col + j < a.cols) partial[col + j] = dw[i][j];
  }
}

// The same for aligned rows that fit the registers, with rows in a ring.
template <int TYPE, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS >= 512 ? 1 : 512 / THREADS)
    rmsnorm_backward_ring_kernel(const __grid_constant__ NormBackwardArgs a) {
  grid_begin();
  using Ring = RowRing<TYPE, ITEMS, THREADS, 3>;
  using G = typename Ring::G;
  constexpr int V = Ring::V;
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  __shared__ float2 scratch[2][THREADS / 32];
  const Ring ring{smem_u32(ring_bytes)};
  const int t = threadIdx.x;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  G w[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = (i * THREADS + t) * V;
    load_weight(a.weight, col, a.cols - col, w[i]);
  }
  auto fetch = [&](int64_t row, int slot) {
    if (row < a.rows) {
      ring.copy(slot, 0, a.h, row * a.h_ld, a.cols);
      ring.copy(slot, 1, a.dy, row * a.dy_ld, a.cols);
      if (a.dsum) ring.copy(slot, 2, a.dsum, row * a.dsum_ld, a.cols);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int r = 0; r < Ring::kRows - 1; ++r) fetch(blockIdx.x + static_cast<int64_t>(r) * a.strips, r);
  float dw[ITEMS][V] = {};
  int slot = 0, turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += a.strips, turn ^= 1) {
    const int free_slot = slot == 0 ? Ring::kRows - 1 : slot - 1;  // the previous row's
    fetch(row + (Ring::kRows - 1) * static_cast<int64_t>(a.strips), free_slot);
    cp_async_wait_group<Ring::kRows - 1>();
    G h[ITEMS], dy[ITEMS];
    float ss = 0.f, gh = 0.f;  // sums of h^2 and of g h
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      h[i] = ring.get(slot, 0, i);
      dy[i] = ring.get(slot, 1, i);
      add_sums(h[i], dy[i], w[i], ss, gh);
    }
    row_reduce<THREADS, false>(ss, gh, t, scratch[turn]);
    const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
    const float mean = gh * rstd * inv_cols;  // of g n
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int col = (i * THREADS + t) * V;
      G s;
      if (a.dsum) s = ring.get(slot, 2, i);
      put_group(row_gradient(h[i], dy[i], w[i], s, a.dsum != nullptr, rstd, mean, dw[i]), a.dx, row * a.dx_ld + col,
                a.cols - col, a.vec_out);
    }
    slot = slot + 1 == Ring::kRows ? 0 : slot + 1;
  }
  cp_async_wait_all();
  if (!a.partial) return;
  float *const partial = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = (i * THREADS + t) * V;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (col + j < a.cols) partial[col + j] = dw[i][j];
  }
}

// CTAs of a ring kernel on an SM: 512 threads, whose up to 128 registers hold their rows
// without spilling (backward of 8192 x 4096: 54 us, with 768 threads 67, with 1024 81).
constexpr int ring_ctas(int threads, int bytes) {
  const int by_threads = threads >= 512 ? 1 : 512 / threads, by_memory = 227 * 1024 / (bytes + 2048);
  return by_threads < by_memory ? by_threads : by_memory;
}

constexpr int kRingItems = 2;

// A ring kernel's threads for aligned rows of `cols` columns: f(THREADS) with the
// fewest of 128 .. 1024 that hold them, or false.
template <typename F>
bool with_ring_threads(int cols, int per_thread, F f) {
  if (cols <= 32 * per_thread || cols > 1024 * per_thread) return false;
  if (cols <= 128 * per_thread) f(std::integral_constant<int, 128>());
  else if (cols <= 256 * per_thread) f(std::integral_constant<int, 256>());
  else if (cols <= 384 * per_thread) f(std::integral_constant<int, 384>());
  else if (cols <= 512 * per_thread) f(std::integral_constant<int, 512>());
  else if (cols <= 640 * per_thread) f(std::integral_constant<int, 640>());
  else f(std::integral_constant<int, 1024>());
  return true;
}

template <typename Kernel, typename Args>
cudaError_t launch_ring(Kernel kernel, const Args &a, unsigned grid, int threads, int bytes, cudaStream_t stream) {
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void *>(kernel), bytes);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, 1, grid, threads, bytes, stream, a);
}

// f(THREADS) with the fewest of 32, 128, 256, 512, 1024 threads that hold `cols` columns.
template <typename F>
cudaError_t with_threads(int cols, int per_thread, F f) {
  if (cols <= 32 * per_thread) return f(std::integral_constant<int, 32>());
  if (cols <= 128 * per_thread) return f(std::integral_constant<int, 128>());
  if (cols <= 256 * per_thread) return f(std::integral_constant<int, 256>());
  if (cols <= 512 * per_thread) return f(std::integral_constant<int, 512>());
  return f(std::integral_constant<int, 1024>());
}

// f(TYPE, V): groups of 16 bytes, or single elements where rows are not aligned.
template <typename F>
cudaError_t with_groups(int type, int vec, F f) {
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;
  using Eight = std::integral_constant<int, 8>;
  switch (type) {
    case PHOBOS_TYPE_F32: {
      const std::integral_constant<int, PHOBOS_TYPE_F32> t;
      return vec ? f(t, Four()) : f(t, One());
    }
    case PHOBOS_TYPE_F16: {
      const std::integral_constant<int, PHOBOS_TYPE_F16> t;
      return vec ? f(t, Eight()) : f(t, One());
    }
    case PHOBOS_TYPE_BF16: {
      const std::integral_constant<int, PHOBOS_TYPE_BF16> t;
      return vec ? f(t, Eight()) : f(t, One());
    }
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs &a, int sm_count, cudaStream_t stream) {
  return with_groups(a.type, a.vec, [&](auto type, auto v) {
    constexpr int TYPE = decltype(type)::value, V = decltype(v)::value, ITEMS = V == 1 ? 16 : 4;
    if constexpr (V > 1) {
      cudaError_t e = cudaSuccess;
      if (a.rows > 2 * sm_count && with_ring_threads(a.cols, V * kRingItems, [&](auto threads) {
            constexpr int THREADS = decltype(threads)::value;
            constexpr int kBytes = RowRing<TYPE, kRingItems, THREADS, 2>::kBytes;
            const unsigned grid = static_cast<unsigned>(std::min(a.rows, ring_ctas(THREADS, kBytes) * sm_count));
            e = launch_ring(rmsnorm_ring_kernel<TYPE, kRingItems, THREADS>, a, grid, THREADS, kBytes, stream);
          }))
        return e;
    }
    // rows of one warp: eight a CTA, with no more registers than they need
    const unsigned grid8 = static_cast<unsigned>((a.rows + 7ll) / 8);
    if (a.cols <= 32 * V * (ITEMS / 4)) {
      return launch_kernel(rmsnorm_kernel<TYPE, V, ITEMS / 4, 32>, 1, grid8, 256, 0, stream, a);
    }
    if (a.cols <= 32 * V * (ITEMS / 2)) {
      return launch_kernel(rmsnorm_kernel<TYPE, V, ITEMS / 2, 32>, 1, grid8, 256, 0, stream, a);
    }
    return with_threads(a.cols, V * ITEMS, [&](auto threads) {
      constexpr int THREADS = decltype(threads)::value, ROWS = THREADS == 32 ? 8 : 1;
      const unsigned grid = static_cast<unsigned>((a.rows + ROWS - 1ll) / ROWS);
      return launch_kernel(rmsnorm_kernel<TYPE, V, ITEMS, THREADS>, 1, grid, THREADS * ROWS, 0, stream, a);
    });
  });
}

int rmsnorm_backward_ctas(const NormBackwardArgs &a) {
  const int per_thread = (a.vec ? kRingItems * (a.type == PHOBOS_TYPE_F32 ? 4 : 8) : 8);
  int ctas = 4;  // of 256 threads where rows are one warp
  if (a.vec && with_ring_threads(a.cols, per_thread, [&](auto threads) {
        constexpr int THREADS = decltype(threads)::value;
        ctas = ring_ctas(THREADS, RowRing<PHOBOS_TYPE_F32, kRingItems, THREADS, 3>::kBytes);
      }))
    return ctas;
  with_threads(a.cols, per_thread, [&](auto threads) {
    if (decltype(threads)::value >= 128) ctas = 1024 / decltype(threads)::value;
    return cudaSuccess;
  });
  return ctas;
}

cudaError_t launch_rmsnorm_backward(const NormBackwardArgs &a, cudaStream_t stream) {
  return with_groups(a.type, a.vec, [&](auto type, auto v) {
    constexpr int TYPE = decltype(type)::value, V = decltype(v)::value, ITEMS = V == 1 ? 8 : 2;
    const unsigned grid = static_cast<unsigned>(a.strips);
    if constexpr (V > 1) {
      cudaError_t e = cudaSuccess;
      if (with_ring_threads(a.cols, V * kRingItems, [&](auto threads) {
            constexpr int THREADS = decltype(threads)::value;
            constexpr int kBytes = RowRing<TYPE, kRingItems, THREADS, 3>::kBytes;
            e = launch_ring(rmsnorm_backward_ring_kernel<TYPE, kRingItems, THREADS>, a, grid, THREADS, kBytes, stream);
          }))
        return e;
    }
    return with_threads(a.cols, V * ITEMS, [&](auto threads) {
      constexpr int THREADS = decltype(threads)::value;
      return launch_kernel(rmsnorm_backward_kernel<TYPE, V, ITEMS, THREADS>, 1, grid, THREADS == 32 ? 256 : THREADS, 0, stream, a);
    });
  });
}

}  // namespace phobos
