// Operands of the tensor-core product that cannot be read where they are.
//
// Copy: a 16-bit or 8-bit operand whose base or row stride is not a multiple of 16
// bytes, which the TMA needs, is copied with padded rows.
//
// Split: an fp32 operand becomes two fp16 terms.  Each operand row (a vector along
// the contraction) is scaled by the power of two that brings its largest
// magnitude into [2^14, 2^15): x' = x 2^-exp, exactly; then
//   hi = fp16(x'),  lo = fp16(x' - hi),   |x' - hi - lo| <= 2^-22 |x'|
// while lo is a normal fp16 number, that is for |x'| >= 2^-2 or so; below, the
// error stays under 2^-25, 2^-40 of the row's largest.  Three products of 11-bit
// terms at the fp16 rate cost half of three tf32 products with the same 22 bits.
//
// Rows that are contiguous are split by a warp or a CTA each: one pass for the
// maximum, one for the split, which hits the caches.  For an operand with its rows
// side by side (contraction strided) a cluster of CTAs takes 64 rows, each CTA a
// share of the contraction, and the row maxima meet in distributed shared memory.
// Both read 4 bytes and write 4 per element, the bound (two operands of 4096 x 4096:
// 43 us, 6.2 TB/s).
#include "epilogue.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace phobos {

namespace {

// The exponent that brings a row with largest magnitude bits `amax` to [2^14, 2^15);
// a row of zeros, or with an infinity or a NaN, takes any.
__device__ __forceinline__ int row_exponent(unsigned amax) {
  const int e = amax >> 23 ? static_cast<int>(amax >> 23) - 127 : 31 - __clz(amax | 1u) - 149;
  return min(e, 127) - 14;
}
__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ void split_store4(void *hi, void *lo, int64_t i, int n, const float (&v)[4],
                                             const int (&e)[4]) {
  float h[4], l[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const float x = times_pow2(v[t], -e[t]);
    h[t] = __half2float(__float2half_rn(x));
    l[t] = x - h[t];
  }
  store4<PHOBOS_TYPE_F16>(hi, i, n, true, h);
  store4<PHOBOS_TYPE_F16>(lo, i, n, true, l);
}

struct SplitShared {
  unsigned maxima[16][64];
  alignas(16) unsigned row_max[64];
};

// Rows along the contraction, block `block` of them: a warp each (eight a CTA) for
// short rows, else a CTA each.
template <int THREADS>
__device__ __forceinline__ void split_rows(const PrepArgs &a, int block, SplitShared &shared) {
  const int t = threadIdx.x % THREADS;
  const int64_t row = block * static_cast<int64_t>(256 / THREADS) + threadIdx.x / THREADS;
  if (row >= a.rows) return;  // several rows a CTA only where a row is one warp
  unsigned m = 0;
#pragma unroll 4
  for (int k = t * 4; k < a.k; k += THREADS * 4) {
    float v[4];
    load4<PHOBOS_TYPE_F32>(a.in.ptr, row * a.in.ld + k, min(4, a.k - k), a.vec, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, magnitude(v[j]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (THREADS > 32) {
    unsigned *maxima = &shared.maxima[0][0];
    if ((t & 31) == 0) maxima[t >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) m = max(m, maxima[w]);
  }
  const int e = row_exponent(m);
  if (t == 0) a.exp[row] = e;
  const int e4[4] = {e, e, e, e};
#pragma unroll 4
  for (int k = t * 4; k < a.k; k += THREADS * 4) {
    float v[4];
    const int n = min(4, a.k - k);
    load4<PHOBOS_TYPE_F32>(a.in.ptr, row * a.in.ld + k, n, a.vec, v);
    split_store4(a.hi, a.lo, row * a.ld + k, n, v, e4);
  }
}

constexpr int kAhead = 8;

// 64 operand rows side by side: 16 threads of four rows, 16 steps at a time; the
// cluster's `ctas` CTAs take a share of the contraction each.
__device__ __forceinline__ void split_strided(const PrepArgs &a, int block, int ctas, SplitShared &shared) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int strip = block / ctas, share = block % ctas;
  const int64_t r = strip * 64ll + tx * 4;
  const int n = static_cast<int>(min(static_cast<int64_t>(4), a.rows - r));
  const int k0 = static_cast<int>(static_cast<int64_t>(a.k) * share / ctas);
  const int k1 = static_cast<int>(static_cast<int64_t>(a.k) * (share + 1) / ctas);
  // eight loads in flight a thread, in both passes
  auto each = [&](auto f) {
    for (int k = k0 + ty; k < k1; k += 16 * kAhead) {
      float v[kAhead][4];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = k + 16 * i;
        load4<PHOBOS_TYPE_F32>(a.in.ptr, at < k1 ? at * a.in.ld + r : 0, at < k1 ? n : 0, a.vec, v[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f(k + 16 * i, v[i]);
    }
  };
  unsigned m[4] = {0, 0, 0, 0};
  if (n > 0)
    each([&](int, const float (&v)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = max(m[j], magnitude(v[j]));
    });
#pragma unroll
  for (int j = 0; j < 4; ++j) shared.maxima[ty][tx * 4 + j] = m[j];
  __syncthreads();
  if (threadIdx.x < 64) {
    unsigned x = 0;
#pragma unroll
    for (int y = 0; y < 16; ++y) x = max(x, shared.maxima[y][threadIdx.x]);
    shared.row_max[threadIdx.x] = x;
  }
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  uint4 x = *reinterpret_cast<const uint4 *>(&shared.row_max[tx * 4]);
  for (int c = 0; c < ctas && ctas > 1; ++c) {
    const float4 f = ld_shared_cluster_v4(mapa_shared(smem_u32(&shared.row_max[tx * 4]), c));
    x.x = max(x.x, __float_as_uint(f.x));
    x.y = max(x.y, __float_as_uint(f.y));
    x.z = max(x.z, __float_as_uint(f.z));
    x.w = max(x.w, __float_as_uint(f.w));
  }
  const int e[4] = {row_exponent(x.x), row_exponent(x.y), row_exponent(x.z), row_exponent(x.w)};
  if (n > 0) {
    if (share == 0 && ty == 0)
      for (int j = 0; j < n; ++j) a.exp[r + j] = e[j];
    each([&](int k, const float (&v)[4]) {
      if (k < k1) split_store4(a.hi, a.lo, k * a.ld + r, n, v, e);
    });
  }
  if (ctas > 1) cluster_sync();  // the peers read this CTA's maxima until here
}

// Two operands in one launch: blocks [0, blocks_first) (whole clusters) split the
// first.  Both lie along the contraction, or neither does: in one kernel the strided
// way's registers halve the other's CTAs (4096 x 4096 each: 73 us for one of each
// kind, 22 + 28 in two launches; 41 for two of a kind, 43 in two launches).
template <bool STRIDED>
__global__ void __launch_bounds__(256) split_kernel(const __grid_constant__ PrepArgs first,
                                                    const __grid_constant__ PrepArgs second, int blocks_first,
                                                    int ctas) {
  __shared__ SplitShared shared;
  grid_begin();
  const bool is_first = static_cast<int>(blockIdx.x) < blocks_first;
  const PrepArgs a = is_first ? first : second;
  const int block = static_cast<int>(blockIdx.x) - (is_first ? 0 : blocks_first);
  if (STRIDED) split_strided(a, block, ctas, shared);
  else if (a.k <= 1024) split_rows<32>(a, block, shared);
  else split_rows<256>(a, block, shared);
}

// Rows of `cols` elements of ELEM bytes to aligned rows; element by element from
// the unaligned side, 16 bytes at a time to the other.
template <typename T>
__global__ void __launch_bounds__(256) copy_rows_kernel(const T *in, int64_t in_ld, T *out, int64_t out_ld,
                                                        int64_t rows, int64_t cols) {
  grid_begin();
  constexpr int kGroup = 16 / sizeof(T);
  const int64_t groups = (cols + kGroup - 1) / kGroup, total = rows * groups;
  for (int64_t g = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; g < total;
       g += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = g / groups, c = (g - row * groups) * kGroup;
    struct alignas(16) Group { T x[kGroup]; } v;
#pragma unroll
    for (int t = 0; t < kGroup; ++t) v.x[t] = c + t < cols ? in[row * in_ld + c + t] : T(0);
    *reinterpret_cast<Group *>(out + row * out_ld + c) = v;  // the row is padded to whole groups
  }
}

}  // namespace

cudaError_t launch_copy(const PrepArgs &a, int sm_count, cudaStream_t stream) {
  const int64_t rows = a.in.kmajor ? a.rows : a.k, cols = a.in.kmajor ? a.k : a.rows;
  const unsigned grid = static_cast<unsigned>(8 * sm_count);
  if (a.type == PHOBOS_TYPE_E4M3)
    return launch_kernel(copy_rows_kernel<uint8_t>, 1, grid, 256, 0, stream, static_cast<const uint8_t *>(a.in.ptr),
                         a.in.ld, static_cast<uint8_t *>(a.hi), a.ld, rows, cols);
  return launch_kernel(copy_rows_kernel<uint16_t>, 1, grid, 256, 0, stream, static_cast<const uint16_t *>(a.in.ptr),
                       a.in.ld, static_cast<uint16_t *>(a.hi), a.ld, rows, cols);
}

cudaError_t launch_split(const PrepArgs &first, const PrepArgs *second, int sm_count, cudaStream_t stream) {
  const bool strided = !first.in.kmajor;
  // clusters for strided operands: enough CTAs to fill the SMs about twice, at least 64
  // steps each
  int ctas = 1;
  for (const PrepArgs *a : {&first, second}) {
    if (!a || !strided) continue;
    const int64_t strips = (a->rows + 63ll) / 64;
    int c = 1;
    while (c < 8 && strips * c < 2 * sm_count && a->k / (2 * c) >= 64) c *= 2;
    if (c > ctas) ctas = c;
  }
  auto blocks = [&](const PrepArgs &a) -> int64_t {
    return strided ? (a.rows + 63ll) / 64 * ctas : a.k <= 1024 ? (a.rows + 7ll) / 8 : a.rows;
  };
  const int64_t blocks_first = blocks(first), all = blocks_first + (second ? blocks(*second) : 0);
  if (all > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_kernel(strided ? split_kernel<true> : split_kernel<false>, static_cast<unsigned>(ctas),
                       static_cast<unsigned>(all), 256, 0, stream, first, second ? *second : first,
                       static_cast<int>(blocks_first), ctas);
}

}  // namespace phobos
