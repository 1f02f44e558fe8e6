// Element types and the epilogue shared by the layer kernels.
#pragma once

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "layers_internal.h"

namespace phobos {

// ---------------------------------------------------------------- element types

template <int TYPE>
struct Elem;
template <>
struct Elem<PHOBOS_TYPE_F32> {
  using T = float;
  static __device__ __forceinline__ float load(float x) { return x; }
  static __device__ __forceinline__ float store(float x) { return x; }
};
template <>
struct Elem<PHOBOS_TYPE_F16> {
  using T = __half;
  static __device__ __forceinline__ float load(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half store(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<PHOBOS_TYPE_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float load(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 store(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<PHOBOS_TYPE_E4M3> {
  using T = __nv_fp8_e4m3;
  static __device__ __forceinline__ float load(__nv_fp8_e4m3 x) { return static_cast<float>(x); }
};

// Four consecutive elements, of which the first n exist (zeros elsewhere); vec:
// the address is aligned for all four at once.
template <int TYPE>
__device__ __forceinline__ void load4(const void *base, int64_t i, int n, bool vec, float (&v)[4]) {
  using E = Elem<TYPE>;
  const typename E::T *p = static_cast<const typename E::T *>(base) + i;
  if (vec && n >= 4) {
    struct alignas(4 * sizeof(typename E::T)) Group { typename E::T x[4]; };
    const Group g = *reinterpret_cast<const Group *>(p);
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = E::load(g.x[t]);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = t < n ? E::load(p[t]) : 0.f;
  }
}

template <int TYPE>
__device__ __forceinline__ void store4(void *base, int64_t i, int n, bool vec, const float (&v)[4]) {
  using E = Elem<TYPE>;
  typename E::T *p = static_cast<typename E::T *>(base) + i;
  if (vec && n >= 4) {
    struct alignas(4 * sizeof(typename E::T)) Group { typename E::T x[4]; } g;
#pragma unroll
    for (int t = 0; t < 4; ++t) g.x[t] = E::store(v[t]);
    *reinterpret_cast<Group *>(p) = g;
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t < n) p[t] = E::store(v[t]);
  }
}

__device__ __forceinline__ void load4(int type, const void *base, int64_t i, int n, bool vec,
                                      float (&v)[4]) {
  if (type == PHOBOS_TYPE_F32) load4<PHOBOS_TYPE_F32>(base, i, n, vec, v);
  else if (type == PHOBOS_TYPE_BF16) load4<PHOBOS_TYPE_BF16>(base, i, n, vec, v);
  else load4<PHOBOS_TYPE_F16>(base, i, n, vec, v);
}

// V consecutive elements as they are stored.  load and store: the first n exist (zeros
// elsewhere), and with V > 1 the address is aligned for all of them at once;
// load_any and store_any: any alignment.  16-bit types are converted in pairs.
template <int TYPE, int V>
struct Group {
  using T = typename Elem<TYPE>::T;
  static constexpr int kSize = V;
  alignas(V * sizeof(T)) T x[V];

  __device__ __forceinline__ void load(const void *base, int64_t i, int n) {
    const T *p = static_cast<const T *>(base) + i;
    if (V == 1 ? n > 0 : n >= V) {
      *this = *reinterpret_cast<const Group *>(p);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = j < n ? p[j] : Elem<TYPE>::store(0.f);
    }
  }
  __device__ __forceinline__ void load_any(const void *base, int64_t i, int n) {
    const T *p = static_cast<const T *>(base) + i;
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = j < n ? p[j] : Elem<TYPE>::store(0.f);
  }
  __device__ __forceinline__ void store_any(void *base, int64_t i, int n) const {
    T *p = static_cast<T *>(base) + i;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) p[j] = x[j];
  }
  __device__ __forceinline__ void store(void *base, int64_t i, int n) const {
    if (V == 1 ? n > 0 : n >= V) *reinterpret_cast<Group *>(static_cast<T *>(base) + i) = *this;
    else store_any(base, i, n);
  }
  __device__ __forceinline__ void unpack(float (&v)[V]) const {
    if constexpr (TYPE == PHOBOS_TYPE_BF16 && V > 1) {
      const uint32_t *w = reinterpret_cast<const uint32_t *>(x);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        v[j] = __uint_as_float(w[j / 2] << 16);
        v[j + 1] = __uint_as_float(w[j / 2] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = Elem<TYPE>::load(x[j]);
    }
  }
  __device__ __forceinline__ void pack(const float (&v)[V]) {
    if constexpr (TYPE == PHOBOS_TYPE_BF16 && V > 1) {
      __nv_bfloat162 *w = reinterpret_cast<__nv_bfloat162 *>(x);
#pragma unroll
      for (int j = 0; j < V; j += 2) w[j / 2] = __floats2bfloat162_rn(v[j], v[j + 1]);
    } else if constexpr (TYPE == PHOBOS_TYPE_F16 && V > 1) {
      __half2 *w = reinterpret_cast<__half2 *>(x);
#pragma unroll
      for (int j = 0; j < V; j += 2) w[j / 2] = __floats2half2_rn(v[j], v[j + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = Elem<TYPE>::store(v[j]);
    }
  }
  __device__ __forceinline__ void fill(float value) {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = Elem<TYPE>::store(value);
  }
};

// ------------------------------------------------------------------ activations

// The logistic function; exp(-z) = inf gives 0.
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kGeluIn = 1.5957691216057308f;  // sqrt(8 / pi)
constexpr float kGeluCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == PHOBOS_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays
  if (ACT == PHOBOS_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
  // tanh(u) = 2 s(2u) - 1 turns z (1 + tanh(u)) / 2 into z s(2u), which also
  // keeps its relative accuracy where 1 + tanh(u) cancels
  if (ACT == PHOBOS_ACT_GELU_TANH) return z * logistic(kGeluIn * z * fmaf(kGeluCubic * z, z, 1.0f));
  if (ACT == PHOBOS_ACT_SILU) return z * logistic(z);
  return z;
}

// The choice is made once for all values: a branch per value would keep their
// exponentials and divisions from overlapping (measured: 570 us more at 8192^3).
template <int N>
__device__ __forceinline__ void activate_all(int act, float (&z)[N]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = f(z[i]);
  };
  switch (act) {
    case PHOBOS_ACT_RELU: each(activate<PHOBOS_ACT_RELU>); break;
    case PHOBOS_ACT_GELU: each(activate<PHOBOS_ACT_GELU>); break;
    case PHOBOS_ACT_GELU_TANH: each(activate<PHOBOS_ACT_GELU_TANH>); break;
    case PHOBOS_ACT_SILU: each(activate<PHOBOS_ACT_SILU>); break;
    default: break;
  }
}

// Far from zero the slope is that of z or of zero: the terms that vanish there are left
// out, as their other factors may have overflowed (infinite z, whose products with zero
// are NaNs; the cube of a finite one).
template <int ACT>
__device__ __forceinline__ float activate_slope(float z) {
  if (ACT == PHOBOS_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if (ACT == PHOBOS_ACT_GELU) {  // Phi(z) + z phi(z), phi(0) = 1 / sqrt(2 pi)
    const float cdf = 0.5f * (1.0f + erff(z * 0.70710678118654752f)), e = __expf(-0.5f * z * z);
    return e == 0.0f ? cdf : fmaf(z * 0.3989422804014327f, e, cdf);
  }
  if (ACT == PHOBOS_ACT_GELU_TANH) {
    const float p = logistic(kGeluIn * z * fmaf(kGeluCubic * z, z, 1.0f)), q = p * (1.0f - p);
    return q == 0.0f ? p : fmaf(z * q, kGeluIn * fmaf(3.0f * kGeluCubic * z, z, 1.0f), p);
  }
  if (ACT == PHOBOS_ACT_SILU) {
    const float p = logistic(z), q = 1.0f - p;
    return p == 0.0f || q == 0.0f ? p : p * fmaf(z, q, 1.0f);
  }
  return 1.0f;
}

// --------------------------------------------------------------------- epilogue

// s * 2^e in two factors, so that neither overflows or vanishes when the product does
// not; e <= 254, and below -252 the product is as good as zero (|s| < 2^100).
__device__ __forceinline__ float times_pow2(float s, int e) {
  e = max(e, -252);
  const int half = e >> 1;
  return s * __int_as_float((half + 127) << 23) * __int_as_float((e - half + 127) << 23);
}

// The column factors of columns col .. col+3: loaded once, used for many rows.
struct EpilogueColumns {
  float bias[4], scale[4];
};

__device__ __forceinline__ void epilogue_columns(const Epilogue &e, int col, int n, bool vec,
                                                 EpilogueColumns &c) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    c.bias[t] = 0.f;
    c.scale[t] = 0.f;
    if (t < n && e.col_scale) c.scale[t] = e.col_scale[col + t];
  }
  if (e.bias) load4(e.type, e.bias, col, n, vec, c.bias);
}

// Sums s of row `row`, columns col .. col+3 (n of them exist) to the output.
template <int TYPE>
__device__ __forceinline__ void epilogue_row4(const Epilogue &e, const EpilogueColumns &c, int row,
                                              int col, int n, float (&s)[4]) {
  float r[4] = {};
  if (e.residual) load4<TYPE>(e.residual, row * e.residual_ld + col, n, e.vec, r);
  if (e.row_scale) {
    const float f = e.row_scale[row];
#pragma unroll
    for (int t = 0; t < 4; ++t) s[t] = fmaf(s[t] * f, c.scale[t], c.bias[t]);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) s[t] += c.bias[t];
  }
  if (e.preact) store4<TYPE>(e.preact, row * e.preact_ld + col, n, e.vec, s);
  activate_all(e.act, s);
  if (e.residual) {
#pragma unroll
    for (int t = 0; t < 4; ++t) s[t] += r[t];
  }
  store4<TYPE>(e.out, row * e.out_ld + col, n, e.vec, s);
}

// f(std::integral_constant<int, type>()) for a floating type.
template <typename F>
__device__ __forceinline__ void with_type(int type, F f) {
  switch (type) {
    case PHOBOS_TYPE_F32: f(std::integral_constant<int, PHOBOS_TYPE_F32>()); break;
    case PHOBOS_TYPE_F16: f(std::integral_constant<int, PHOBOS_TYPE_F16>()); break;
    default: f(std::integral_constant<int, PHOBOS_TYPE_BF16>()); break;
  }
}

}  // namespace phobos
