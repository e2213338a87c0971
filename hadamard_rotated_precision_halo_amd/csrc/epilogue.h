// epilogue.h -- activations of the layer's epilogue and their slopes, and the loads and stores of
// an epilogue's columns.
#pragma once

#include "rowops.h"

namespace halo {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGeluTanh = 3, kActGeluErf = 4 };

// 1 / (1 + exp(-x)): v_exp_f32 and v_rcp_f32, 1 ulp each; the argument's scaling to base 2 adds
// |x| 2^-24 relative.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

// 2 sqrt(2 / pi) (z + 0.044715 z^3): gelu's tanh form is z (1 + tanh u) / 2 = z sigmoid(2 u)
__device__ __forceinline__ float gelu_arg(float z) {
  const float t = z * z;
  return z * __builtin_fmaf(t, 0.07135481627159f, 1.5957691216057308f);
}

// erfc(x) / 2 for x >= 0 and exp(-x^2), by formula 7.1.26 of Abramowitz and Stegun, "Handbook of
// Mathematical Functions" (absolute error of erf below 1.5e-7, 2.5 units of 2^-24): one
// exponential, one reciprocal and five multiply-adds, a quarter of the library erf's time.  For
// bf16 outputs and for slopes; the tail's relative error (5e-5 at z = -3, 1.6e-3 at -5) would show
// in fp32 outputs, which take the library's erfc.
__device__ __forceinline__ float half_erfc(float x, float* gauss) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.f));
  float p = __builtin_fmaf(1.061405429f, t, -1.453152027f);
  p = __builtin_fmaf(p, t, 1.421413741f);
  p = __builtin_fmaf(p, t, -0.284496736f);
  p = __builtin_fmaf(p, t, 0.254829592f);
  *gauss = __builtin_amdgcn_exp2f(x * x * -1.4426950408889634f);
  return 0.5f * p * t * *gauss;
}

// The normal distribution at z and exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float* gauss) {
  const float h = half_erfc(fabsf(z) * 0.7071067811865476f, gauss);
  return z < 0.f ? h : 1.f - h;
}

// FULL: for fp32 outputs.
template <int ACT, bool FULL>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == kActRelu) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (ACT == kActSilu) return z * sigmoid_fast(z);
  if constexpr (ACT == kActGeluTanh) return z * sigmoid_fast(gelu_arg(z));
  if constexpr (ACT == kActGeluErf) {
    if constexpr (FULL) return z * (0.5f * erfcf(z * -0.7071067811865476f));
    float gauss;
    return z * normal_cdf(z, &gauss);
  }
  return z;
}

// d act / dz.  silu: p + z p (1 - p); gelu's tanh form the same with p = sigmoid(2 u) and the
// slope of 2 u; gelu: the normal distribution plus z times its density.
template <int ACT>
__device__ __forceinline__ float slope_of(float z) {
  if constexpr (ACT == kActRelu) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  if constexpr (ACT == kActSilu) {
    const float p = sigmoid_fast(z);
    return __builtin_fmaf(z * p, 1.f - p, p);
  }
  if constexpr (ACT == kActGeluTanh) {
    const float p = sigmoid_fast(gelu_arg(z));
    // z^2 would be infinite, and zero times it NaN, from 1.8e19 on, where p (1 - p) is long 0
    const float zz = fminf(z * z, 1e30f);
    const float du = __builtin_fmaf(zz, 3.f * 0.07135481627159f, 1.5957691216057308f);
    return __builtin_fmaf(z * (p * (1.f - p)), du, p);
  }
  if constexpr (ACT == kActGeluErf) {
    float gauss;
    const float cdf = normal_cdf(z, &gauss);
    return __builtin_fmaf(z * 0.3989422804014327f, gauss, cdf);
  }
  return 1.f;
}

// The activation (a wave-uniform choice) of 8 values, for outputs of type T.
template <typename T>
__device__ __forceinline__ void act8(int act, const float* z, float* y) {
#define HALO_ACT8(A) \
  _Pragma("unroll") for (int e = 0; e < 8; ++e) y[e] = act_of<A, sizeof(T) == 4>(z[e])
  switch (act) {
    case kActRelu: HALO_ACT8(kActRelu); break;
    case kActSilu: HALO_ACT8(kActSilu); break;
    case kActGeluTanh: HALO_ACT8(kActGeluTanh); break;
    case kActGeluErf: HALO_ACT8(kActGeluErf); break;
    default: HALO_ACT8(kActNone); break;
  }
#undef HALO_ACT8
}

// d[e] *= slope(z[e]) for N values.
template <int N>
__device__ __forceinline__ void slope_mul(int act, const float* z, float* d) {
#define HALO_SLOPE(A) \
  _Pragma("unroll") for (int e = 0; e < N; ++e) d[e] *= slope_of<A>(z[e])
  switch (act) {
    case kActRelu: HALO_SLOPE(kActRelu); break;
    case kActSilu: HALO_SLOPE(kActSilu); break;
    case kActGeluTanh: HALO_SLOPE(kActGeluTanh); break;
    case kActGeluErf: HALO_SLOPE(kActGeluErf); break;
    default: break;
  }
#undef HALO_SLOPE
}

// 8 columns of an epilogue row, of which cnt (1 .. 8) exist.  Rows start 16-byte aligned and
// lanes take multiples of 8 columns, so a whole group is one 16-byte access (two for fp32).
template <typename T>
__device__ __forceinline__ void load_cols(const T* p, int cnt, float* o) {
  if (cnt == 8) {
    load8<T>(p, o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = e < cnt ? elem_f32<T>(p + e) : 0.f;
  }
}

// Whole groups are stored non-temporally, as the bare product's: whether the next operator then finds
// them in a cache does not show (a chain of join, layer, layer and join at 8192 x 4096: 379 us, with
// these stores through the caches 378 us).
template <typename T>
__device__ __forceinline__ void store_cols(T* p, int cnt, const float* v) {
  if (cnt == 8) {
    if constexpr (sizeof(T) == 2) {
      const uint4 w = pack16<uint16_t>(v);
      const v4i o = {(int)w.x, (int)w.y, (int)w.z, (int)w.w};
      __builtin_nontemporal_store(o, reinterpret_cast<v4i*>(p));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4i o = {__float_as_int(v[4 * h]), __float_as_int(v[4 * h + 1]),
                       __float_as_int(v[4 * h + 2]), __float_as_int(v[4 * h + 3])};
        __builtin_nontemporal_store(o, reinterpret_cast<v4i*>(p + 4 * h));
      }
    }
  } else {
    for (int e = 0; e < cnt; ++e) elem_store<T>(p + e, v[e]);
  }
}

}  // namespace halo
