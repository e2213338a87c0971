// checkpoint.h -- activations kept in 8 bits for the backward pass: a row in groups of 32 values,
// each with a power of two.
//
// A group's power 2^(s - 127) is the least with max |v| <= qmax 2^(s - 127) (qmax 127 for INT8, 448
// for E4M3), s in [16, 248 or 246], and its codes are v / 2^(s - 127) rounded once, ties to even, and
// kept within +-qmax.  A power of two rather than max / qmax: the division and every code times its
// power are then exact, in bf16 too (8 significant bits), so a kept value means the same number to
// every reader and the rotation passes take it as they take a bf16 one; it costs INT8 half a bit on
// average.  The lower
// bound on s keeps values and products out of the subnormals (what is below 2^-112 is lost), the
// upper one keeps the largest finite ones finite.  A group with an infinity or a NaN has s = 255 and
// stands for NaN throughout.
#pragma once

#include "halo_device.h"
#include "rowops.h"

namespace halo {

constexpr int kGroup = 32;
constexpr uint32_t kLostGroup = 255;  // s of a group that holds an infinity or a NaN

// Kept forms: 0 not kept in 8 bits, else 1 + the code type (0 INT8, 1 E4M3).
enum Kept { kKeptPlain = 0, kKeptI8 = 1, kKeptE4M3 = 2 };

// s of a group from the bits of its largest |v| (unsigned order, so that a NaN is the largest).
template <int QT>
__device__ __forceinline__ uint32_t group_power(uint32_t top) {
  constexpr uint32_t full = QT == 0 ? 0x7E0000u : 0x600000u;  // mantissa of qmax
  constexpr int drop = QT == 0 ? 6 : 8;                       // exponent of qmax
  int s = (int)(top >> 23) - drop + ((top & 0x7fffffu) > full ? 1 : 0);
  s = min(max(s, 16), 254 - drop);
  return top >= 0x7f800000u ? kLostGroup : (uint32_t)s;
}

// 2^(s - 127); infinity for a lost group, whose codes make it NaN.
__device__ __forceinline__ float power_of(uint32_t s) { return __uint_as_float(s << 23); }

// 8 values as codes of a group with s.
template <int QT>
__device__ __forceinline__ uint2 keep8(const float* v, uint32_t s) {
  constexpr float qmax = QT == 0 ? 127.f : 448.f;
  const float inv = __uint_as_float((254u - min(s, 254u)) << 23);
  float t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = __builtin_amdgcn_fmed3f(v[e] * inv, -qmax, qmax);
  uint2 w = encode8<QT>(t, 1.f);
  constexpr uint32_t lost = QT == 0 ? 0u : 0x7f7f7f7fu;  // 0 x infinity, and NaN
  if (s == kLostGroup) w = make_uint2(lost, lost);
  return w;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Largest of a value over the 4 lanes of a quad.
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
}

// The values of 4 codes (unscaled).
template <int QT>
__device__ __forceinline__ void codes4(uint32_t w, float* o) {
  if constexpr (QT == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = (float)((int)(w << (24 - 8 * e)) >> 24);
  } else {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    o[0] = lo[0];
    o[1] = lo[1];
    o[2] = hi[0];
    o[3] = hi[1];
  }
}

// 8 kept values of one group.
template <int QT>
__device__ __forceinline__ void kept8(uint2 w, uint32_t s, float* o) {
  codes4<QT>(w.x, o);
  codes4<QT>(w.y, o + 4);
  const float p = power_of(s);
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] *= p;
}

// A row's 8 values at columns col .. (col a multiple of 8, a quad's lanes the four parts of one
// group) into a checkpoint of rows of n (a multiple of 8): every lane of the quad takes part, and
// stores where `in`.
template <int QT>
__device__ __forceinline__ void keep_cols(void* codes, uint8_t* powers, int64_t row, int64_t n,
                                          int64_t col, bool in, const float* z) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, abs_bits(z[e]));
  const uint32_t s = group_power<QT>(quad_umax(col < n ? top : 0u));
  if (!in || col >= n) return;
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(codes) + row * n + col) = keep8<QT>(z, s);
  if (col % kGroup == 0) powers[row * ((n + kGroup - 1) / kGroup) + col / kGroup] = (uint8_t)s;
}
__device__ __forceinline__ void keep_cols(int kept, void* codes, uint8_t* powers, int64_t row,
                                          int64_t n, int64_t col, bool in, const float* z) {
  if (kept == kKeptI8) keep_cols<0>(codes, powers, row, n, col, in, z);
  else keep_cols<1>(codes, powers, row, n, col, in, z);
}

}  // namespace halo
