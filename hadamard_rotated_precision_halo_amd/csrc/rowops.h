// rowops.h -- row access and reductions shared by the memory-bound row operators (block_norm,
// distill): 16-byte chunks of a row in registers, whatever the row's alignment and length.
#pragma once

#include "halo_device.h"

namespace halo {

// Chunk of VEC consecutive elements of type T in its stored form.
template <typename T>
struct RowType;
template <>
struct RowType<uint16_t> {  // bf16
  static constexpr int VEC = 8;
};
template <>
struct RowType<float> {
  static constexpr int VEC = 4;
};

// 16 bytes at an address aligned to its element only (global loads and stores take any
// alignment on this target; rows of odd length or stride start anywhere).
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ uint4 load16u(const void* p) {
  const v4i_any w = *reinterpret_cast<const v4i_any*>(p);
  return make_uint4((uint32_t)w.x, (uint32_t)w.y, (uint32_t)w.z, (uint32_t)w.w);
}
__device__ __forceinline__ void store16u(void* p, uint4 v) {
  const v4i_any w = {(int)v.x, (int)v.y, (int)v.z, (int)v.w};
  *reinterpret_cast<v4i_any*>(p) = w;
}

// The same past the caches, for what is read or written once.
__device__ __forceinline__ uint4 load16u_nt(const void* p) {
  const v4i_any w = __builtin_nontemporal_load(reinterpret_cast<const v4i_any*>(p));
  return make_uint4((uint32_t)w.x, (uint32_t)w.y, (uint32_t)w.z, (uint32_t)w.w);
}
__device__ __forceinline__ void store16u_nt(void* p, uint4 v) {
  const v4i_any w = {(int)v.x, (int)v.y, (int)v.z, (int)v.w};
  __builtin_nontemporal_store(w, reinterpret_cast<v4i_any*>(p));
}

typedef __bf16 bf16v2 __attribute__((ext_vector_type(2)));
typedef float f32v2 __attribute__((ext_vector_type(2)));

// Two fp32 values to packed bf16, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32v2){a, b}, bf16v2));
}

template <typename T>
__device__ __forceinline__ float elem_f32(const T* p);
template <>
__device__ __forceinline__ float elem_f32<uint16_t>(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}
template <>
__device__ __forceinline__ float elem_f32<float>(const float* p) {
  return *p;
}
template <typename T>
__device__ __forceinline__ void elem_store(T* p, float v);
template <>
__device__ __forceinline__ void elem_store<uint16_t>(uint16_t* p, float v) {
  *p = (uint16_t)bf16x2_of(v, 0.f);
}
template <>
__device__ __forceinline__ void elem_store<float>(float* p, float v) {
  *p = v;
}

// The 16 raw bytes as fp32 values, and back (one rounding).
template <typename T>
__device__ __forceinline__ void unpack16(uint4 w, float* o);
template <>
__device__ __forceinline__ void unpack16<uint16_t>(uint4 w, float* o) {
  unpack_bf16x8(w, o);
}
template <>
__device__ __forceinline__ void unpack16<float>(uint4 w, float* o) {
  o[0] = __uint_as_float(w.x);
  o[1] = __uint_as_float(w.y);
  o[2] = __uint_as_float(w.z);
  o[3] = __uint_as_float(w.w);
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* v);
template <>
__device__ __forceinline__ uint4 pack16<uint16_t>(const float* v) {
  return make_uint4(bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]), bf16x2_of(v[4], v[5]),
                    bf16x2_of(v[6], v[7]));
}
template <>
__device__ __forceinline__ uint4 pack16<float>(const float* v) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]));
}

// Keeps chunks in their stored form from here on: the compiler would otherwise keep the fp32 values
// of an earlier pass over them, twice the registers.
__device__ __forceinline__ void keep_raw1(uint4& w) {
  asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
}
template <int CH>
__device__ __forceinline__ void keep_raw(uint4 (&raw)[CH]) {
#pragma unroll
  for (int j = 0; j < CH; ++j) keep_raw1(raw[j]);
}

// Sum and maximum over the 64 lanes of a wave (every lane receives it; fixed order).
__device__ __forceinline__ float wave_sum(float v) {
  v += partner<0>(v);
  v += partner<1>(v);
  v += partner<2>(v);
  v += partner<3>(v);
  v += partner<4>(v);
  v += partner<5>(v);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
  v = xmax<0>(v);
  v = xmax<1>(v);
  v = xmax<2>(v);
  v = xmax<3>(v);
  v = xmax<4>(v);
  v = xmax<5>(v);
  return v;
}

}  // namespace halo
