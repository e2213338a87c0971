// fwht_wave_kept.h -- the rotation passes of a layer backward from kept activations
// (fwht_wave.h): x and z as bf16 or as 8-bit checkpoints (checkpoint.h), dz = dy act'(z) formed in
// fp32 as its inputs are loaded, or the gated layer's, stored.  bf16 dy and w, nearest rounding, blocks
// 64 .. 1024.  One source file per pair of code types, so that they compile in parallel.
#pragma once

#include "fwht_wave.h"

namespace halo {

template <int QG, int QW, int ACT>
static hipError_t batch_kept(const FqArgs* rows, const FqArgs& cw, void* ws_w, const FqArgs& cdy,
                             void* ws_dy, const FqArgs& cx, void* ws_x, hipStream_t st) {
  if (cw.sr || cx.sr || cdy.sr || (rows && rows->sr)) return hipErrorInvalidValue;
#define HALO_K_CASE(BB) \
  case BB: return launch_batch_t<BB, QG, QW, false, ACT, true>(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, st);
  switch (cw.block) {
    HALO_K_CASE(64) HALO_K_CASE(128) HALO_K_CASE(256) HALO_K_CASE(512) HALO_K_CASE(1024)
    default: return hipErrorInvalidValue;
  }
#undef HALO_K_CASE
}

template <int QT>
static hipError_t rows_kept(const FqPair& a, hipStream_t st) {
  if (a.p0.sr || a.has1) return hipErrorInvalidValue;
#define HALO_K_CASE(BB) \
  case BB: return launch_rows2_t<uint16_t, BB, QT, false, kDyKept>(a, st);
  switch (a.p0.block) {
    HALO_K_CASE(64) HALO_K_CASE(128) HALO_K_CASE(256) HALO_K_CASE(512) HALO_K_CASE(1024)
    default: return hipErrorInvalidValue;
  }
#undef HALO_K_CASE
}

// The instantiations of a pair (codes of dY, of W and X), and of the rows of dY.
#define HALO_KEPT_DECL(NAME)                                                                     \
  hipError_t batch_kept_##NAME(const FqArgs* rows, const FqArgs& cw, void* ws_w,                 \
                               const FqArgs& cdy, void* ws_dy, const FqArgs& cx, void* ws_x,     \
                               int form, hipStream_t st);                                        \
  hipError_t rows_kept_##NAME(const FqPair& a, hipStream_t st);
HALO_KEPT_DECL(i8)
HALO_KEPT_DECL(e5m2)
HALO_KEPT_DECL(e4m3)
#undef HALO_KEPT_DECL

#define HALO_KEPT_DEF(NAME, QG, QW)                                                              \
  hipError_t batch_kept_##NAME(const FqArgs* rows, const FqArgs& cw, void* ws_w,                 \
                               const FqArgs& cdy, void* ws_dy, const FqArgs& cx, void* ws_x,     \
                               int form, hipStream_t st) {                                       \
    switch (form) {                                                                              \
      case kDyPlain: return batch_kept<QG, QW, kDyPlain>(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, st);   \
      case kDyKept: return batch_kept<QG, QW, kDyKept>(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, st);     \
      case kDyStored: return batch_kept<QG, QW, kDyStored>(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, st); \
    }                                                                                            \
    return hipErrorInvalidValue;                                                                 \
  }                                                                                              \
  hipError_t rows_kept_##NAME(const FqPair& a, hipStream_t st) { return rows_kept<QG>(a, st); }

}  // namespace halo
