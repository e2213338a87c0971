// fwht_wave_act.hip -- the activation-gradient instantiations of the wave-slice rotation kernels
// (fwht_wave.h): the rotation passes of a layer backward whose gradient is dz = dy act'(z), formed
// in fp32 as dy and z are loaded, so that dz never goes to memory, and the bias gradient beside
// them from the columns pass.  bf16 input, nearest rounding, blocks 64 .. 1024.
#include "fwht_wave.h"

namespace halo {

bool fq_act_block_ok(int block) { return block >= 64 && block <= 1024; }

int64_t fq_act_parts(int64_t rows, int block) {
  const int R = cols2_rows_per_task(rows, block);
  return R == 0 ? 0 : rows / R;
}

namespace {

template <int QG, int QW>
hipError_t batch_act(const FqArgs* rows, const FqArgs& cw, void* ws_w, const FqArgs& cdy,
                     void* ws_dy, const FqArgs& cx, void* ws_x, hipStream_t st) {
#define HALO_A_CASE(BB) \
  case BB: return launch_batch_t<BB, QG, QW, false, true>(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, st);
  switch (cw.block) {
    HALO_A_CASE(64) HALO_A_CASE(128) HALO_A_CASE(256) HALO_A_CASE(512) HALO_A_CASE(1024)
    default: return hipErrorInvalidValue;
  }
#undef HALO_A_CASE
}

template <int QT>
hipError_t rows_act(const FqPair& a, hipStream_t st) {
#define HALO_A_CASE(BB) \
  case BB: return launch_rows2_t<uint16_t, BB, QT, false, true>(a, st);
  switch (a.p0.block) {
    HALO_A_CASE(64) HALO_A_CASE(128) HALO_A_CASE(256) HALO_A_CASE(512) HALO_A_CASE(1024)
    default: return hipErrorInvalidValue;
  }
#undef HALO_A_CASE
}

}  // namespace

hipError_t launch_fq_batch_act(const FqArgs* rows, const FqArgs& cw, void* ws_w, const FqArgs& cdy,
                               void* ws_dy, const FqArgs& cx, void* ws_x, int qg, int qw,
                               hipStream_t st) {
  if (cw.sr || cx.sr || cdy.sr || (rows && rows->sr)) return hipErrorInvalidValue;
  if (qg == 0 && qw == 0) return batch_act<0, 0>(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, st);
  if (qg == 2 && qw == 1) return batch_act<2, 1>(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, st);
  if (qg == 1 && qw == 1) return batch_act<1, 1>(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, st);
  return hipErrorInvalidValue;
}

hipError_t launch_fq_rows2_act(const FqPair& a, int qt, hipStream_t st) {
  if (a.p0.sr || a.has1) return hipErrorInvalidValue;
  switch (qt) {
    case 0: return rows_act<0>(a, st);
    case 1: return rows_act<1>(a, st);
    case 2: return rows_act<2>(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace halo
