// fwht_wave_kept.hip -- launch interface of the rotation passes from kept activations
// (fwht_wave_kept.h), and their INT8 instantiations.
#include "fwht_wave_kept.h"

namespace halo {

HALO_KEPT_DEF(i8, 0, 0)

hipError_t launch_fq_batch_kept(const FqArgs* rows, const FqArgs& cw, void* ws_w, const FqArgs& cdy,
                                void* ws_dy, const FqArgs& cx, void* ws_x, int qg, int qw, int form,
                                hipStream_t st) {
  if (qg == 0 && qw == 0) return batch_kept_i8(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, form, st);
  if (qg == 2 && qw == 1) return batch_kept_e5m2(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, form, st);
  if (qg == 1 && qw == 1) return batch_kept_e4m3(rows, cw, ws_w, cdy, ws_dy, cx, ws_x, form, st);
  return hipErrorInvalidValue;
}

hipError_t launch_fq_rows2_kept(const FqPair& a, int qt, hipStream_t st) {
  switch (qt) {
    case 0: return rows_kept_i8(a, st);
    case 1: return rows_kept_e4m3(a, st);
    case 2: return rows_kept_e5m2(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace halo
