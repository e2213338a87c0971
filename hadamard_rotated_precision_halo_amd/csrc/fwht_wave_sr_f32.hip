// fwht_wave_sr_f32.hip -- the stochastic-rounding rows kernels (fwht_wave.h) of fp32 input: the rows of
// a layer's dz or fp32 dY that are longer than a workgroup of fwht_quant.hip holds.
#include "fwht_wave.h"

namespace halo {

hipError_t rows2_dispatch_sr_f32(const FqPair& a, int qt, hipStream_t st) {
  switch (qt) {
    case 0: return rows2_block<float, 0, true>(a, st);
    case 1: return rows2_block<float, 1, true>(a, st);
    case 2: return rows2_block<float, 2, true>(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace halo
