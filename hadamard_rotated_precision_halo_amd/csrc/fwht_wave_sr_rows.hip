// fwht_wave_sr_rows.hip -- the stochastic-rounding rows kernels (fwht_wave.h) of bf16 input.
#include "fwht_wave.h"

namespace halo {

hipError_t rows2_dispatch_sr(const FqPair& a, int qt, hipStream_t st) {
  switch (qt) {
    case 0: return rows2_block<uint16_t, 0, true>(a, st);
    case 1: return rows2_block<uint16_t, 1, true>(a, st);
    case 2: return rows2_block<uint16_t, 2, true>(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace halo
