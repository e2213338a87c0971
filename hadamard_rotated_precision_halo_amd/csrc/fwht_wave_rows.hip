// fwht_wave_rows.hip -- the wave-slice rows kernels (fwht_wave.h): nearest-even codes of bf16 and fp32
// rows, and the rotated values.
#include "fwht_wave.h"

namespace halo {

hipError_t rows2_dispatch(const FqPair& a, int in_bf16, int qt, hipStream_t st) {
  if (in_bf16) {
    switch (qt) {
      case 0: return rows2_block<uint16_t, 0, false>(a, st);
      case 1: return rows2_block<uint16_t, 1, false>(a, st);
      case 2: return rows2_block<uint16_t, 2, false>(a, st);
      case 3: return rows2_block<uint16_t, 3, false>(a, st);
    }
  } else {
    switch (qt) {
      case 0: return rows2_block<float, 0, false>(a, st);
      case 1: return rows2_block<float, 1, false>(a, st);
      case 2: return rows2_block<float, 2, false>(a, st);
      case 3: return rows2_block<float, 3, false>(a, st);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace halo
