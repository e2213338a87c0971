// fwht_wave_kept_e4m3.hip -- the E4M3 gradient's instantiations of the rotation passes from kept
// activations (fwht_wave_kept.h); W and X take E4M3 codes.
#include "fwht_wave_kept.h"

namespace halo {

HALO_KEPT_DEF(e4m3, 1, 1)

}  // namespace halo
