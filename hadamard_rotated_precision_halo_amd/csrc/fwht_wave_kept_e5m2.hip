// fwht_wave_kept_e5m2.hip -- the E5M2 gradient's instantiations of the rotation passes from kept
// activations (fwht_wave_kept.h); W and X take E4M3 codes.
#include "fwht_wave_kept.h"

namespace halo {

HALO_KEPT_DEF(e5m2, 2, 1)

}  // namespace halo
