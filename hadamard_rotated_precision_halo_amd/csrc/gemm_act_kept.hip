// gemm_act_kept.hip -- the kernels of the layer's product with its epilogue that keep z in 8 bits
// (gemm_act.h).
#include "gemm_act.h"

namespace halo {

hipError_t launch_gemm_act_kept(const GemmArgs& g, int kind, int out, hipStream_t st) {
  return launch_act<true>(g, kind, out, st);
}

}  // namespace halo
