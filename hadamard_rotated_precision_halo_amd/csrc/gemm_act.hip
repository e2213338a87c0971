// gemm_act.hip -- launch interface of the layer's product with its epilogue (gemm_act.h), and the
// kernels that keep z as plain elements or not at all.
#include "gemm_act.h"

namespace halo {

hipError_t launch_gemm_act(const GemmArgs& g, int kind, int out, hipStream_t st) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  if (g.m <= kSkinnyRows) return launch_gemm_skinny(g, kind, out, st);
  return g.kept ? launch_gemm_act_kept(g, kind, out, st) : launch_act<false>(g, kind, out, st);
}

}  // namespace halo
