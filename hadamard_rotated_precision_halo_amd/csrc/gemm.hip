// gemm.hip -- the layer's 8-bit products: the kernel of gemm_tile.h, one or two products per launch.
#include "gemm_tile.h"

namespace halo {

template <int KIND, int AF, int BF, int OUT, bool MASK, int BK, typename CFG>
static hipError_t launch_cfg(const GemmArgs& g0, const GemmArgs* g1, hipStream_t st) {
  constexpr int BM = CFG::BT, BN = CFG::BT, NT = 64 * CFG::WM * CFG::WN;
  const hipError_t attr_err =
      allow_dynamic_lds<&gemm_kernel<KIND, AF, BF, OUT, MASK, BK, CFG, kEpiNone>>(CFG::LDS);
  if (attr_err != hipSuccess) return attr_err;
  GemmPair gp{};
  gp.g[0] = g0;
  gp.g[1] = g1 ? *g1 : g0;
  gp.split = ((g0.m + BM - 1) / BM) * ((g0.n + BN - 1) / BN);
  const int64_t t1 = g1 ? ((g1->m + BM - 1) / BM) * ((g1->n + BN - 1) / BN) : 0;
  if (gp.split == 0) {  // keep the first slot filled: the kernel picks by workgroup index
    gp.g[0] = gp.g[1];
    gp.split = t1;
    if (t1 == 0) return hipSuccess;
    hipLaunchKernelGGL((gemm_kernel<KIND, AF, BF, OUT, MASK, BK, CFG, kEpiNone>), dim3((unsigned)t1),
                       dim3(NT), CFG::LDS, st, gp);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((gemm_kernel<KIND, AF, BF, OUT, MASK, BK, CFG, kEpiNone>),
                     dim3((unsigned)(gp.split + t1)), dim3(NT), CFG::LDS, st, gp);
  return hipGetLastError();
}

// The largest tile that still gives the 256 compute units a tile each (see pick of gemm_act.hip; each
// output's sum runs in the same order in all of them, so the choice changes no result).
template <int KIND, int AF, int BF, int OUT, bool MASK>
static hipError_t pick(const GemmArgs& g, const GemmArgs* g1, hipStream_t st) {
  constexpr int BK = GEMM_BK;
  auto tiles = [&](int64_t bt) {
    auto of = [&](const GemmArgs& p) { return ((p.m + bt - 1) / bt) * ((p.n + bt - 1) / bt); };
    return of(g) + (g1 ? of(*g1) : 0);
  };
  if (tiles(256) >= 224) return launch_cfg<KIND, AF, BF, OUT, MASK, BK, BigTile>(g, g1, st);
  if (tiles(128) >= 224) return launch_cfg<KIND, AF, BF, OUT, MASK, BK, MidTile>(g, g1, st);
  return launch_cfg<KIND, AF, BF, OUT, MASK, BK, SmallTile>(g, g1, st);
}

template <int KIND, int AF, int BF, int OUT>
static hipError_t launch_t(const GemmArgs& g, const GemmArgs* g1, hipStream_t st) {
  const bool mask = needs_mask<KIND, GEMM_BK>(g) || (g1 && needs_mask<KIND, GEMM_BK>(*g1));
  return mask ? pick<KIND, AF, BF, OUT, true>(g, g1, st) : pick<KIND, AF, BF, OUT, false>(g, g1, st);
}

hipError_t launch_gemm_pair(const GemmArgs& g_in, const GemmArgs* g1_in, int kind, int afmt,
                            int bfmt, int out, hipStream_t st) {
  // The product with the longer contraction takes the first workgroups: its tiles run longer,
  // and dispatching the longer tasks first leaves a shorter tail when the two products' tiles
  // do not divide evenly over the compute units (each workgroup's outputs are its own, so the
  // order changes no result).
  const bool swap = g1_in && g1_in->k > g_in.k;
  const GemmArgs& g = swap ? *g1_in : g_in;
  const GemmArgs* g1 = swap ? &g_in : g1_in;
  if (kind == 0) {
    switch (out) {
      case 0: return launch_t<0, 0, 0, 0>(g, g1, st);
      case 1: return launch_t<0, 0, 0, 1>(g, g1, st);
      case 2: return launch_t<0, 0, 0, 2>(g, g1, st);
    }
    return hipErrorInvalidValue;
  }
  const int sel = afmt * 2 + bfmt;
#define HALO_FP8_CASE(AFv, BFv)                                       \
  if (sel == AFv * 2 + BFv) {                                         \
    if (out == 1) return launch_t<1, AFv, BFv, 1>(g, g1, st);         \
    if (out == 2) return launch_t<1, AFv, BFv, 2>(g, g1, st);         \
  }
  HALO_FP8_CASE(0, 0)
  HALO_FP8_CASE(0, 1)
  HALO_FP8_CASE(1, 0)
  HALO_FP8_CASE(1, 1)
#undef HALO_FP8_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_gemm(const GemmArgs& g, int kind, int afmt, int bfmt, int out, hipStream_t st) {
  return launch_gemm_pair(g, nullptr, kind, afmt, bfmt, out, st);
}

}  // namespace halo
