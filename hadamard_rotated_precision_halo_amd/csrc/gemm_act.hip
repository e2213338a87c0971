// gemm_act.hip -- the layer's product with its epilogue (bias, activation, residual, the kept
// pre-activation): the kernel of gemm_tile.h with EPI, on the tile that fills the device.
#include "gemm_tile.h"

namespace halo {

namespace {

// The gated layer's smallest: its waves are 64 columns of b wide, 32 of each half.  And its tile for
// at most one workgroup per compute unit: four slabs on their way instead of two, since no second
// workgroup covers the loads (203 x 2 x 5504 x 4096 FP8 with the rows pass: 23.2 us a call, 28.7 with
// two slabs or on the 64 tile; 17 rows of 2 x 11008: 29.7 against 39.6; from 257 tiles on two
// workgroups of two slabs are as good: 300 x 2 x 5504 29.7).
using SmallGluTile = TileCfg<64, 2, 1, 4>;
using DeepGluTile = TileCfg<128, 2, 2, 4>;

template <int KIND, int OUT, bool MASK, typename CFG, int EPI>
hipError_t run(const GemmArgs& g, hipStream_t st) {
  constexpr int BK = GEMM_BK, NT = 64 * CFG::WM * CFG::WN;
  const hipError_t e =
      allow_dynamic_lds<&gemm_kernel<KIND, 0, 0, OUT, MASK, BK, CFG, EPI>>(CFG::LDS);
  if (e != hipSuccess) return e;
  GemmPair gp{};
  gp.g[0] = gp.g[1] = g;
  constexpr int YN = EPI == kEpiGlu ? CFG::BT / 2 : CFG::BT;
  gp.split = ((g.m + CFG::BT - 1) / CFG::BT) * ((g.n + YN - 1) / YN);
  if (gp.split == 0) return hipSuccess;
  hipLaunchKernelGGL((gemm_kernel<KIND, 0, 0, OUT, MASK, BK, CFG, EPI>), dim3((unsigned)gp.split),
                     dim3(NT), CFG::LDS, st, gp);
  return hipGetLastError();
}

// The largest tile that still gives the 256 compute units a tile each, since a workgroup of the
// 256 tile needs a whole unit and fewer tiles leave units idle for the whole contraction, while
// smaller tiles read each operand more often from the L2 (8192 x 11008 x 4096 INT8: 403 us a call;
// on 128 x 128 tiles 9 % longer).  Below that 64 x 64 tiles: two
// workgroups per unit, or, where there is not even one tile per unit, the kernel whose waves
// split the contraction (256 x 4096 x 4096 INT8: 16.3 us a call against 18.4 us; but 400 rows:
// 24.3 against 21.7 us).
template <int KIND, int OUT, bool MASK>
hipError_t pick(const GemmArgs& g, hipStream_t st) {
  const int64_t n = g.glu ? 2 * g.n : g.n;
  auto tiles = [&](int64_t bt) { return ((g.m + bt - 1) / bt) * ((n + bt - 1) / bt); };
  if (tiles(256) >= 224)
    return g.glu ? run<KIND, OUT, MASK, BigTile, kEpiGlu>(g, st)
                 : run<KIND, OUT, MASK, BigTile, kEpiAct>(g, st);
  if (g.glu && tiles(128) >= 128 && tiles(128) <= 256)
    return run<KIND, OUT, MASK, DeepGluTile, kEpiGlu>(g, st);
  if (tiles(128) >= 224)
    return g.glu ? run<KIND, OUT, MASK, MidTile, kEpiGlu>(g, st)
                 : run<KIND, OUT, MASK, MidTile, kEpiAct>(g, st);
  if (tiles(64) > 256)
    return g.glu ? run<KIND, OUT, MASK, SmallGluTile, kEpiGlu>(g, st)
                 : run<KIND, OUT, MASK, SmallTile, kEpiAct>(g, st);
  return launch_gemm_ksplit(g, KIND, OUT, st);
}

template <int KIND, int OUT>
hipError_t pick_mask(const GemmArgs& g, hipStream_t st) {
  return needs_mask<KIND, GEMM_BK>(g) ? pick<KIND, OUT, true>(g, st) : pick<KIND, OUT, false>(g, st);
}

}  // namespace

hipError_t launch_gemm_act(const GemmArgs& g, int kind, int out, hipStream_t st) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  // the few-rows kernel's lanes hold single columns: z kept in 8 bits takes the next larger one
  if (g.m <= kSkinnyRows && !g.kept) return launch_gemm_skinny(g, kind, out, st);
  if (kind == 0) return out == 1 ? pick_mask<0, 1>(g, st) : pick_mask<0, 2>(g, st);
  return out == 1 ? pick_mask<1, 1>(g, st) : pick_mask<1, 2>(g, st);
}

}  // namespace halo
