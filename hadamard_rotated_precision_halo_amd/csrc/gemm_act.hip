// gemm_act.hip -- the layer's product with its epilogue (bias, activation, residual, the kept
// pre-activation): the kernel of gemm_tile.h with EPI, on the tile that fills the device.
#include "gemm_tile.h"

namespace halo {

namespace {

// 128 x 128 and 64 x 64 tiles of 4 waves, two workgroups per compute unit.
using MidTile = TileCfg<128, 2, 2, 2>;
using SmallTile = TileCfg<64, 2, 2, 4>;

template <int KIND, int OUT, bool MASK, typename CFG>
hipError_t run(const GemmArgs& g, hipStream_t st) {
  constexpr int BK = GEMM_BK, NT = 64 * CFG::WM * CFG::WN;
  const hipError_t e =
      allow_dynamic_lds<&gemm_kernel<KIND, 0, 0, OUT, MASK, BK, CFG, true>>(CFG::LDS);
  if (e != hipSuccess) return e;
  GemmPair gp{};
  gp.g[0] = gp.g[1] = g;
  gp.split = ((g.m + CFG::BT - 1) / CFG::BT) * ((g.n + CFG::BT - 1) / CFG::BT);
  if (gp.split == 0) return hipSuccess;
  hipLaunchKernelGGL((gemm_kernel<KIND, 0, 0, OUT, MASK, BK, CFG, true>), dim3((unsigned)gp.split),
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
  auto tiles = [&](int64_t bt) { return ((g.m + bt - 1) / bt) * ((g.n + bt - 1) / bt); };
  if (tiles(256) >= 224) return run<KIND, OUT, MASK, BigTile>(g, st);
  if (tiles(128) >= 224) return run<KIND, OUT, MASK, MidTile>(g, st);
  if (tiles(64) > 256) return run<KIND, OUT, MASK, SmallTile>(g, st);
  return launch_gemm_ksplit(g, KIND, OUT, st);
}

template <int KIND, int OUT>
hipError_t pick_mask(const GemmArgs& g, hipStream_t st) {
  return needs_mask<KIND, GEMM_BK>(g) ? pick<KIND, OUT, true>(g, st) : pick<KIND, OUT, false>(g, st);
}

}  // namespace

hipError_t launch_gemm_act(const GemmArgs& g, int kind, int out, hipStream_t st) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  if (g.m <= kSkinnyRows) return launch_gemm_skinny(g, kind, out, st);
  if (kind == 0) return out == 1 ? pick_mask<0, 1>(g, st) : pick_mask<0, 2>(g, st);
  return out == 1 ? pick_mask<1, 1>(g, st) : pick_mask<1, 2>(g, st);
}

}  // namespace halo
