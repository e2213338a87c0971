// gemm_act.h -- the layer's product with its epilogue (bias, activation, residual, the kept
// pre-activation): the kernel of gemm_tile.h with EPI, on the tile that fills the device.  The kernels
// that code z in 8 bits are built in a source file of their own, beside the others.
#pragma once

#include "gemm_tile.h"

namespace halo {

// The gated layer's smallest: its waves are 64 columns of b wide, 32 of each half.
using SmallGluTile = TileCfg<64, 2, 1, 4>;

template <int KIND, int OUT, bool MASK, typename CFG, int EPI>
static hipError_t run_act(const GemmArgs& g, hipStream_t st) {
  constexpr int BK = GEMM_BK, NT = 64 * CFG::WM * CFG::WN;
  const hipError_t e =
      allow_dynamic_lds<&gemm_kernel<KIND, 0, 0, OUT, MASK, BK, CFG, EPI>>(CFG::LDS);
  if (e != hipSuccess) return e;
  GemmPair gp{};
  gp.g[0] = gp.g[1] = g;
  constexpr int YN = EPI == kEpiGlu || EPI == kEpiGluKept ? CFG::BT / 2 : CFG::BT;
  gp.split = ((g.m + CFG::BT - 1) / CFG::BT) * ((g.n + YN - 1) / YN);
  if (gp.split == 0) return hipSuccess;
  hipLaunchKernelGGL((gemm_kernel<KIND, 0, 0, OUT, MASK, BK, CFG, EPI>), dim3((unsigned)gp.split),
                     dim3(NT), CFG::LDS, st, gp);
  return hipGetLastError();
}

// The largest tile that fills the device (see big_tiles), since smaller ones read each operand more
// often from the L2 (8192 x 11008 x 4096 INT8: 403 us a call; on 128 x 128 tiles 9 % longer).  64 x 64
// tiles while two of them per unit are enough, and below one tile per unit the kernel whose waves
// split the contraction.  INT8, 4096 long, with a rows pass, us on 128 tiles of four slabs, of two, on 64
// tiles, and split: 256 x 4096: 24.4, 28.5, 19.0, 16.4; 512 x 4096 26.2, 30.2, 23.4, 25.1; 700 x 4096
// 27.7, 30.6, 34.4, 33.4; 256 x 11008 26.2, 29.7, 32.8, 31.8; 300 x 11008 42.4, 30.6, 38.1, 38.5.  Up to
// 512 long two slabs do (1024 x 4096, 256 long: 14.1, 13.6).
template <int KIND, int OUT, bool MASK, bool KEPT>
static hipError_t pick_act(const GemmArgs& g, hipStream_t st) {
  constexpr int ACT = KEPT ? kEpiActKept : kEpiAct, GLU = KEPT ? kEpiGluKept : kEpiGlu;
  const int64_t n = g.glu ? 2 * g.n : g.n;
  auto tiles = [&](int64_t bt) { return ((g.m + bt - 1) / bt) * ((n + bt - 1) / bt); };
  if (big_tiles(tiles(128), fill_of(tiles(256), 256), fill_of(tiles(128), 512), g.k))
    return g.glu ? run_act<KIND, OUT, MASK, BigTile, GLU>(g, st)
                 : run_act<KIND, OUT, MASK, BigTile, ACT>(g, st);
  if (tiles(128) > 256 || (tiles(64) > 512 && g.k <= 4 * GEMM_BK))
    return g.glu ? run_act<KIND, OUT, MASK, MidTile, GLU>(g, st)
                 : run_act<KIND, OUT, MASK, MidTile, ACT>(g, st);
  if (tiles(64) > 512)
    return g.glu ? run_act<KIND, OUT, MASK, DeepTile, GLU>(g, st)
                 : run_act<KIND, OUT, MASK, DeepTile, ACT>(g, st);
  if (tiles(64) > 256)
    return g.glu ? run_act<KIND, OUT, MASK, SmallGluTile, GLU>(g, st)
                 : run_act<KIND, OUT, MASK, SmallTile, ACT>(g, st);
  return launch_gemm_ksplit(g, KIND, OUT, st);
}

template <int KIND, int OUT, bool KEPT>
static hipError_t pick_mask(const GemmArgs& g, hipStream_t st) {
  return needs_mask<KIND, GEMM_BK>(g) ? pick_act<KIND, OUT, true, KEPT>(g, st)
                                      : pick_act<KIND, OUT, false, KEPT>(g, st);
}

// kind: 0 INT8, 1 E4M3.  out: 1 fp32, 2 bf16.
template <bool KEPT>
static hipError_t launch_act(const GemmArgs& g, int kind, int out, hipStream_t st) {
  if (kind == 0) return out == 1 ? pick_mask<0, 1, KEPT>(g, st) : pick_mask<0, 2, KEPT>(g, st);
  return out == 1 ? pick_mask<1, 1, KEPT>(g, st) : pick_mask<1, 2, KEPT>(g, st);
}

hipError_t launch_gemm_act_kept(const GemmArgs& g, int kind, int out, hipStream_t st);

}  // namespace halo
