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

static int64_t tiles_of(const GemmArgs& p, int64_t bt) {
  return ((p.m + bt - 1) / bt) * ((p.n + bt - 1) / bt);
}

// fill_of a launch of one or two products: the second one's tiles, of the shorter contraction, run on
// the units that the first one's last round leaves idle, and behind it (2048 x 4096 over 4096 beside 4096 x
// 4096 over 2048: 384 tiles of 256 fill two rounds of the longer's half length, 109.7 us of a gradient
// against 114.9 in two launches and 118 on 128 tiles).
static double pair_fill(const GemmArgs& g, const GemmArgs* g1, int64_t bt, int64_t slots) {
  const int64_t t0 = tiles_of(g, bt);
  if (!g1 || tiles_of(*g1, bt) == 0) return fill_of(t0, slots);
  const int64_t t1 = tiles_of(*g1, bt), rest = t0 % slots;
  const double p = (double)g.k / (double)g1->k;  // rounds of the second in one of the first
  const int64_t beside = rest ? (slots - rest) * (int64_t)p : 0;
  const int64_t behind = t1 > beside ? t1 - beside : 0;
  const double rounds = (double)((t0 + slots - 1) / slots) * p + (double)((behind + slots - 1) / slots);
  return ((double)t0 * p + (double)t1) / ((double)slots * rounds);
}

// The tile (see big_tiles, and pick_act of gemm_act.h).  Each output's sum runs in the same order in all
// of them, so the choice changes no result.
enum Tile { kBig, kMid, kDeep, kSmall };
static Tile tile_of(const GemmArgs& g, const GemmArgs* g1) {
  auto tiles = [&](int64_t bt) { return tiles_of(g, bt) + (g1 ? tiles_of(*g1, bt) : 0); };
  if (big_tiles(tiles(128), pair_fill(g, g1, 256, 256), pair_fill(g, g1, 128, 512), g.k)) return kBig;
  if (tiles(128) > 256) return kMid;
  return tiles(64) > 512 ? kDeep : kSmall;
}

// Microseconds of a launch on a tile, to choose between launches: the device's rate with all compute
// units busy, or its longest tile's slabs (128 bytes of the contraction) one after the other.  The
// constants are INT8's; FP8's rates lie within a tenth of them (22016 x 4096 x 4096 on 256 tiles 379 and
// 346 us) and favour the same launch.  Over 476 gradients the choice lies 2 % above the best of one launch
// on any tile and two, and none over 3 % behind one launch on 256 tiles.
static double launch_us(const GemmArgs& g, const GemmArgs* g1, Tile t) {
  constexpr double kRate[] = {2.2e9, 1.8e9, 1.9e9, 1.2e9};  // operations per us
  constexpr double kSlab[] = {1.3, 0.75, 0.5, 0.22};
  auto ops = [](const GemmArgs& p) { return 2.0 * (double)p.m * (double)p.n * (double)p.k; };
  const double work = (ops(g) + (g1 ? ops(*g1) : 0.0)) / kRate[t];
  const double chain = (double)g.k / 128 * kSlab[t];  // g's contraction is the longer one
  return work > chain ? work : chain;
}

// Two products with tiles of their own, one launch after the other, against one launch on common
// tiles: a few tiles of a long contraction beside many of a short one keep their compute units long
// after the others' are done (gradients of few tokens: 128 x 4096 over 22016 beside 22016 x 4096 over
// 128 takes 186 us in one launch, 44 + 55 in two; 512 tokens 266 and 91 + 80; a gated layer's gradient of
// 1024 tokens 507 a call and 459).
static bool apart(const GemmArgs& g, const GemmArgs& g1) {
  constexpr double kLaunch = 8.0;  // of a second launch and the first one's tail
  return launch_us(g, nullptr, tile_of(g, nullptr)) + launch_us(g1, nullptr, tile_of(g1, nullptr)) +
             kLaunch < launch_us(g, &g1, tile_of(g, &g1));
}

template <int KIND, int AF, int BF, int OUT, bool MASK>
static hipError_t pick(const GemmArgs& g, const GemmArgs* g1, hipStream_t st) {
  constexpr int BK = GEMM_BK;
  switch (tile_of(g, g1)) {
    case kBig: return launch_cfg<KIND, AF, BF, OUT, MASK, BK, BigTile>(g, g1, st);
    case kMid: return launch_cfg<KIND, AF, BF, OUT, MASK, BK, MidTile>(g, g1, st);
    case kDeep: return launch_cfg<KIND, AF, BF, OUT, MASK, BK, DeepTile>(g, g1, st);
    default: return launch_cfg<KIND, AF, BF, OUT, MASK, BK, SmallTile>(g, g1, st);
  }
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
  if (g1 && g.m > 0 && g.n > 0 && g1->m > 0 && g1->n > 0 && apart(g, *g1)) {
    const hipError_t e = launch_gemm_pair(g, nullptr, kind, afmt, bfmt, out, st);
    return e == hipSuccess ? launch_gemm_pair(*g1, nullptr, kind, afmt, bfmt, out, st) : e;
  }
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
