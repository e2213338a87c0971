// gemm_ksplit.hip -- the layer's product with its epilogue where the output has too few tiles for
// the kernel of gemm_tile.h (batches of some tens to some hundreds of rows), on gfx950.
//
// What is computed is that of gemm_tile.h's epilogue form.  A workgroup of 4 waves owns a 64 x 64
// output tile and its waves split the contraction: wave w takes K slabs w, w + 4, .. (128 bytes of
// every row) of both operands, with a private two-slab ring in LDS (64 KB of loads in flight per
// two waves), and accumulates the whole tile.  So every staged byte is read from LDS once (waves
// that share a slab and split the tile read each byte twice, and the LDS was their bound), and no
// wave waits for another before the end, where the four partial tiles meet in LDS and are added in
// wave order.  Bound by the loads: a tile reads 128 bytes for each K byte, 1.4 MB per compute unit
// at 203 x 4096 x 11008 FP8, 12 to 14 us at the 100 to 120 bytes/ns that a unit loads of data in
// its L2; the product takes 21 us of a call's 26 (4 % less with its LDS reads and MFMAs left out;
// touching the lines of b ahead of their loads made it half as long again).
#include "gemm_tile.h"

namespace halo {

namespace {

constexpr int kT = 64;                    // tile rows and columns
constexpr int kSlab = 2 * kT * GEMM_BK;   // bytes of both operands
constexpr int kPitch = kT + 4;            // words of a staged row
constexpr int kLds = 4 * 2 * kSlab;
static_assert(4 * kT * kPitch * 4 <= kLds, "the partial tiles fit where the rings were");

// GLU: the gated layer's epilogue: a tile is 32 columns of the gate and the 32 of the up projection
// that they meet.
template <int KIND, int OUT, bool MASK, bool GLU>
__global__ __launch_bounds__(256, 1) void ksplit_kernel(GemmArgs g) {
  using SL = Slab<GEMM_BK, kT>;
  using Acc = typename std::conditional<KIND == 0, v16i, v16f>::type;
  using Frag = typename std::conditional<KIND == 0, v4i, v8i>::type;
  using T = typename std::conditional<OUT == 2, uint16_t, float>::type;
  constexpr int KS = GEMM_BK / (KIND == 0 ? 32 : 64);  // MFMA steps per slab
  constexpr int RPF = KIND == 0 ? 1 : 2;               // 16-byte reads per fragment
  constexpr int NI = kT / SL::RPI;                     // load instructions per operand and slab
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // each XCD (workgroup i runs on XCD i % 8) gets a contiguous run of tiles, rows fastest, so its
  // L2 reads a column strip of b once
  const int tiles_m = (int)((g.m + kT - 1) / kT);
  constexpr int YN = GLU ? kT / 2 : kT;  // output columns of a tile
  const int total = tiles_m * (int)((g.n + YN - 1) / YN);
  const int q8 = total / 8, r8 = total % 8, xcd = blockIdx.x % 8, slot = blockIdx.x / 8;
  const int tile = xcd < r8 ? xcd * (q8 + 1) + slot : r8 * (q8 + 1) + (xcd - r8) * q8 + slot;
  const int64_t m0 = (int64_t)(tile % tiles_m) * kT, n0 = (int64_t)(tile / tiles_m) * YN;

  const __amdgpu_buffer_rsrc_t ra = raw_rsrc(g.a), rb = raw_rsrc(g.b);
  uint32_t aoff[NI], boff[NI];  // byte offsets of the lane's chunk in slab 0 (operands are < 4 GB)
  uint32_t cb[NI];              // of which within the row
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = i * SL::RPI + lane / SL::CHUNKS;
    cb[i] = (uint32_t)(((lane % SL::CHUNKS) ^ SL::swz(r)) << 4);
    aoff[i] = (uint32_t)(min(m0 + r, g.m - 1) * g.lda);  // clamped rows feed unused outputs
    const int64_t br = GLU ? min(n0 + r % YN, g.n - 1) + (r < YN ? 0 : g.n) : min(n0 + r, g.n - 1);
    boff[i] = (uint32_t)(br * g.ldb);
  }
  const int nk = (int)((g.k + GEMM_BK - 1) / GEMM_BK);
  const int count = nk > wave ? (nk - wave + 3) / 4 : 0;  // slabs of this wave
  const uint32_t klast = (uint32_t)g.k - 16;
  char* ring = smem + wave * 2 * kSlab;
  auto stage = [&](int i) __attribute__((always_inline)) {  // the wave's slab i into its slot
    char* sa = ring + (i & 1) * kSlab;
    char* sb = sa + kSlab / 2;
    const uint32_t kb = (uint32_t)(wave + 4 * i) * GEMM_BK;
#pragma unroll
    for (int q = 0; q < NI; ++q) {
      uint32_t kc = kb + cb[q];
      if constexpr (MASK) kc = min(kc, klast);  // past k: any chunk of the row, zeroed below
      dma16(ra, aoff[q] + kc, (lds_void*)(sa + q * 1024));
      dma16(rb, boff[q] + kc, (lds_void*)(sb + q * 1024));
    }
  };

  Acc acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  const int fr = lane & 31, fh = lane >> 5;
  if (count > 0) stage(0);
  if (count > 1) stage(1);
  for (int i = 0; i < count; ++i) {
    // the wave's own loads of slab i have landed (those of slab i + 1 may still be under way)
    if (i + 1 < count) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * NI) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const char* sa = ring + (i & 1) * kSlab;
    const char* sb = sa + kSlab / 2;
    Frag fa[KS][2], fb[KS][2];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int h = 0; h < RPF; ++h) {
          const int c = KIND == 0 ? ks * 2 + fh : ks * 4 + fh * 2 + h;
          int keep = -1;
          if constexpr (MASK) keep = (wave + 4 * i) * GEMM_BK + c * 16 < g.k ? -1 : 0;
          const v4i va = *reinterpret_cast<const v4i*>(sa + SL::off(t * 32 + fr, c)) & keep;
          const v4i vb = *reinterpret_cast<const v4i*>(sb + SL::off(t * 32 + fr, c)) & keep;
          if constexpr (KIND == 0) {
            fa[ks][t] = va;
            fb[ks][t] = vb;
          } else if (h == 0) {
            fa[ks][t].lo = va;
            fb[ks][t].lo = vb;
          } else {
            fa[ks][t].hi = va;
            fb[ks][t].hi = vb;
          }
        }
    if (i + 2 < count) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot has been read
      stage(i + 2);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if constexpr (KIND == 0)
            acc[x][y] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[ks][x], fa[ks][y], acc[x][y], 0, 0, 0);
          else
            acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                fb[ks][x], fa[ks][y], acc[x][y], 0, 0, 0, 127, 0, 127);
        }
  }

  // ---- join and epilogue -----------------------------------------------------------------
  // lane (fr, fh) holds of tile (x, y) row y * 32 + fr, columns x * 32 + q * 8 + fh * 4 + [0, 4)
  __syncthreads();  // every wave is done with its ring, and its loads have landed
  using E = typename std::conditional<KIND == 0, int, float>::type;
  using E4 = typename std::conditional<KIND == 0, int4, float4>::type;
  E* part = reinterpret_cast<E*>(smem);
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        E4 w;
        w.x = acc[x][y][q * 4];
        w.y = acc[x][y][q * 4 + 1];
        w.z = acc[x][y][q * 4 + 2];
        w.w = acc[x][y][q * 4 + 3];
        *reinterpret_cast<E4*>(part + (wave * kT + y * 32 + fr) * kPitch + x * 32 + q * 8 + fh * 4) = w;
      }
  __syncthreads();
  if constexpr (GLU) {  // a thread per row and 8 columns of both halves
    const int cg = (tid & 3) * 8, r = tid >> 2;
    const int64_t col0 = n0 + cg, row = m0 + r;
    const int cnt = (int)max((int64_t)0, min((int64_t)8, g.n - col0));
    const float sar = g.sa[min(row, g.m - 1)];
    float z[2][8], y[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      E s[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = part[r * kPitch + h * YN + cg + e];
#pragma unroll
      for (int w = 1; w < 4; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += part[(w * kT + r) * kPitch + h * YN + cg + e];
      float sbv[8], bias[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) sbv[e] = bias[e] = 0.f;
      if (cnt > 0) load_cols<float>(g.sb + h * g.n + col0, cnt, sbv);
      if (g.bias && cnt > 0) load_cols<T>(reinterpret_cast<const T*>(g.bias) + h * g.n + col0, cnt, bias);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[h][e] = __builtin_fmaf((float)s[e] * sar, sbv[e], bias[e]);
    }
    act8<T>(g.act, z[0], y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= z[1][e];
    if (g.kept) {
      keep_cols(g.kept, g.z, g.zp, 2 * row, g.n, col0, row < g.m, z[0]);
      keep_cols(g.kept, g.z, g.zp, 2 * row + 1, g.n, col0, row < g.m, z[1]);
    }
    if (row >= g.m || cnt <= 0) return;
    store_cols<T>(reinterpret_cast<T*>(g.c) + row * g.ldc + col0, cnt, y);
    if (g.z && !g.kept) {
      store_cols<T>(reinterpret_cast<T*>(g.z) + 2 * row * g.n + col0, cnt, z[0]);
      store_cols<T>(reinterpret_cast<T*>(g.z) + (2 * row + 1) * g.n + col0, cnt, z[1]);
    }
    return;
  }
  const int cg = (tid & 7) * 8;
  const int64_t col0 = n0 + cg;
  const int cnt = (int)max((int64_t)0, min((int64_t)8, g.n - col0));
  if (cnt <= 0 && !g.kept) return;  // z kept in 8 bits: a quad's lanes stay together
  float sbv[8], bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sbv[e] = bias[e] = 0.f;
  if (cnt > 0) load_cols<float>(g.sb + col0, cnt, sbv);
  if (g.bias && cnt > 0) load_cols<T>(reinterpret_cast<const T*>(g.bias) + col0, cnt, bias);
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int r = it * 32 + (tid >> 3);
    const int64_t row = m0 + r;
    if (row >= g.m) continue;
    float res[8];
    const int64_t at = row * g.ldc + col0;
    if (g.res && cnt > 0) load_cols<T>(reinterpret_cast<const T*>(g.res) + at, cnt, res);
    E s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = part[r * kPitch + cg + e];
#pragma unroll
    for (int w = 1; w < 4; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += part[(w * kT + r) * kPitch + cg + e];
    const float sar = g.sa[row];
    float z[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = __builtin_fmaf((float)s[e] * sar, sbv[e], bias[e]);
    act8<T>(g.act, z, y);
    if (g.res) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] += res[e];
    }
    if (g.kept) keep_cols(g.kept, g.z, g.zp, row, g.n, col0, true, z);
    if (cnt <= 0) continue;
    store_cols<T>(reinterpret_cast<T*>(g.c) + at, cnt, y);
    if (g.z && !g.kept) store_cols<T>(reinterpret_cast<T*>(g.z) + at, cnt, z);
  }
}

template <int KIND, int OUT, bool MASK, bool GLU>
hipError_t run_form(const GemmArgs& g, hipStream_t st) {
  const hipError_t e = allow_dynamic_lds<&ksplit_kernel<KIND, OUT, MASK, GLU>>(kLds);
  if (e != hipSuccess) return e;
  constexpr int YN = GLU ? kT / 2 : kT;
  const int64_t tiles = ((g.m + kT - 1) / kT) * ((g.n + YN - 1) / YN);
  hipLaunchKernelGGL((ksplit_kernel<KIND, OUT, MASK, GLU>), dim3((unsigned)tiles), dim3(256), kLds, st, g);
  return hipGetLastError();
}

template <int KIND, int OUT, bool MASK>
hipError_t run(const GemmArgs& g, hipStream_t st) {
  return g.glu ? run_form<KIND, OUT, MASK, true>(g, st) : run_form<KIND, OUT, MASK, false>(g, st);
}

template <int KIND, int OUT>
hipError_t run_mask(const GemmArgs& g, hipStream_t st) {
  return g.k % GEMM_BK != 0 ? run<KIND, OUT, true>(g, st) : run<KIND, OUT, false>(g, st);
}

}  // namespace

hipError_t launch_gemm_ksplit(const GemmArgs& g, int kind, int out, hipStream_t st) {
  if (kind == 0) return out == 1 ? run_mask<0, 1>(g, st) : run_mask<0, 2>(g, st);
  return out == 1 ? run_mask<1, 1>(g, st) : run_mask<1, 2>(g, st);
}

}  // namespace halo
