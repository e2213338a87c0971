// gemm_skinny.hip -- the layer's product with its epilogue for a few rows of activations (serving
// single tokens and small batches) on gfx950.
//
// What is computed is that of gemm_tile.h's epilogue form: acc[i, j] = sum_t a[i, t] b[j, t] over
// 8-bit codes, z = (acc sa[i]) sb[j] + bias[j], y = act(z) + residual.
//
// Bound by reading b (the weights' codes) once.  A workgroup takes 16 rows of b and its 8 waves
// split the contraction, so a 4096 x 4096 layer keeps all 256 compute units busy and every byte
// of b is asked for at the start; the codes go from memory into MFMA operands directly (16 rows x
// 64 bytes per load, no LDS), since no other wave uses them.  MT 16-row tiles of a are read from
// the L2.  The waves' partial sums meet in LDS and are added in wave order.
#include "epilogue.h"
#include "halo_kernels.h"

namespace halo {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
constexpr int kWaves = 8;

// Contraction order: a step is 64 (INT8) or 128 (FP8) codes; lane l holds row l % 16 and the
// 16-byte chunk l / 16 of each 64 bytes of the step, of a and b alike.
template <int KIND>
struct Step;
template <>
struct Step<0> {
  static constexpr int K = 64, CH = 1;
  using Acc = v4i;
  __device__ static __forceinline__ Acc mul(const v4i* b, const v4i* a, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(b[0], a[0], c, 0, 0, 0);
  }
};
template <>
struct Step<1> {
  static constexpr int K = 128, CH = 2;
  using Acc = v4f;
  __device__ static __forceinline__ Acc mul(const v4i* b, const v4i* a, Acc c) {
    v8i x, y;
    x.lo = b[0];
    x.hi = b[1];
    y.lo = a[0];
    y.hi = a[1];
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 0, 0, 0, 127, 0, 127);
  }
};

template <int KIND, int OUT, int MT>
__global__ __launch_bounds__(64 * kWaves) void skinny_kernel(GemmArgs g) {
  using S = Step<KIND>;
  using T = typename std::conditional<OUT == 2, uint16_t, float>::type;
  constexpr int UN = MT <= 2 ? 8 / S::CH : 4 / S::CH;  // steps whose loads are in flight together
  __shared__ typename S::Acc s_acc[kWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, q16 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const char* pb = static_cast<const char*>(g.b) + min(n0 + r16, g.n - 1) * g.ldb + q16 * 16;
  const char* pa[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
    pa[t] = static_cast<const char*>(g.a) + min((int64_t)(t * 16 + r16), g.m - 1) * g.lda + q16 * 16;

  typename S::Acc acc[MT] = {};
  const int steps = (int)((g.k + S::K - 1) / S::K);
  const int s0 = (int)((int64_t)steps * wave / kWaves), s1 = (int)((int64_t)steps * (wave + 1) / kWaves);
  for (int s = s0; s < s1; s += UN) {
    v4i fb[UN][S::CH], fa[UN][MT][S::CH];
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int h = 0; h < S::CH; ++h) {
        // a chunk past the contraction or the wave's steps reads the row's first bytes
        const int64_t k = (int64_t)(s + u) * S::K + h * 64;
        const bool in = s + u < s1 && k + q16 * 16 < g.k;
        fb[u][h] = *reinterpret_cast<const v4i*>(pb + (in ? k : -(int64_t)q16 * 16));
#pragma unroll
        for (int t = 0; t < MT; ++t)
          fa[u][t][h] = *reinterpret_cast<const v4i*>(pa[t] + (in ? k : -(int64_t)q16 * 16));
      }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
#pragma unroll
      for (int h = 0; h < S::CH; ++h) {
        const int64_t k = (int64_t)(s + u) * S::K + h * 64;
        const int keep = s + u < s1 && k + q16 * 16 < g.k ? -1 : 0;
        fb[u][h] &= keep;
        if constexpr (KIND == 1) {  // 0 x NaN is not 0
#pragma unroll
          for (int t = 0; t < MT; ++t) fa[u][t][h] &= keep;
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = S::mul(fb[u], fa[u][t], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) s_acc[wave][t][lane] = acc[t];
  __syncthreads();
  // lane (r16, q16) of tile t holds row t * 16 + r16 and columns n0 + q16 * 4 + [0, 4)
  for (int i = threadIdx.x; i < MT * 64; i += 64 * kWaves) {
    const int t = i >> 6, l = i & 63;
    typename S::Acc v = s_acc[0][t][l];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += s_acc[w][t][l];
    const int64_t row = t * 16 + (l & 15), col = n0 + (l >> 4) * 4;
    if (row >= g.m) continue;
    const float sa = g.sa[row];
    const int64_t at = row * g.ldc + col;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (col + e >= g.n) break;
      float z = ((float)v[e] * sa) * g.sb[col + e];
      if (g.bias) z += elem_f32<T>(reinterpret_cast<const T*>(g.bias) + col + e);
      float y;
      switch (g.act) {
        case kActRelu: y = act_of<kActRelu>(z); break;
        case kActSilu: y = act_of<kActSilu>(z); break;
        case kActGeluTanh: y = act_of<kActGeluTanh>(z); break;
        case kActGeluErf: y = act_of<kActGeluErf>(z); break;
        default: y = z;
      }
      if (g.res) y += elem_f32<T>(reinterpret_cast<const T*>(g.res) + at + e);
      elem_store<T>(reinterpret_cast<T*>(g.c) + at + e, y);
      if (g.z) elem_store<T>(reinterpret_cast<T*>(g.z) + at + e, z);
    }
  }
}

template <int KIND, int OUT>
hipError_t run(const GemmArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)((g.n + 15) / 16)), block(64 * kWaves);
  if (g.m <= 16) hipLaunchKernelGGL((skinny_kernel<KIND, OUT, 1>), grid, block, 0, st, g);
  else if (g.m <= 32) hipLaunchKernelGGL((skinny_kernel<KIND, OUT, 2>), grid, block, 0, st, g);
  else hipLaunchKernelGGL((skinny_kernel<KIND, OUT, 4>), grid, block, 0, st, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_skinny(const GemmArgs& g, int kind, int out, hipStream_t st) {
  if (kind == 0) return out == 1 ? run<0, 1>(g, st) : run<0, 2>(g, st);
  return out == 1 ? run<1, 1>(g, st) : run<1, 2>(g, st);
}

}  // namespace halo
