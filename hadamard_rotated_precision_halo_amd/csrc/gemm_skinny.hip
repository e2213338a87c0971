// gemm_skinny.hip -- the layer's product with its epilogue for a few rows of activations (serving
// single tokens and small batches) on gfx950.
//
// What is computed is that of gemm_tile.h's epilogue form: acc[i, j] = sum_t a[i, t] b[j, t] over
// 8-bit codes, z = (acc sa[i]) sb[j] + bias[j], y = act(z) + residual.
//
// Bound by reading b (the weights' codes) once.  A workgroup takes 16 rows of b and its 8 waves
// split the contraction, so a 4096 x 4096 layer keeps all 256 compute units busy and every byte
// of b is asked for at the start; the codes go from memory into MFMA operands directly (16 rows x
// 64 bytes per load, no LDS), since no other wave uses them.  The rows of a (up to 16) are read from
// the L2.  The waves' partial sums meet in LDS and are added in wave order.  For the fewest rows
// the rotation and quantisation of a run in the same kernel (skinny_fused_kernel).
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

// The epilogue of one element.
template <typename T>
__device__ __forceinline__ void finish(const GemmArgs& g, float acc, float sa, int64_t row,
                                       int64_t col) {
  const int64_t at = row * g.ldc + col;
  float z = (acc * sa) * g.sb[col];
  if (g.bias) z += elem_f32<T>(reinterpret_cast<const T*>(g.bias) + col);
  constexpr bool FULL = sizeof(T) == 4;
  float y;
  switch (g.act) {
    case kActRelu: y = act_of<kActRelu, FULL>(z); break;
    case kActSilu: y = act_of<kActSilu, FULL>(z); break;
    case kActGeluTanh: y = act_of<kActGeluTanh, FULL>(z); break;
    case kActGeluErf: y = act_of<kActGeluErf, FULL>(z); break;
    default: y = z;
  }
  if (g.res) y += elem_f32<T>(reinterpret_cast<const T*>(g.res) + at);
  elem_store<T>(reinterpret_cast<T*>(g.c) + at, y);
  if (g.z) elem_store<T>(reinterpret_cast<T*>(g.z) + at, z);
}

// An operand's fragments of UN steps from s on; chunks past the contraction or the wave's steps
// read the row's first bytes (the caller zeroes them).
template <int KIND, int UN>
__device__ __forceinline__ void load_steps(v4i (&f)[UN][Step<KIND>::CH], const char* p, int s, int s1,
                                       int64_t k_end, int q16) {
  using S = Step<KIND>;
#pragma unroll
  for (int u = 0; u < UN; ++u)
#pragma unroll
    for (int h = 0; h < S::CH; ++h) {
      const int64_t k = (int64_t)(s + u) * S::K + h * 64;
      const bool in = s + u < s1 && k + q16 * 16 < k_end;
      f[u][h] = *reinterpret_cast<const v4i*>(p + (in ? k : -(int64_t)q16 * 16));
    }
}

// The waves' partial tiles, added in wave order, and the epilogue: element (row i % 16, column
// i / 16) of thread i is value column % 4 of lane (row, column / 4).
template <typename T, int KIND, typename Scale>
__device__ __forceinline__ void join(const GemmArgs& g, const typename Step<KIND>::Acc (*s_acc)[64],
                                     int64_t n0, Scale scale) {
  using E = typename std::conditional<KIND == 0, int, float>::type;
  const int i = threadIdx.x, row = i & 15, cl = i >> 4;
  const int64_t col = n0 + cl;
  if (i >= 256 || row >= g.m || col >= g.n) return;
  E sum = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += s_acc[w][(cl >> 2) * 16 + row][cl & 3];
  finish<T>(g, (float)sum, scale(row), row, col);
}

template <int KIND, int OUT>
__global__ __launch_bounds__(64 * kWaves) void skinny_kernel(GemmArgs g) {
  using S = Step<KIND>;
  using T = typename std::conditional<OUT == 2, uint16_t, float>::type;
  constexpr int UN = 8 / S::CH;  // steps whose loads are in flight together
  __shared__ typename S::Acc s_acc[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, q16 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const char* pb = static_cast<const char*>(g.b) + min(n0 + r16, g.n - 1) * g.ldb + q16 * 16;
  const char* pa = static_cast<const char*>(g.a) + min((int64_t)r16, g.m - 1) * g.lda + q16 * 16;

  typename S::Acc acc = {};
  const int steps = (int)((g.k + S::K - 1) / S::K);
  const int s0 = (int)((int64_t)steps * wave / kWaves), s1 = (int)((int64_t)steps * (wave + 1) / kWaves);
  for (int s = s0; s < s1; s += UN) {
    v4i fb[UN][S::CH], fa[UN][S::CH];
    load_steps<KIND, UN>(fb, pb, s, s1, g.k, q16);
    load_steps<KIND, UN>(fa, pa, s, s1, g.k, q16);
#pragma unroll
    for (int u = 0; u < UN; ++u) {
#pragma unroll
      for (int h = 0; h < S::CH; ++h) {
        const int64_t k = (int64_t)(s + u) * S::K + h * 64;
        const int keep = s + u < s1 && k + q16 * 16 < g.k ? -1 : 0;
        fb[u][h] &= keep;
        if constexpr (KIND == 1) fa[u][h] &= keep;  // 0 x NaN is not 0
      }
      acc = S::mul(fb[u], fa[u], acc);
    }
  }
  s_acc[wave][lane] = acc;
  __syncthreads();
  join<T, KIND>(g, s_acc, n0, [&](int row) { return g.sa[row]; });
}

// Butterflies of one stage across lanes at distance 2^S where the block spans them.
template <int S>
__device__ __forceinline__ void lane_stage(float* v, int lane, int block) {
  if (block <= (8 << S)) return;
  const float c = (lane >> S) & 1 ? -1.f : 1.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = xbutterfly<S>(v[e], c);
}

// Rotation of a 512-element slice, 8 consecutive elements per lane, by blocks of `block` (a
// wave-uniform power of two up to 512): stages in increasing index-bit order with the operand
// order of the rows pass (fwht_wave.h), so the values are the same bits.
__device__ __forceinline__ void rotate8(float* v, int lane, int block) {
#pragma unroll
  for (int d = 1; d < 8; d *= 2) {
    if (block > d) {
#pragma unroll
      for (int i = 0; i < 8; i += 2 * d)
#pragma unroll
        for (int t = i; t < i + d; ++t) {
          const float p = v[t], q = v[t + d];
          v[t] = p + q;
          v[t + d] = p - q;
        }
    }
  }
  lane_stage<0>(v, lane, block);
  lane_stage<1>(v, lane, block);
  lane_stage<2>(v, lane, block);
  lane_stage<3>(v, lane, block);
  lane_stage<4>(v, lane, block);
  lane_stage<5>(v, lane, block);
}

// The same product with the rotation and quantisation of a's rows inside: f describes the rows
// pass (x, block, signs), whose codes stay in LDS.  Every workgroup repeats that pass; it runs
// while the workgroup's first reads of b are on their way, and the call is one launch without a
// scratch (one token, 4096 x 4096 INT8: 10.2 us a call, 14.3 us with the pass in a launch of its
// own).  A wave takes 512-element slices of the rows, kUnits at most.
constexpr int kUnits = 4;

template <typename TX, int KIND, int OUT>
__global__ __launch_bounds__(64 * kWaves) void skinny_fused_kernel(GemmArgs g, FqArgs f) {
  using S = Step<KIND>;
  using T = typename std::conditional<OUT == 2, uint16_t, float>::type;
  constexpr int UN = 8 / S::CH;
  __shared__ typename S::Acc s_acc[kWaves][64];
  __shared__ float s_unit[kWaves * kUnits], s_sa[16];
  extern __shared__ __attribute__((aligned(16))) char s_codes[];  // [m][pitch]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q16 = lane >> 4;
  const int kq = (int)g.k, m = (int)g.m;
  const int pitch = kq + 16;  // rows 16 bytes apart in the banks
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const char* pb = static_cast<const char*>(g.b) + min(n0 + r16, g.n - 1) * g.ldb + q16 * 16;
  const int steps = (kq + S::K - 1) / S::K;
  const int s0 = steps * wave / kWaves, s1 = steps * (wave + 1) / kWaves;
  v4i fb[UN][S::CH];
  load_steps<KIND, UN>(fb, pb, s0, s1, g.k, q16);

  // ---- the rows of x ---------------------------------------------------------------------
  const int slices = (kq + 511) / 512, units = m * slices;
  float v[kUnits][8];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = wave + i * kWaves;
    if (u >= units) break;
    const int row = u / slices, pos = (u - row * slices) * 512 + lane * 8;
    const TX* x = reinterpret_cast<const TX*>(f.x) + (int64_t)row * f.ldx;
    if (pos < kq) {
      load8_vec<TX>(x, pos, f.in_len, f.signs, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = wave + i * kWaves;
    if (u >= units) break;
    rotate8(v[i], lane, f.block);
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[i][e]));
    mx = wave_max(mx);
    if (lane == 0) s_unit[u] = mx;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = wave + i * kWaves;
    if (u >= units) break;
    const int row = u / slices, pos = (u - row * slices) * 512 + lane * 8;
    float mx = 0.f;
    for (int t = 0; t < slices; ++t) mx = fmaxf(mx, s_unit[row * slices + t]);
    float pre;
    const float mul = code_mul(f.qmax, mx, &pre);
    if (pre != 1.f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= pre;
    }
    if (pos < kq) *reinterpret_cast<uint2*>(s_codes + row * pitch + pos) = encode8<KIND>(v[i], mul);
    if (pos == 0) s_sa[row] = mx / f.denom;
  }
  __syncthreads();

  // ---- the product -----------------------------------------------------------------------
  typename S::Acc acc = {};
  const char* la = s_codes + min(r16, m - 1) * pitch + q16 * 16;
  for (int s = s0; s < s1; s += UN) {
    if (s > s0) load_steps<KIND, UN>(fb, pb, s, s1, g.k, q16);
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      v4i fa[S::CH];
#pragma unroll
      for (int h = 0; h < S::CH; ++h) {
        const int k = (s + u) * S::K + h * 64;
        const bool in = s + u < s1 && k + q16 * 16 < kq;
        const v4i zero = {0, 0, 0, 0};
        fa[h] = *reinterpret_cast<const v4i*>(la + (in ? k : -q16 * 16));
        fa[h] = in ? fa[h] : zero;
        if constexpr (KIND == 1) fb[u][h] = in ? fb[u][h] : zero;  // 0 x NaN is not 0
      }
      acc = S::mul(fb[u], fa, acc);
    }
  }
  s_acc[wave][lane] = acc;
  __syncthreads();
  join<T, KIND>(g, s_acc, n0, [&](int row) { return s_sa[row]; });
}

template <typename TX, int KIND, int OUT>
hipError_t run_fused(const GemmArgs& g, const FqArgs& f, hipStream_t st) {
  const int lds = (int)(g.m * (g.k + 16));
  hipLaunchKernelGGL((skinny_fused_kernel<TX, KIND, OUT>), dim3((unsigned)((g.n + 15) / 16)),
                     dim3(64 * kWaves), lds, st, g, f);
  return hipGetLastError();
}

template <typename TX>
hipError_t run_fused_x(const GemmArgs& g, const FqArgs& f, int kind, int out, hipStream_t st) {
  if (kind == 0) return out == 1 ? run_fused<TX, 0, 1>(g, f, st) : run_fused<TX, 0, 2>(g, f, st);
  return out == 1 ? run_fused<TX, 1, 1>(g, f, st) : run_fused<TX, 1, 2>(g, f, st);
}

template <int KIND, int OUT>
hipError_t run(const GemmArgs& g, hipStream_t st) {
  hipLaunchKernelGGL((skinny_kernel<KIND, OUT>), dim3((unsigned)((g.n + 15) / 16)),
                     dim3(64 * kWaves), 0, st, g);
  return hipGetLastError();
}

}  // namespace

// Up to 16 rows of 512 and more codes whose slices (of 512) the 8 waves hold at once, in blocks
// that a slice holds whole, and whose codes fit the default LDS limit.
bool skinny_fused_ok(int64_t m, int64_t kq, int block) {
  return m >= 1 && m <= 16 && kq >= 512 && block <= 512 &&
         m * ((kq + 511) / 512) <= kWaves * kUnits && m * (kq + 16) <= 48 * 1024;
}

hipError_t launch_skinny_fused(const GemmArgs& g, const FqArgs& f, int in_bf16, int kind, int out,
                               hipStream_t st) {
  return in_bf16 ? run_fused_x<uint16_t>(g, f, kind, out, st)
                 : run_fused_x<float>(g, f, kind, out, st);
}

hipError_t launch_gemm_skinny(const GemmArgs& g, int kind, int out, hipStream_t st) {
  if (kind == 0) return out == 1 ? run<0, 1>(g, st) : run<0, 2>(g, st);
  return out == 1 ? run<1, 1>(g, st) : run<1, 2>(g, st);
}

}  // namespace halo
