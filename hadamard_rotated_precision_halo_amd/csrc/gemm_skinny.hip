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
// the rotation and quantisation of a run in the same kernel (skinny_fused_kernel).  The gated layer
// (y = act(zg) zu) takes 8 rows of the gate and the 8 of the up projection that they meet; with z kept
// in 8 bits a workgroup takes the 32 columns of a group (skinny_kept_kernel).
#include "checkpoint.h"
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

// The row of b that lane row r16 of a workgroup holds (clamped rows feed unused outputs), and the
// output columns of a workgroup.
template <bool GLU>
constexpr int kCols = GLU ? 8 : 16;
template <bool GLU>
__device__ __forceinline__ int64_t brow(const GemmArgs& g, int64_t n0, int r16) {
  if constexpr (GLU) return min(n0 + (r16 & 7), g.n - 1) + (r16 < 8 ? 0 : g.n);
  return min(n0 + r16, g.n - 1);
}

// z of column col of b.
template <typename T>
__device__ __forceinline__ float z_of(const GemmArgs& g, float acc, float sa, int64_t col) {
  float z = (acc * sa) * g.sb[col];
  if (g.bias) z += elem_f32<T>(reinterpret_cast<const T*>(g.bias) + col);
  return z;
}
template <typename T>
__device__ __forceinline__ float act1(int act, float z) {
  constexpr bool FULL = sizeof(T) == 4;
  switch (act) {
    case kActRelu: return act_of<kActRelu, FULL>(z);
    case kActSilu: return act_of<kActSilu, FULL>(z);
    case kActGeluTanh: return act_of<kActGeluTanh, FULL>(z);
    case kActGeluErf: return act_of<kActGeluErf, FULL>(z);
    default: return z;
  }
}

// z of a workgroup's group of 32 columns until it is coded: [half x 16 + row][column].
constexpr int kZPitch = kGroup + 4;
typedef float ZTile[kZPitch];

// The epilogue of one element, and of one gated pair; KEEP: z goes to column zc of the tile.
template <typename T, bool KEEP>
__device__ __forceinline__ void finish_pair(const GemmArgs& g, float gate, float up, float sa,
                                            int64_t row, int64_t col, ZTile* s_z, int zc) {
  const float zg = z_of<T>(g, gate, sa, col), zu = z_of<T>(g, up, sa, g.n + col);
  elem_store<T>(reinterpret_cast<T*>(g.c) + row * g.ldc + col, act1<T>(g.act, zg) * zu);
  if constexpr (KEEP) {
    s_z[row][zc] = zg;
    s_z[16 + row][zc] = zu;
  } else if (g.z) {
    T* z = reinterpret_cast<T*>(g.z) + 2 * row * g.n + col;
    elem_store<T>(z, zg);
    elem_store<T>(z + g.n, zu);
  }
}
template <typename T, bool KEEP>
__device__ __forceinline__ void finish(const GemmArgs& g, float acc, float sa, int64_t row,
                                       int64_t col, ZTile* s_z, int zc) {
  const int64_t at = row * g.ldc + col;
  const float z = z_of<T>(g, acc, sa, col);
  float y = act1<T>(g.act, z);
  if (g.res) y += elem_f32<T>(reinterpret_cast<const T*>(g.res) + at);
  elem_store<T>(reinterpret_cast<T*>(g.c) + at, y);
  if constexpr (KEEP) s_z[row][zc] = z;
  else if (g.z) elem_store<T>(reinterpret_cast<T*>(g.z) + at, z);
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
template <typename T, int KIND, bool GLU, bool KEEP, typename Scale>
__device__ __forceinline__ void join(const GemmArgs& g, const typename Step<KIND>::Acc (*s_acc)[64],
                                     int64_t n0, Scale scale, int i, ZTile* s_z = nullptr,
                                     int z0 = 0) {
  using E = typename std::conditional<KIND == 0, int, float>::type;
  const int row = i & 15, cl = i >> 4;
  const int64_t col = n0 + cl;
  if (cl >= kCols<GLU> || row >= g.m || col >= g.n) return;
  E sum = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += s_acc[w][(cl >> 2) * 16 + row][cl & 3];
  if constexpr (GLU) {
    E up = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) up += s_acc[w][((cl + 8) >> 2) * 16 + row][cl & 3];
    return finish_pair<T, KEEP>(g, (float)sum, (float)up, scale(row), row, col, s_z, z0 + cl);
  }
  finish<T, KEEP>(g, (float)sum, scale(row), row, col, s_z, z0 + cl);
}

template <int KIND, int OUT, bool GLU>
__global__ __launch_bounds__(64 * kWaves) void skinny_kernel(GemmArgs g) {
  using S = Step<KIND>;
  using T = typename std::conditional<OUT == 2, uint16_t, float>::type;
  // steps whose loads are in flight together: 8 of 64 codes, 2 of 128, so that the registers leave 7 and 8
  // waves per SIMD (FP8 with 4 of them: 4 waves, 16 x 14336 x 4096 24.8 us a call for 22.8)
  constexpr int UN = KIND == 0 ? 8 : 2;
  __shared__ typename S::Acc s_acc[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, q16 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kCols<GLU>;
  const char* pb = static_cast<const char*>(g.b) + brow<GLU>(g, n0, r16) * g.ldb + q16 * 16;
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
  join<T, KIND, GLU, false>(g, s_acc, n0, [&](int row) { return g.sa[row]; }, threadIdx.x);
}

// The same with z kept in 8 bits: a workgroup holds the 2 (gated: 4) runs of columns that make a group
// of 32.  Every sum runs as above, so y and z have the same bits however z is kept.  Two 64-byte loads of
// every run are in flight together: with eight, steps behind a wave's last are read again (gated, 16 x 2 x
// 512 x 2048 a call 18.7 us for 14.5).  Another kernel whose waves split the contraction through the LDS took
// 13.8 there, and 66 us for 75 at 16 x 2 x 4096 x 11008, with other last bits.
template <int KIND, int OUT, bool GLU>
__global__ __launch_bounds__(64 * kWaves) void skinny_kept_kernel(GemmArgs g) {
  using S = Step<KIND>;
  using T = typename std::conditional<OUT == 2, uint16_t, float>::type;
  constexpr int UN = 2 / S::CH, RUNS = kGroup / kCols<GLU>, H = GLU ? 2 : 1;
  static_assert(RUNS * 16 * kCols<GLU> == 64 * kWaves, "a thread per element of the group's rows");
  __shared__ typename S::Acc s_acc[RUNS][kWaves][64];
  __shared__ ZTile s_z[16 * H];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, q16 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kGroup;
  const char* pa = static_cast<const char*>(g.a) + min((int64_t)r16, g.m - 1) * g.lda + q16 * 16;
  const char* pb[RUNS];
#pragma unroll
  for (int r = 0; r < RUNS; ++r)  // (a run behind the last column reads the last one: unused)
    pb[r] = static_cast<const char*>(g.b) + brow<GLU>(g, n0 + r * kCols<GLU>, r16) * g.ldb + q16 * 16;

  typename S::Acc acc[RUNS] = {};
  const int steps = (int)((g.k + S::K - 1) / S::K);
  const int s0 = (int)((int64_t)steps * wave / kWaves), s1 = (int)((int64_t)steps * (wave + 1) / kWaves);
  for (int s = s0; s < s1; s += UN) {
    v4i fb[RUNS][UN][S::CH], fa[UN][S::CH];
#pragma unroll
    for (int r = 0; r < RUNS; ++r) load_steps<KIND, UN>(fb[r], pb[r], s, s1, g.k, q16);
    load_steps<KIND, UN>(fa, pa, s, s1, g.k, q16);
#pragma unroll
    for (int u = 0; u < UN; ++u) {
#pragma unroll
      for (int h = 0; h < S::CH; ++h) {
        const int64_t k = (int64_t)(s + u) * S::K + h * 64;
        const int keep = s + u < s1 && k + q16 * 16 < g.k ? -1 : 0;
#pragma unroll
        for (int r = 0; r < RUNS; ++r) fb[r][u][h] &= keep;
        if constexpr (KIND == 1) fa[u][h] &= keep;  // 0 x NaN is not 0
      }
#pragma unroll
      for (int r = 0; r < RUNS; ++r) acc[r] = S::mul(fb[r][u], fa[u], acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < RUNS; ++r) s_acc[r][wave][lane] = acc[r];
  __syncthreads();
  const int t = threadIdx.x, run = t / (16 * kCols<GLU>);
  join<T, KIND, GLU, true>(g, s_acc[run], n0 + run * kCols<GLU>, [&](int row) { return g.sa[row]; },
                           t % (16 * kCols<GLU>), s_z, run * kCols<GLU>);
  __syncthreads();
  // a quad per row and half, 8 columns a lane (n is a multiple of 8: a lane's columns are whole)
  const int part = (t & 3) * 8, row = (t >> 2) & 15, h = t >> 6;
  if (h >= H) return;
  const int64_t col = n0 + part;
  const bool in = row < g.m && col < g.n;
  float z[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = in ? s_z[h * 16 + row][part + e] : 0.f;
  keep_cols(g.kept, g.z, g.zp, (int64_t)row * H + h, g.n, col, in, z);
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
// own).  A wave takes 512-element slices of the rows, kUnits at most.  More output columns than
// kFusedGrid workgroups hold are dealt to them in turn: a workgroup keeps its codes of a, and reads
// its next rows of b while it joins the last ones' sums.
constexpr int kUnits = 4;
constexpr int kFusedGrid = 512;  // two workgroups per compute unit

template <typename TX, int KIND, int OUT, bool GLU>
__global__ __launch_bounds__(64 * kWaves) void skinny_fused_kernel(GemmArgs g, FqArgs f) {
  using S = Step<KIND>;
  using T = typename std::conditional<OUT == 2, uint16_t, float>::type;
  constexpr int UN = 8 / S::CH;
  __shared__ typename S::Acc s_acc[2][kWaves][64];
  __shared__ float s_unit[kWaves * kUnits], s_sa[16];
  extern __shared__ __attribute__((aligned(16))) char s_codes[];  // [m][pitch]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q16 = lane >> 4;
  const int kq = (int)g.k, m = (int)g.m;
  const int pitch = kq + 16;  // rows 16 bytes apart in the banks
  const int tiles = (int)((g.n + kCols<GLU> - 1) / kCols<GLU>);
  auto rows_of_b = [&](int tile) __attribute__((always_inline)) {
    return static_cast<const char*>(g.b) + brow<GLU>(g, (int64_t)tile * kCols<GLU>, r16) * g.ldb +
           q16 * 16;
  };
  const char* pb = rows_of_b(blockIdx.x);
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
  const char* la = s_codes + min(r16, m - 1) * pitch + q16 * 16;
  int turn = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1) {
    typename S::Acc acc = {};
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
    if (tile + (int)gridDim.x < tiles) {
      pb = rows_of_b(tile + gridDim.x);
      load_steps<KIND, UN>(fb, pb, s0, s1, g.k, q16);
    }
    // the turns alternate between two areas: a barrier lies between a join and the next sums there
    s_acc[turn][wave][lane] = acc;
    __syncthreads();
    join<T, KIND, GLU, false>(g, s_acc[turn], (int64_t)tile * kCols<GLU>,
                              [&](int row) { return s_sa[row]; }, threadIdx.x);
  }
}

template <typename TX, int KIND, int OUT>
hipError_t run_fused(const GemmArgs& g, const FqArgs& f, hipStream_t st) {
  const int lds = (int)(g.m * (g.k + 16));
  const int64_t tiles = g.glu ? (g.n + 7) / 8 : (g.n + 15) / 16;
  const dim3 grid((unsigned)(tiles < kFusedGrid ? tiles : kFusedGrid));
  if (g.glu)
    hipLaunchKernelGGL((skinny_fused_kernel<TX, KIND, OUT, true>), grid, dim3(64 * kWaves), lds, st, g,
                       f);
  else
    hipLaunchKernelGGL((skinny_fused_kernel<TX, KIND, OUT, false>), grid, dim3(64 * kWaves), lds, st, g,
                       f);
  return hipGetLastError();
}

template <typename TX>
hipError_t run_fused_x(const GemmArgs& g, const FqArgs& f, int kind, int out, hipStream_t st) {
  if (kind == 0) return out == 1 ? run_fused<TX, 0, 1>(g, f, st) : run_fused<TX, 0, 2>(g, f, st);
  return out == 1 ? run_fused<TX, 1, 1>(g, f, st) : run_fused<TX, 1, 2>(g, f, st);
}

template <int KIND, int OUT, bool GLU>
hipError_t run_form(const GemmArgs& g, hipStream_t st) {
  if (g.kept)
    hipLaunchKernelGGL((skinny_kept_kernel<KIND, OUT, GLU>), dim3((unsigned)((g.n + kGroup - 1) / kGroup)),
                       dim3(64 * kWaves), 0, st, g);
  else
    hipLaunchKernelGGL((skinny_kernel<KIND, OUT, GLU>),
                       dim3((unsigned)((g.n + kCols<GLU> - 1) / kCols<GLU>)), dim3(64 * kWaves), 0, st, g);
  return hipGetLastError();
}

template <int KIND, int OUT>
hipError_t run(const GemmArgs& g, hipStream_t st) {
  return g.glu ? run_form<KIND, OUT, true>(g, st) : run_form<KIND, OUT, false>(g, st);
}

}  // namespace

// Up to 16 rows of 512 and more codes whose slices (of 512) the 8 waves hold at once, in blocks
// that a slice holds whole.
bool skinny_fused_ok(int64_t m, int64_t kq, int block) {
  // their codes then fit the default LDS limit beside the sums, the slices' maxima and the scales
  static_assert(kWaves * kUnits * 512 + 16 * 16 + (int)sizeof(v4i) * 2 * kWaves * 64 +
                        4 * (kWaves * kUnits + 16) <= 64 * 1024, "LDS of skinny_fused_kernel");
  return m >= 1 && m <= 16 && kq >= 512 && block <= 512 && m * ((kq + 511) / 512) <= kWaves * kUnits;
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
