// act_grad.hip -- the layer's gradient at its pre-activation: dz = dy act'(z) in fp32, and the
// bias gradient db = sum over the rows of dz (gfx950).
//
// dz stays in fp32: it is rotated and quantised next, and a rounding to bf16 in between would
// move a code in a few per cent of the places (0.6 % of the products' result), which the
// formula does not have.
// A workgroup takes 512 columns (8 per lane, every wave the same columns) and a run of rows, its
// 4 waves in turn; a wave sums its rows, the waves are added in order through LDS, and a second
// launch adds the workgroups' partial rows in order.
#include "checkpoint.h"
#include "epilogue.h"
#include "halo_kernels.h"

namespace halo {

namespace {

constexpr int kCols = 512;

// z plain or kept in 8 bits; GLU: the gated layer's pair of halves from one read of dy (dz and db are
// then 2 n wide, z is 2 m rows of n).
template <typename T, bool GLU>
__global__ __launch_bounds__(256) void dz_kernel(DzArgs a, int64_t rows_per_wg, float* part) {
  constexpr int H = GLU ? 2 : 1;
  __shared__ float s[3][kCols];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t n = a.n, col = (int64_t)blockIdx.x * kCols + lane * 8;
  const bool in = col < n;  // n is a multiple of 8: a lane's columns are whole
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_wg, r1 = min(a.m, r0 + rows_per_wg);
  const int64_t groups = (n + kGroup - 1) / kGroup;
  float sum[H][8] = {};
  if (in) {
    for (int64_t r = r0 + w; r < r1; r += 4) {
      float d[8], z[H][8], g[H][8];
      load_cols<T>(static_cast<const T*>(a.dy) + r * n + col, 8, d);
      if (GLU || a.act != kActNone) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int64_t zr = r * H + h;
          if (a.kept == kKeptPlain) {
            load_cols<T>(static_cast<const T*>(a.z) + zr * n + col, 8, z[h]);
          } else {
            const uint2 q =
                *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.z) + zr * n + col);
            const uint32_t p = a.zp[zr * groups + col / kGroup];
            if (a.kept == kKeptI8) kept8<0>(q, p, z[h]);
            else kept8<1>(q, p, z[h]);
          }
        }
      }
      if constexpr (GLU) {
        gated_grad<8, sizeof(T) == 4>(a.act, d, z[0], z[1], g[0], g[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[0][e] = d[e];
        if (a.act != kActNone) slope_mul<8>(a.act, z[0], g[0]);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[h][e] += g[h][e];
        if (!a.dz) continue;
        float* o = a.dz + r * (n * H) + h * n + col;
        reinterpret_cast<float4*>(o)[0] = make_float4(g[h][0], g[h][1], g[h][2], g[h][3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(g[h][4], g[h][5], g[h][6], g[h][7]);
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (h > 0) __syncthreads();
    if (w > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[w - 1][e * 64 + lane] = sum[h][e];
    }
    __syncthreads();
    if (w == 0 && in) {
      float* o = part + (int64_t)blockIdx.y * (n * H) + h * n + col;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = ((sum[h][e] + s[0][e * 64 + lane]) + s[1][e * 64 + lane]) + s[2][e * 64 + lane];
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void part_sum_kernel(const float* part, int64_t parts, int64_t n,
                                                       T* db) {
  __shared__ float s[4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  float v = 0.f;
  if (col < n) {
#pragma unroll 8
    for (int64_t i = w; i < parts; i += 4) v += part[i * n + col];
  }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && col < n) elem_store<T>(db + col, (s[0][lane] + s[1][lane]) + (s[2][lane] + s[3][lane]));
}

int64_t rows_per(int64_t m, int64_t n) {
  const int64_t strips = n > 0 ? (n + kCols - 1) / kCols : 1;
  const int64_t want = (2048 + strips - 1) / strips;  // about 2048 workgroups in all
  const int64_t rows = (m + want - 1) / want;
  return rows < 16 ? 16 : rows;
}

template <typename T>
hipError_t run(const DzArgs& a, hipStream_t st) {
  const int64_t rows = rows_per(a.m, a.n), parts = (a.m + rows - 1) / rows;
  const int64_t width = a.glu ? 2 * a.n : a.n;
  const dim3 grid((unsigned)((a.n + kCols - 1) / kCols), (unsigned)parts);
  float* part = a.db ? a.part : nullptr;
  if (a.glu) hipLaunchKernelGGL((dz_kernel<T, true>), grid, dim3(256), 0, st, a, rows, part);
  else hipLaunchKernelGGL((dz_kernel<T, false>), grid, dim3(256), 0, st, a, rows, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.db) return e;
  hipLaunchKernelGGL((part_sum_kernel<T>), dim3((unsigned)((width + 63) / 64)), dim3(256), 0, st, part,
                     parts, width, static_cast<T*>(a.db));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dz(const DzArgs& a, int in_bf16, hipStream_t st) {
  return in_bf16 ? run<uint16_t>(a, st) : run<float>(a, st);
}

hipError_t launch_part_sum(const float* part, int64_t parts, int64_t n, uint16_t* db,
                           hipStream_t st) {
  hipLaunchKernelGGL((part_sum_kernel<uint16_t>), dim3((unsigned)((n + 63) / 64)), dim3(256), 0, st,
                     part, parts, n, db);
  return hipGetLastError();
}

int64_t act_grad_parts(int64_t m, int64_t n) {
  const int64_t rows = rows_per(m, n);
  return (m + rows - 1) / rows;
}

}  // namespace halo
