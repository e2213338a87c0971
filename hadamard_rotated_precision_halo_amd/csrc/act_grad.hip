// act_grad.hip -- the layer's gradient at its pre-activation: dz = dy act'(z) in fp32, and the
// bias gradient db = sum over the rows of dz (gfx950).
//
// dz stays in fp32: it is rotated and quantised next, and a rounding to bf16 in between would
// move a code in a few per cent of the places (0.6 % of the products' result), which the
// formula does not have.
// A workgroup takes 512 columns (8 per lane, every wave the same columns) and a run of rows, its
// 4 waves in turn; a wave sums its rows, the waves are added in order through LDS, and a second
// launch adds the workgroups' partial rows in order.
#include "epilogue.h"
#include "halo_kernels.h"

namespace halo {

namespace {

constexpr int kCols = 512;

template <typename T>
__global__ __launch_bounds__(256) void act_grad_kernel(const T* dy, const T* z, int act, int64_t m,
                                                       int64_t n, int64_t rows_per_wg, float* dz,
                                                       float* part) {
  __shared__ float s[3][kCols];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * kCols + lane * 8;
  const int cnt = (int)max((int64_t)0, min((int64_t)8, n - col));
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_wg, r1 = min(m, r0 + rows_per_wg);
  float sum[8] = {};
  if (cnt > 0) {
    for (int64_t r = r0 + w; r < r1; r += 4) {
      float d[8], zv[8];
      load_cols<T>(dy + r * n + col, cnt, d);
      if (act != kActNone) {
        load_cols<T>(z + r * n + col, cnt, zv);
        slope_mul<8>(act, zv, d);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += d[e];
      if (dz) {
        float* o = dz + r * n + col;
        if (cnt == 8) {
          reinterpret_cast<float4*>(o)[0] = make_float4(d[0], d[1], d[2], d[3]);
          reinterpret_cast<float4*>(o)[1] = make_float4(d[4], d[5], d[6], d[7]);
        } else {
          for (int e = 0; e < cnt; ++e) o[e] = d[e];
        }
      }
    }
  }
  if (!part) return;
  if (w > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[w - 1][e * 64 + lane] = sum[e];
  }
  __syncthreads();
  if (w == 0 && cnt > 0) {
    float* o = part + (int64_t)blockIdx.y * n + col;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = ((sum[e] + s[0][e * 64 + lane]) + s[1][e * 64 + lane]) + s[2][e * 64 + lane];
      if (e < cnt) o[e] = v;
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
hipError_t run(const void* dy, const void* z, int act, int64_t m, int64_t n, float* dz, void* db,
               float* part, hipStream_t st) {
  const int64_t rows = rows_per(m, n), parts = (m + rows - 1) / rows;
  hipLaunchKernelGGL((act_grad_kernel<T>), dim3((unsigned)((n + kCols - 1) / kCols), (unsigned)parts),
                     dim3(256), 0, st, static_cast<const T*>(dy), static_cast<const T*>(z), act, m,
                     n, rows, dz, db ? part : nullptr);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !db) return e;
  hipLaunchKernelGGL((part_sum_kernel<T>), dim3((unsigned)((n + 63) / 64)), dim3(256), 0, st, part,
                     parts, n, static_cast<T*>(db));
  return hipGetLastError();
}

}  // namespace

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

hipError_t launch_act_grad(const void* dy, const void* z, int act, int in_bf16, int64_t m,
                           int64_t n, float* dz, void* db, float* part, hipStream_t st) {
  return in_bf16 ? run<uint16_t>(dy, z, act, m, n, dz, db, part, st)
                 : run<float>(dy, z, act, m, n, dz, db, part, st);
}

}  // namespace halo
