// checkpoint.hip -- rows of activations to 8-bit codes with a power of two per group of 32, and back
// (checkpoint.h has the form), on gfx950.
//
// Bound by memory: bf16 rows move 3.03 bytes a value each way.  A lane takes 8 consecutive values (a quad
// a group), TPR lanes a row, the workgroup's lanes 256 / TPR rows at a time, and every lane has the
// loads of kItems chunks under way together.
#include "checkpoint.h"
#include "halo_kernels.h"

namespace halo {

namespace {

constexpr int kThreads = 256, kItems = 4;

// cnt (0 .. 8) elements at p, zeros behind them; any alignment of whole elements.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* p, int cnt) {
    if (cnt == 8) {
      w = load16u(p);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < cnt ? p[e] : 0u;
      w = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
  }
  __device__ __forceinline__ void get(float* o) const { unpack_bf16x8(w, o); }
};
template <>
struct Raw8<float> {
  uint4 w[2];
  __device__ __forceinline__ void load(const float* p, int cnt) {
    if (cnt == 8) {
      w[0] = load16u(p);
      w[1] = load16u(p + 4);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < cnt ? __float_as_uint(p[e]) : 0u;
      w[0] = make_uint4(v[0], v[1], v[2], v[3]);
      w[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
  __device__ __forceinline__ void get(float* o) const {
    unpack16<float>(w[0], o);
    unpack16<float>(w[1], o + 4);
  }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, int cnt, const float* v) {
  if (cnt == 8) {
#pragma unroll
    for (int h = 0; h < 8 / RowType<T>::VEC; ++h)
      store16u(p + h * RowType<T>::VEC, pack16<T>(v + h * RowType<T>::VEC));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < cnt) elem_store<T>(p + e, v[e]);
  }
}

typedef int v2i_any __attribute__((ext_vector_type(2), aligned(1)));

// Walks a workgroup's chunks: its rows `step` at a time, a row's chunks `stride` apart.
struct Walk {
  int64_t row, end;
  int c, c0, chunks, stride, step;
  __device__ __forceinline__ void next() {
    c += stride;
    if (c >= chunks) {
      c = c0;
      row += step;
    }
  }
};

__device__ __forceinline__ Walk walk_of(const KeepArgs& a) {
  Walk w;
  w.chunks = (int)((a.cols + kGroup - 1) / kGroup) * 4;
  w.stride = a.tpr;
  w.step = kThreads / a.tpr;
  w.c0 = w.c = threadIdx.x % a.tpr;
  w.row = (int64_t)blockIdx.x * a.rows_per_wg + threadIdx.x / a.tpr;
  w.end = min(a.rows, (int64_t)(blockIdx.x + 1) * a.rows_per_wg);
  if (w.c >= w.chunks) w.row = w.end;
  return w;
}

template <typename T, int QT>
__global__ __launch_bounds__(kThreads) void pack_kernel(KeepArgs a) {
  Walk w = walk_of(a);
  const T* x = static_cast<const T*>(a.x);
  // quads stay whole: chunks come in fours and a row's chunks are dealt to whole quads
  while (w.row < w.end) {
    Raw8<T> raw[kItems];
    Walk u = w;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int64_t left = a.cols - (int64_t)u.c * 8;
      const int cnt = u.row < u.end ? (int)max((int64_t)0, min((int64_t)8, left)) : 0;
      raw[i].load(x + u.row * a.ldx + (int64_t)u.c * 8, cnt);
      u.next();
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (w.row >= w.end) return;
      float v[8];
      raw[i].get(v);
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[e]));
      const uint32_t s = group_power<QT>(quad_umax(top));
      const uint2 q = keep8<QT>(v, s);
      const int64_t left = a.cols - (int64_t)w.c * 8;
      uint8_t* d = static_cast<uint8_t*>(a.codes) + w.row * a.ldc + (int64_t)w.c * 8;
      if (left >= 8) {
        *reinterpret_cast<v2i_any*>(d) = (v2i_any){(int)q.x, (int)q.y};
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < left) d[e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
      }
      if ((w.c & 3) == 0) a.powers[w.row * a.ldp + (w.c >> 2)] = (uint8_t)s;
      w.next();
    }
  }
}

template <typename T, int QT>
__global__ __launch_bounds__(kThreads) void unpack_kernel(KeepArgs a) {
  Walk w = walk_of(a);
  const uint8_t* codes = static_cast<const uint8_t*>(a.codes);
  while (w.row < w.end) {
    uint2 q[kItems];
    uint32_t s[kItems];
    Walk u = w;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int64_t left = a.cols - (int64_t)u.c * 8;
      const uint8_t* p = codes + u.row * a.ldc + (int64_t)u.c * 8;
      q[i] = make_uint2(0u, 0u);
      s[i] = 0;
      if (u.row < u.end) {
        if (left >= 8) {
          const v2i_any t = *reinterpret_cast<const v2i_any*>(p);
          q[i] = make_uint2((uint32_t)t.x, (uint32_t)t.y);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t b = e < left ? p[e] : 0u;
            if (e < 4) q[i].x |= b << (8 * e);
            else q[i].y |= b << (8 * (e - 4));
          }
        }
        s[i] = a.powers[u.row * a.ldp + (u.c >> 2)];
      }
      u.next();
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (w.row >= w.end) return;
      float v[8];
      kept8<QT>(q[i], s[i], v);
      const int64_t left = a.cols - (int64_t)w.c * 8;
      store8<T>(static_cast<T*>(a.x_out) + w.row * a.ldx + (int64_t)w.c * 8,
                (int)max((int64_t)0, min((int64_t)8, left)), v);
      w.next();
    }
  }
}

template <typename T, int QT>
hipError_t run(KeepArgs a, bool pack, hipStream_t st) {
  const int64_t chunks = (a.cols + kGroup - 1) / kGroup * 4;
  // lanes per row: the most that leave no more than an eighth of them idle over a row, else those
  // that leave the fewest idle
  int64_t best = -1;
  for (int t = kThreads; t >= 4; t /= 2) {
    const int64_t cover = (chunks + t - 1) / t * t;
    if (best < 0 || cover < best) {
      best = cover;
      a.tpr = t;
    }
    if (cover * 8 <= chunks * 9) break;
  }
  const int64_t step = kThreads / a.tpr, per_row = (chunks + a.tpr - 1) / a.tpr;
  // rows of a workgroup: at least kItems chunks a lane, while there are many workgroups
  int64_t passes = (kItems + per_row - 1) / per_row;
  while (passes > 1 && (a.rows + step * passes - 1) / (step * passes) < 512) passes /= 2;
  a.rows_per_wg = step * passes;
  // more rows than a launch has workgroups for go in pieces
  const int64_t most = max_workgroups(kThreads);
  for (int64_t r = 0; r < a.rows; r += most * a.rows_per_wg) {
    KeepArgs b = a;
    b.rows = min(a.rows - r, most * a.rows_per_wg);
    if (pack) b.x = static_cast<const T*>(a.x) + r * a.ldx;
    else b.x_out = static_cast<T*>(a.x_out) + r * a.ldx;
    b.codes = static_cast<uint8_t*>(a.codes) + r * a.ldc;
    b.powers = a.powers + r * a.ldp;
    const dim3 grid((unsigned)((b.rows + b.rows_per_wg - 1) / b.rows_per_wg));
    if (pack) hipLaunchKernelGGL((pack_kernel<T, QT>), grid, dim3(kThreads), 0, st, b);
    else hipLaunchKernelGGL((unpack_kernel<T, QT>), grid, dim3(kThreads), 0, st, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_keep(const KeepArgs& a, int in_bf16, int qt, bool pack, hipStream_t st) {
  if (in_bf16) return qt == 0 ? run<uint16_t, 0>(a, pack, st) : run<uint16_t, 1>(a, pack, st);
  return qt == 0 ? run<float, 0>(a, pack, st) : run<float, 1>(a, pack, st);
}

}  // namespace halo
