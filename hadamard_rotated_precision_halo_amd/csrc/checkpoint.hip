// checkpoint.hip -- rows of activations to 8-bit codes with a power of two per group of 32, and back
// (checkpoint.h has the form), on gfx950.
//
// Bound by memory: bf16 rows move 3.03 bytes a value each way.  A lane takes chunks of 8 consecutive
// values (a quad a group), dealt to the workgroups through all rows, so that no lane idles at a row's end;
// every lane has the loads of kItems chunks under way together.
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

// A workgroup's chunks: kThreads kItems consecutive ones of all rows', four (a group) at least a row.
// Its first chunk's row and place are found once; the others lie behind it by less than a row where
// rows are long, else by a quotient of small numbers.
struct Place {
  int64_t row;
  int c;
  bool in;
};
struct Items {
  int64_t row, last;  // row of the first chunk, chunks of the launch from it on
  int off, chunks;    // the first chunk's place in its row
  float inv;
  __device__ __forceinline__ explicit Items(const KeepArgs& a) {
    chunks = a.chunks;
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kItems);
    row = first / chunks;
    off = (int)(first - row * chunks);
    last = a.rows * chunks - first;
    inv = 1.f / (float)chunks;
  }
  __device__ __forceinline__ Place at(int i) const {
    Place p;
    p.in = i < last;
    int local = off + i, r;
    if (chunks >= kThreads * kItems) {
      r = local >= chunks ? 1 : 0;
    } else {  // both below 2^12: the quotient is off by one at most
      r = (int)((float)local * inv);
      r += local - r * chunks >= chunks ? 1 : 0;
      r -= local < r * chunks ? 1 : 0;
    }
    p.row = row + r;
    p.c = local - r * chunks;
    return p;
  }
};

template <typename T, int QT>
__global__ __launch_bounds__(kThreads) void pack_kernel(KeepArgs a) {
  const Items items(a);
  const T* x = static_cast<const T*>(a.x);
  Raw8<T> raw[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const Place p = items.at(i * kThreads + threadIdx.x);
    const int64_t left = a.cols - (int64_t)p.c * 8;
    const int cnt = p.in ? (int)max((int64_t)0, min((int64_t)8, left)) : 0;
    raw[i].load(x + p.row * a.ldx + (int64_t)p.c * 8, cnt);
  }
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const Place p = items.at(i * kThreads + threadIdx.x);
    float v[8];
    raw[i].get(v);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[e]));
    const uint32_t s = group_power<QT>(quad_umax(top));  // quads are whole: chunks come in fours
    if (!p.in) return;
    const uint2 q = keep8<QT>(v, s);
    const int64_t left = a.cols - (int64_t)p.c * 8;
    uint8_t* d = static_cast<uint8_t*>(a.codes) + p.row * a.ldc + (int64_t)p.c * 8;
    if (left >= 8) {
      *reinterpret_cast<v2i_any*>(d) = (v2i_any){(int)q.x, (int)q.y};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) d[e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
    }
    if ((p.c & 3) == 0) a.powers[p.row * a.ldp + (p.c >> 2)] = (uint8_t)s;
  }
}

template <typename T, int QT>
__global__ __launch_bounds__(kThreads) void unpack_kernel(KeepArgs a) {
  const Items items(a);
  const uint8_t* codes = static_cast<const uint8_t*>(a.codes);
  uint2 q[kItems];
  uint32_t s[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const Place p = items.at(i * kThreads + threadIdx.x);
    const int64_t left = a.cols - (int64_t)p.c * 8;
    const uint8_t* d = codes + p.row * a.ldc + (int64_t)p.c * 8;
    q[i] = make_uint2(0u, 0u);
    s[i] = 0;
    if (!p.in) continue;
    if (left >= 8) {
      const v2i_any t = *reinterpret_cast<const v2i_any*>(d);
      q[i] = make_uint2((uint32_t)t.x, (uint32_t)t.y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = e < left ? d[e] : 0u;
        if (e < 4) q[i].x |= b << (8 * e);
        else q[i].y |= b << (8 * (e - 4));
      }
    }
    s[i] = a.powers[p.row * a.ldp + (p.c >> 2)];
  }
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const Place p = items.at(i * kThreads + threadIdx.x);
    if (!p.in) return;
    float v[8];
    kept8<QT>(q[i], s[i], v);
    const int64_t left = a.cols - (int64_t)p.c * 8;
    store8<T>(static_cast<T*>(a.x_out) + p.row * a.ldx + (int64_t)p.c * 8,
              (int)max((int64_t)0, min((int64_t)8, left)), v);
  }
}

template <typename T, int QT>
hipError_t run(KeepArgs a, bool pack, hipStream_t st) {
  a.chunks = (int)((a.cols + kGroup - 1) / kGroup) * 4;
  // more rows than a launch has workgroups for go in pieces
  const int64_t most = max_workgroups(kThreads) * (kThreads * kItems) / a.chunks;
  for (int64_t r = 0; r < a.rows; r += most) {
    KeepArgs b = a;
    b.rows = a.rows - r < most ? a.rows - r : most;
    if (pack) b.x = static_cast<const T*>(a.x) + r * a.ldx;
    else b.x_out = static_cast<T*>(a.x_out) + r * a.ldx;
    b.codes = static_cast<uint8_t*>(a.codes) + r * a.ldc;
    b.powers = a.powers + r * a.ldp;
    const int64_t per = kThreads * kItems;
    const dim3 grid((unsigned)((b.rows * b.chunks + per - 1) / per));
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
