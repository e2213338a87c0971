// glu_rows.hip -- the rows pass of the gated layer's gradient on gfx950: dz = [dy u act'(g), dy act(g)]
// in fp32 from dy and z's halves g and u, stored for the columns pass, and rotated and quantised along
// its 2 n columns as the rows kernel of fwht_wave.h does it (natural-order butterflies over blocks of B
// contiguous indices, one absmax scale per row).
//
// A workgroup owns a row.  A wave holds 2048 columns of the gate's half and the same 2048 of the up
// half, 32 + 32 values per lane, so that dy, g and u are read once and the activation is evaluated once for
// both: the pass is bound by the vector ALU and by memory alike, and evaluating it for each half, with dz
// formed again by the columns pass in place of the store, took no less.  Half a slice: chunk j (of 8) of lane
// lo of a block's G = B / 32 lanes sits at block offset (j G + lo) 8, so the 3 low and the 2 high
// index bits are butterflied in registers and log2(G) stages cross lanes, in increasing bit order and
// with the operand order of a sequential fp32 butterfly.
//
// Where the block does not divide n, a block spans both halves and the up half's blocks start at other
// columns than the gate's: what lies behind the gate's whole blocks (its last columns, the up half, the
// zero padding) then passes through LDS to the lanes that hold its blocks (SHIFT).
#include "fwht_wave.h"

namespace halo {

namespace {

constexpr int kHalf = 2048;                              // columns of a half per wave
constexpr int kHalfStage = kHalf + kHalf / 256 * 32;     // its codes in LDS (stage_off)

template <int B>
struct HalfSlice {
  static constexpr int G = B / 32;  // lanes per block
  __device__ static __forceinline__ int off(int lane, int j) {
    return (lane / G) * B + (j * G + lane % G) * 8;
  }
};

__device__ __forceinline__ void put8(uint8_t* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <int D>
__device__ __forceinline__ void reg_stage32(float* v) {
#pragma unroll
  for (int i = 0; i < 32; i += 2 * D)
#pragma unroll
    for (int t = i; t < i + D; ++t) {
      const float p = v[t], q = v[t + D];
      v[t] = p + q;
      v[t + D] = p - q;
    }
}

template <int S>
__device__ __forceinline__ void lane_stage32(float* v, float c) {
  if constexpr (S < 2) {
#pragma unroll
    for (int i = 0; i < 32; i += 8) dpp_fmac8<S>(&v[i], c);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = xbutterfly<S>(v[i], c);
  }
}

// Rotates a lane's 32 values in place; returns the sign the DPP stages left on them.
template <int B>
__device__ __forceinline__ float rotate32(float* v, int lane) {
  constexpr int G = HalfSlice<B>::G;
  const int lo = lane % G;
  reg_stage32<1>(v);
  reg_stage32<2>(v);
  reg_stage32<4>(v);
  float sgn = 1.f;
  if constexpr (G >= 2) {
    const float c = (lo & 1) ? -1.f : 1.f;
    lane_stage32<0>(v, c);
    sgn *= c;
  }
  if constexpr (G >= 4) {
    const float c = (lo & 2) ? -1.f : 1.f;
    lane_stage32<1>(v, c);
    sgn *= c;
  }
  if constexpr (G >= 8) lane_stage32<2>(v, (lo & 4) ? -1.f : 1.f);
  if constexpr (G >= 16) lane_stage32<3>(v, (lo & 8) ? -1.f : 1.f);
  if constexpr (G >= 32) lane_stage32<4>(v, (lo & 16) ? -1.f : 1.f);
  reg_stage32<8>(v);
  reg_stage32<16>(v);
  return sgn;
}

// LDS byte of value i of the shifted part: 32 bytes of padding after every 256 spread the lanes'
// chunks, a block apart, over the banks.
__device__ __forceinline__ int shift_off(int i) { return i * 4 + (i >> 6) * 32; }
inline int shift_bytes(int64_t len) { return (int)(len * 4 + (len + 63) / 64 * 32); }

template <int B, int QT, bool SHIFT>
__global__ __launch_bounds__(1024) void glu_rows_kernel(GluRowsArgs a) {
  using S = HalfSlice<B>;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_stage[];
  __shared__ float s_max[16];
  const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (a.zero) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < a.nzero; i += stride)
      a.zero[i] = 0u;
  }
  const int64_t row = blockIdx.x;
  const int n = (int)a.n, col0 = w * kHalf;
  // the first part's length (whole blocks of the gate) and the second's
  const int len0 = SHIFT ? n - n % B : n, len1 = SHIFT ? (int)a.nq - len0 : n;
  bool in[2];  // whole blocks, so whole lanes
  in[0] = col0 + S::off(lane, 0) < len0;
  in[1] = col0 + S::off(lane, 0) < len1;

  // ---- dz ---------------------------------------------------------------------------------
  FqArgs zf{};
  zf.z = a.z;
  zf.zw = a.zw;
  zf.zk = a.zk;
  uint4 d[4];
  ZChunk g[4], u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = col0 + S::off(lane, j), col = at < n ? at : 0;
    d[j] = *reinterpret_cast<const uint4*>(a.dy + row * n + col);
    g[j].load<B >= 128>(zf, 2 * row, n, col);
    u[j].load<B >= 128>(zf, 2 * row + 1, n, col);
  }
  if (B >= 128 && a.zk != kKeptPlain) {
    // a quad's lanes are one group in every chunk: each reads one chunk's two powers
    const int at = col0 + S::off(lane & ~3, lane & 3), groups = (n + kGroup - 1) / kGroup;
    const uint8_t* p = a.zw + 2 * row * groups + (at < n ? at : 0) / kGroup;
    const uint32_t pg = p[0], pu = p[groups];
    g[0].w.z = quad_lane<0>(pg);
    g[1].w.z = quad_lane<1>(pg);
    g[2].w.z = quad_lane<2>(pg);
    g[3].w.z = quad_lane<3>(pg);
    u[0].w.z = quad_lane<0>(pu);
    u[1].w.z = quad_lane<1>(pu);
    u[2].w.z = quad_lane<2>(pu);
    u[3].w.z = quad_lane<3>(pu);
  }
  float v[2][32];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float dv[8], gv[8], uv[8];
    unpack_bf16x8(d[j], dv);
    g[j].get(a.zk, gv);
    u[j].get(a.zk, uv);
    gated_grad<8>(a.act, dv, gv, uv, &v[0][j * 8], &v[1][j * 8]);
    const int col = col0 + S::off(lane, j);
    if (col < n) {
      float* o = a.dz + row * 2 * n + col;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float* p = o + (int64_t)h * n;
        const float* s = &v[h][j * 8];
        reinterpret_cast<float4*>(p)[0] = make_float4(s[0], s[1], s[2], s[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(s[4], s[5], s[6], s[7]);
      }
    }
    if constexpr (SHIFT) {
      // value i of the second part is position len0 + i of the row
      const int up = n - len0 + col;
      if (col < n) put8(s_stage + shift_off(up), &v[1][j * 8]);
      if (col >= len0 && col < n) put8(s_stage + shift_off(col - len0), &v[0][j * 8]);
      if (col >= n && up < len1) {
        const float zero[8] = {};
        put8(s_stage + shift_off(up), zero);
      }
    }
  }
  if constexpr (SHIFT) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = in[1] ? col0 + S::off(lane, j) : 0;
      load8<float>(reinterpret_cast<const float*>(s_stage + shift_off(i)), &v[1][j * 8]);
    }
  }

  // ---- rotation, absmax ---------------------------------------------------------------------
  if (a.signs) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        apply_signs8(&v[h][j * 8], a.signs, in[h] ? h * len0 + col0 + S::off(lane, j) : 0);
  }
  float sgn = 1.f, mx = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sgn = rotate32<B>(v[h], lane);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      top = __builtin_fmaxf(__builtin_fmaxf(top, fabsf(v[h][i])), fabsf(v[h][i + 1]));
    mx = in[h] ? __builtin_fmaxf(mx, top) : mx;
  }
  mx = wave_max(mx);
  if (nw > 1) {
    if (lane == 0) s_max[w] = mx;
    __syncthreads();
    mx = 0.f;
    for (int i = 0; i < nw; ++i) mx = __builtin_fmaxf(mx, s_max[i]);
  }
  if (w == 0 && lane == 0) a.scale[row] = mx / a.denom;

  // ---- codes, through the wave's LDS area so that they leave in whole lines ---------------------
  // (where the shifted part was: every wave has read it, the maxima's barrier lies between)
  float pre;
  const float mul = code_mul(a.qmax, mx, &pre) * sgn;
  uint8_t* st = s_stage + w * 2 * kHalfStage;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (pre != 1.f) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[h][i] *= pre;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint2*>(st + h * kHalfStage + stage_off(S::off(lane, j))) =
          encode8<QT>(&v[h][j * 8], mul);
  }
  // the wave's LDS accesses complete in order: the reads see every lane's writes
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int rest = (h ? len1 : len0) - col0;
    uint8_t* q = a.q + row * a.nq + h * len0 + col0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int b = i * 1024 + lane * 16;
      if (b < rest)
        *reinterpret_cast<uint4*>(q + b) =
            *reinterpret_cast<const uint4*>(st + h * kHalfStage + stage_off(b));
    }
  }
}

template <int B, int QT, bool SHIFT>
hipError_t run_form(const GluRowsArgs& a, hipStream_t st) {
  const int64_t len1 = SHIFT ? a.nq - (a.n - a.n % B) : a.n;  // the longer part
  const int nw = (int)((len1 + kHalf - 1) / kHalf);
  int lds = nw * 2 * kHalfStage;
  if (SHIFT && shift_bytes(len1) > lds) lds = shift_bytes(len1);
  if (lds > 65536) {
    const hipError_t e =
        allow_dynamic_lds<&glu_rows_kernel<B, QT, SHIFT>>(shift_bytes(16 * kHalf));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((glu_rows_kernel<B, QT, SHIFT>), dim3((unsigned)a.rows), dim3(64 * nw), lds, st,
                     a);
  return hipGetLastError();
}

template <int B, int QT>
hipError_t run(const GluRowsArgs& a, hipStream_t st) {
  return a.n % B != 0 ? run_form<B, QT, true>(a, st) : run_form<B, QT, false>(a, st);
}

template <int QT>
hipError_t run_block(const GluRowsArgs& a, hipStream_t st) {
  switch (a.block) {
    case 64: return run<64, QT>(a, st);
    case 128: return run<128, QT>(a, st);
    case 256: return run<256, QT>(a, st);
    case 512: return run<512, QT>(a, st);
    case 1024: return run<1024, QT>(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool glu_rows_ok(int64_t n, int block) {
  // the second part, with a block's rest and the padding, fits 16 waves
  return fq_act_block_ok(block) && n > 0 && n % 8 == 0 && n + 2 * block <= 16 * kHalf;
}

hipError_t launch_glu_rows(const GluRowsArgs& a, int qt, hipStream_t st) {
  switch (qt) {
    case 0: return run_block<0>(a, st);
    case 1: return run_block<1>(a, st);
    case 2: return run_block<2>(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace halo
