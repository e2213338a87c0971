// glu_rows.hip -- the rows pass of the gated layer's gradient on gfx950: dz = [dy u act'(g), dy act(g)]
// in fp32 from dy and z's halves g and u, stored for the columns pass, and rotated and quantised along
// its 2 n columns as the rows kernel of fwht_wave.h does it (natural-order butterflies over blocks of B
// contiguous indices, one absmax scale per row).
//
// A workgroup owns a row.  A lane holds CH chunks of 8 columns of the gate's half and the same of the up
// half, so that dy, g and u are read once and the activation is evaluated once for both.  The pass moves
// 360 MB in 66 us at 4096 x 2 x 5504 bf16 (5.4 TB/s); forming dz in the columns pass again in place of the
// store moved less and took longer (each half evaluates the activation for itself there: 222 against 165 us
// of all columns).  Chunk j of lane lo of a block's G = B / (8 CH) lanes sits at block offset
// (j G + lo) 8, so the 3 low and the top index bits are butterflied in registers and log2(G) stages cross
// lanes, in increasing bit order and with the operand order of a sequential fp32 butterfly.
//
// Where the block does not divide n, a block spans both halves and the up half's blocks start at other
// columns than the gate's: what lies behind the gate's whole blocks (its last columns, the up half, the
// zero padding) then passes through LDS to the lanes that hold its blocks (SHIFT).
#include "fwht_wave.h"

namespace halo {

namespace {

constexpr int kMaxColumns = 16 * 2048;  // of a half: 16 waves of the widest slices

// CH: as few chunks a lane as 16 waves hold of a row, so that a row's waves are many and short (4096 x 2
// x 5504, k 512: 234 us a call with one, 239 with two, 244 with four; 1000 x 2 x 1048: 41.1, 41.6, 42.9).
template <int B, int CH>
struct HalfSlice {
  static constexpr int G = B / (8 * CH);  // lanes per block
  static constexpr int N = 8 * CH;        // values of a half per lane
  static constexpr int kHalf = 64 * N;    // columns of a half per wave
  static constexpr int kStage = kHalf + kHalf / 256 * 32;  // its codes in LDS (stage_off)
  __device__ static __forceinline__ int off(int lane, int j) {
    return (lane / G) * B + (j * G + lane % G) * 8;
  }
};

__device__ __forceinline__ void put8(uint8_t* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <int D, int N>
__device__ __forceinline__ void reg_stage_n(float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 2 * D)
#pragma unroll
    for (int t = i; t < i + D; ++t) {
      const float p = v[t], q = v[t + D];
      v[t] = p + q;
      v[t + D] = p - q;
    }
}

template <int S, int N>
__device__ __forceinline__ void lane_stage_n(float* v, float c) {
  if constexpr (S < 2) {
#pragma unroll
    for (int i = 0; i < N; i += 8) dpp_fmac8<S>(&v[i], c);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = xbutterfly<S>(v[i], c);
  }
}

// Rotates a lane's values of a half in place; returns the sign the DPP stages left on them.
template <int B, int CH>
__device__ __forceinline__ float rotate_half(float* v, int lane) {
  constexpr int G = HalfSlice<B, CH>::G, N = HalfSlice<B, CH>::N;
  static_assert(G <= 64, "a block within a wave");
  const int lo = lane % G;
  reg_stage_n<1, N>(v);
  reg_stage_n<2, N>(v);
  reg_stage_n<4, N>(v);
  float sgn = 1.f;
  if constexpr (G >= 2) {
    const float c = (lo & 1) ? -1.f : 1.f;
    lane_stage_n<0, N>(v, c);
    sgn *= c;
  }
  if constexpr (G >= 4) {
    const float c = (lo & 2) ? -1.f : 1.f;
    lane_stage_n<1, N>(v, c);
    sgn *= c;
  }
  if constexpr (G >= 8) lane_stage_n<2, N>(v, (lo & 4) ? -1.f : 1.f);
  if constexpr (G >= 16) lane_stage_n<3, N>(v, (lo & 8) ? -1.f : 1.f);
  if constexpr (G >= 32) lane_stage_n<4, N>(v, (lo & 16) ? -1.f : 1.f);
  if constexpr (G >= 64) lane_stage_n<5, N>(v, (lo & 32) ? -1.f : 1.f);
  if constexpr (CH >= 2) reg_stage_n<8, N>(v);
  if constexpr (CH >= 4) reg_stage_n<16, N>(v);
  return sgn;
}

// LDS byte of value i of the shifted part: 32 bytes of padding after every 256 spread the lanes'
// chunks, a block apart, over the banks.
__device__ __forceinline__ int shift_off(int i) { return i * 4 + (i >> 6) * 32; }
inline int shift_bytes(int64_t len) { return (int)(len * 4 + (len + 63) / 64 * 32); }

template <int B, int QT, bool SHIFT, int CH>
__global__ __launch_bounds__(1024) void glu_rows_kernel(GluRowsArgs a) {
  using S = HalfSlice<B, CH>;
  constexpr int N = S::N;
  constexpr bool kShare = B >= 128 && CH == 4;  // a quad's lanes are one group of z in every chunk
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
  const int n = (int)a.n, col0 = w * S::kHalf;
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
  uint4 d[CH];
  ZChunk g[CH], u[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int at = col0 + S::off(lane, j), col = at < n ? at : 0;
    d[j] = *reinterpret_cast<const uint4*>(a.dy + row * n + col);
    g[j].template load<kShare>(zf, 2 * row, n, col);
    u[j].template load<kShare>(zf, 2 * row + 1, n, col);
  }
  if constexpr (kShare) {
    if (a.zk != kKeptPlain) {  // each lane reads one chunk's two powers
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
  }
  float v[2][N];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    float dv[8], gv[8], uv[8];
    unpack_bf16x8(d[j], dv);
    g[j].get(a.zk, gv);
    u[j].get(a.zk, uv);
    gated_grad<8, false>(a.act, dv, gv, uv, &v[0][j * 8], &v[1][j * 8]);
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
    for (int j = 0; j < CH; ++j) {
      const int i = in[1] ? col0 + S::off(lane, j) : 0;
      load8<float>(reinterpret_cast<const float*>(s_stage + shift_off(i)), &v[1][j * 8]);
    }
  }

  // ---- rotation, absmax ---------------------------------------------------------------------
  if (a.signs) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < CH; ++j)
        apply_signs8(&v[h][j * 8], a.signs, in[h] ? h * len0 + col0 + S::off(lane, j) : 0);
  }
  float sgn = 1.f, mx = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sgn = rotate_half<B, CH>(v[h], lane);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2)
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
  uint8_t* st = s_stage + w * 2 * S::kStage;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (pre != 1.f) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[h][i] *= pre;
    }
#pragma unroll
    for (int j = 0; j < CH; ++j)
      *reinterpret_cast<uint2*>(st + h * S::kStage + stage_off(S::off(lane, j))) =
          encode8<QT>(&v[h][j * 8], mul);
  }
  // the wave's LDS accesses complete in order: the reads see every lane's writes
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int rest = (h ? len1 : len0) - col0;
    uint8_t* q = a.q + row * a.nq + h * len0 + col0;
#pragma unroll
    for (int i = 0; i < (S::kHalf + 1023) / 1024; ++i) {
      const int b = i * 1024 + lane * 16;
      if (b < rest && b < S::kHalf)
        *reinterpret_cast<uint4*>(q + b) =
            *reinterpret_cast<const uint4*>(st + h * S::kStage + stage_off(b));
    }
  }
}

template <int B, int QT, bool SHIFT, int CH>
hipError_t run_form(const GluRowsArgs& a, hipStream_t st) {
  using S = HalfSlice<B, CH>;
  const int64_t len1 = SHIFT ? a.nq - (a.n - a.n % B) : a.n;  // the longer part
  const int nw = (int)((len1 + S::kHalf - 1) / S::kHalf);
  int lds = nw * 2 * S::kStage;
  if (SHIFT && shift_bytes(len1) > lds) lds = shift_bytes(len1);
  if (lds > 65536) {
    const hipError_t e =
        allow_dynamic_lds<&glu_rows_kernel<B, QT, SHIFT, CH>>(shift_bytes(kMaxColumns));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((glu_rows_kernel<B, QT, SHIFT, CH>), dim3((unsigned)a.rows), dim3(64 * nw), lds,
                     st, a);
  return hipGetLastError();
}

template <int B, int QT, int CH>
hipError_t run_shift(const GluRowsArgs& a, hipStream_t st) {
  return a.n % B != 0 ? run_form<B, QT, true, CH>(a, st) : run_form<B, QT, false, CH>(a, st);
}

template <int B, int QT>
hipError_t run(const GluRowsArgs& a, hipStream_t st) {
  // the second part of a row, with a block's rest and the padding, fits 16 waves; a block fits a wave
  if constexpr (B <= 512)
    if (a.n + 2 * B <= kMaxColumns / 4) return run_shift<B, QT, 1>(a, st);
  if (a.n + 2 * B <= kMaxColumns / 2) return run_shift<B, QT, 2>(a, st);
  return run_shift<B, QT, 4>(a, st);
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
  return fq_act_block_ok(block) && n > 0 && n % 8 == 0 && n + 2 * block <= kMaxColumns;
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
