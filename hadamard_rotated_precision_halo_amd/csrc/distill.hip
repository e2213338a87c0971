// distill.hip -- distillation from a teacher's top logits: loss and gradient per token (gfx950).
//
// For a token with student logits s[V] and the teacher's K kept logits t_k at vocabulary indices
// i_k (an index outside [0, V) is no entry), temperature tau:
//   p = softmax(t / tau) over the kept entries,  q = softmax(s / tau) over the vocabulary,
//   loss = tau^2 sum_k p_k (log p_k - log q[i_k]),
//   dlogits[j] = dloss tau (q_j - sum_k p_k [i_k = j]).
// A token without a kept entry, or whose logits are all -inf, has loss 0 and gradient 0; so has,
// for its gradient, a token with dloss 0.  A kept entry with p_k = 0 adds nothing.
//
// Bound by memory: the logits are read once and the gradient written once.  A workgroup holds a
// token's row in registers in its stored form (CH 16-byte chunks per lane) between the softmax
// statistics and the gradient; rows longer than a workgroup holds are read again, which their
// size makes a cache read for all but the first bytes.  Statistics, exponents and sums are fp32;
// every thread keeps the sum of its own chunks and the threads are added in a fixed order.
// The gradient is written for the whole row as dloss tau q; then the K entries, computed apart
// from their own logits, are written over it (duplicated indices sum their p first, so every
// writer of a position writes the same value).
#include "halo_kernels.h"
#include "rowops.h"

namespace halo {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// exp(s / tau - lse).  fp32 logits: s / tau - lse is rounded once (an fma) before it is scaled to
// base 2, so the error does not grow with |s|; bf16 logits' gradients keep 8 bits, and one fma
// with both factors merged is enough.
template <typename T>
struct Exponent {
  float mul, sub;  // fp32: 1 / tau, lse; bf16: log2(e) / tau, log2(e) lse
  __device__ __forceinline__ Exponent(float inv_tau, float lse) {
    if constexpr (sizeof(T) == 4) {
      mul = inv_tau;
      sub = lse;
    } else {
      mul = inv_tau * kLog2e;
      sub = lse * kLog2e;
    }
  }
  __device__ __forceinline__ float operator()(float s) const {
    const float d = __builtin_fmaf(s, mul, -sub);
    return exp2_fast(sizeof(T) == 4 ? d * kLog2e : d);
  }
};

// Sum and maximum over a workgroup of NW waves; s: NW floats, not in use by an earlier call.
template <int NW>
__device__ __forceinline__ float wg_sum(float v, float* s) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i) v += s[i];
  return v;
}
template <int NW>
__device__ __forceinline__ float wg_max(float v, float* s) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) v = fmaxf(v, s[i]);
  return v;
}

// HELD: the row is in registers (vocab <= NT CH VEC); else it is read twice.
template <typename T, int NT, int CH, bool HELD>
__global__ __launch_bounds__(NT) void distill_kernel(DistillArgs a) {
  constexpr int VEC = RowType<T>::VEC, NW = NT / 64;
  __shared__ float s_max[NW], s_sum[NW], s_tmax[NW], s_tsum[NW], s_loss[NW];
  extern __shared__ float s_top[];  // p[K], logit[K] (fp32), then index[K]
  const int tid = threadIdx.x;
  const int64_t tok = blockIdx.x;
  const int V = a.vocab, K = a.top;
  const T* row = reinterpret_cast<const T*>(a.logits) + tok * a.ldl;
  T* out = reinterpret_cast<T*>(a.dlogits) + tok * a.ldd;
  float* s_p = s_top;
  float* s_z = s_top + K;
  int* s_i = reinterpret_cast<int*>(s_top + 2 * K);
  const int whole = V / VEC;  // full chunks; the V % VEC elements after them go one per thread
  const int rest0 = whole * VEC;
  const float dl = a.dloss ? a.dloss[tok] : 0.f;
  const bool grad = a.dlogits != nullptr;

  if (a.lse_in && dl == 0.f) {  // gradient alone, of a token that takes no part
    const float z[VEC] = {};
    for (int c = tid; c < whole; c += NT) store16u(out + c * VEC, pack16<T>(z));
    if (rest0 + tid < V) elem_store<T>(out + rest0 + tid, 0.f);
    return;
  }

  uint4 raw[HELD ? CH : 1];
  float rest = -__builtin_inff();
  if constexpr (HELD) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = j * NT + tid;
      raw[j] = load16u(row + (c < whole ? c : 0) * VEC);
    }
  }
  if (rest0 + tid < V) rest = elem_f32<T>(row + rest0 + tid);

  // the teacher's entries
  float tm = -__builtin_inff();
  for (int k = tid; k < K; k += NT) {
    const int i = a.idx[tok * a.ldi + k];
    const bool in = i >= 0 && i < V;
    float t = a.t_bf16 ? elem_f32(reinterpret_cast<const uint16_t*>(a.tlogits) + tok * a.ldt + k)
                       : reinterpret_cast<const float*>(a.tlogits)[tok * a.ldt + k];
    t = in ? t * a.inv_tau : -__builtin_inff();
    s_i[k] = in ? i : -1;
    s_p[k] = t;
    s_z[k] = in ? elem_f32<T>(row + i) : 0.f;
    tm = fmaxf(tm, t != t ? __builtin_inff() : t);  // a NaN entry keeps the token in, as NaN
  }
  tm = wg_max<NW>(tm, s_tmax);
  const bool some = tm != -__builtin_inff();
  float ts = 0.f;
  for (int k = tid; k < K; k += NT) ts += some ? exp2_fast((s_p[k] - tm) * kLog2e) : 0.f;
  ts = wg_sum<NW>(ts, s_tsum);

  // statistics of the row
  float lse;
  if (a.lse_in) {
    lse = a.lse_in[tok];
  } else {
    float m = rest;
    if constexpr (HELD) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        float v[VEC];
        unpack16<T>(raw[j], v);
        if (j * NT + tid < whole) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) m = fmaxf(m, v[e]);
        }
      }
    } else {
      for (int c = tid; c < whole; c += NT) {
        float v[VEC];
        unpack16<T>(load16u(row + c * VEC), v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) m = fmaxf(m, v[e]);
      }
    }
    m = wg_max<NW>(m, s_max) * a.inv_tau;
    if (m == -__builtin_inff()) m = 0.f;  // all -inf (sum 0), or all NaN (sum NaN)
    const Exponent<T> ex(a.inv_tau, m);
    float sum = rest0 + tid < V ? ex(rest) : 0.f;
    if constexpr (HELD) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        float v[VEC];
        unpack16<T>(raw[j], v);
        if (j * NT + tid < whole) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) sum += ex(v[e]);
        }
      }
    } else {
      for (int c = tid; c < whole; c += NT) {
        float v[VEC];
        unpack16<T>(load16u(row + c * VEC), v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum += ex(v[e]);
      }
    }
    sum = wg_sum<NW>(sum, s_sum);
    lse = sum == 0.f ? -__builtin_inff() : m + logf(sum);
    if (a.lse && tid == 0) a.lse[tok] = lse;
  }
  const bool empty = !some || lse == -__builtin_inff();

  // the loss, and each entry's p
  float l = 0.f;
  const float logts = logf(ts);
  for (int k = tid; k < K; k += NT) {
    const float lp = (s_p[k] - tm) - logts;
    const float p = empty ? 0.f : exp2_fast(lp * kLog2e);
    s_p[k] = p;
    if (p != 0.f) l += p * (lp - (__builtin_fmaf(s_z[k], a.inv_tau, -lse)));
  }
  if (a.loss) {
    l = wg_sum<NW>(l, s_loss);
    if (tid == 0) a.loss[tok] = l * a.tau * a.tau;
  }
  if (!grad) return;
  const float by = empty ? 0.f : dl * a.tau;
  const bool zero = by == 0.f;
  const Exponent<T> ex(a.inv_tau, zero ? 0.f : lse);
  if constexpr (HELD) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = j * NT + tid;
      float v[VEC];
      unpack16<T>(raw[j], v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = zero ? 0.f : by * ex(v[e]);
      if (c < whole) store16u(out + c * VEC, pack16<T>(v));
    }
  } else {
    for (int c = tid; c < whole; c += NT) {
      float v[VEC];
      unpack16<T>(load16u(row + c * VEC), v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = zero ? 0.f : by * ex(v[e]);
      store16u(out + c * VEC, pack16<T>(v));
    }
  }
  if (rest0 + tid < V) elem_store<T>(out + rest0 + tid, zero ? 0.f : by * ex(rest));
  if (zero) return;
  // the entries, over the row (the barrier orders the two stores of a position)
  __syncthreads();
  for (int k = tid; k < K; k += NT) {
    const int i = s_i[k];
    if (i < 0) continue;
    float p = 0.f;
    for (int o = 0; o < K; ++o) p += s_i[o] == i ? s_p[o] : 0.f;
    elem_store<T>(out + i, by * (ex(s_z[k]) - p));
  }
}

template <typename T, int NT, int CH, bool HELD>
hipError_t run(const DistillArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((distill_kernel<T, NT, CH, HELD>), dim3((unsigned)a.tokens), dim3(NT),
                     (size_t)a.top * 12, st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t pick(const DistillArgs& a, hipStream_t st) {
  const int64_t chunks = a.vocab / RowType<T>::VEC;
  if (chunks <= 256 * 4) return run<T, 256, 4, true>(a, st);
  if (chunks <= 512 * 8) return run<T, 512, 8, true>(a, st);
  if (chunks <= 1024 * 8) return run<T, 1024, 8, true>(a, st);
  if (chunks <= 1024 * 16) return run<T, 1024, 16, true>(a, st);
  return run<T, 1024, 1, false>(a, st);
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, int in_bf16, hipStream_t st) {
  return in_bf16 ? pick<uint16_t>(a, st) : pick<float>(a, st);
}

}  // namespace halo
