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
// Bound by memory: the logits are read once and the gradient written once, past the caches.
//   Held      loss and gradient of a row that fits a workgroup's registers in its stored form (CH
//             16-byte chunks per lane): between the softmax statistics and the gradient it is not
//             read again.
//   Streamed  the loss alone (a running maximum and sum per lane, few registers, many rows in
//             flight), and loss and gradient of longer rows, which read them twice.
//   Parts     the gradient alone under a given lse: no statistics, so a row is split over
//             workgroups.
// Every lane keeps a running (maximum, sum) over groups of 4 chunks of its part of the row, and the
// first 256 threads (or all) one of the teacher's entries; waves combine theirs in a fixed order
// after one barrier.  The order depends on the vocabulary alone (its thread count), so the three
// calls give the same bits (the gradient: up to |lse| = kFar) and a token's values do not depend on
// the others in its batch.
// Statistics, exponents and sums are fp32.  The statistics are of differences from a maximum taken
// before they are scaled by 1 / tau: with s log2(e) / tau and the maximum's product rounded apart, a
// part of the row that a mask fills with -1e10 or the type's lowest value would be off from its own
// maximum by more than an exponential holds.  The gradient is written for the whole row as dloss tau
// q; after a second barrier the entries, computed apart from their own logits, are written over it
// (duplicated indices sum their p first, so every writer of a position writes the same value).
#include "halo_kernels.h"
#include "rowops.h"

namespace halo {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// exp(s / tau - lse).  fp32 logits: s / tau - lse is rounded once (an fma) before it is scaled to
// base 2, so the error does not grow with |s|; bf16 logits' gradients keep 8 bits, and one fma
// with both factors merged is enough.  For |lse| up to kFar: see FarExponent.
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

// The same where lse is so large that its own last bit (2^-12 at kFar) shows in the exponential:
// exp2((s - ref) mul - sub), from the row's maximum ref and sub = log2 of its sum where the call has
// them, else from ref = lse tau and no more than 1, which q is.  NaN stays.
constexpr float kFar = 4096.f;
struct FarExponent {
  float ref, mul, sub;
  __device__ __forceinline__ float operator()(float s) const {
    const float d = __builtin_fmaf(s - ref, mul, -sub);
    return exp2_fast(d > 0.f ? 0.f : d);
  }
};

__device__ __forceinline__ float finite_ref(float m) { return m == -__builtin_inff() ? 0.f : m; }

// A (maximum, sum of exp2((. - maximum) mul)) pair over the lanes of a wave, mul = log2(e) / tau.  A
// part that is -inf everywhere has maximum -inf and sum 0; NaN stays in the sum.
__device__ __forceinline__ void wave_pair(float& m, float& s, float mul) {
  const float top = wave_max(m);
  s = wave_sum(s * exp2_fast((m - finite_ref(top)) * mul));
  m = top;
}
// The same over the pairs of NW waves.
template <int NW>
__device__ __forceinline__ void pair_of(const float (*p)[2], float mul, float& m, float& s) {
  m = p[0][0];
#pragma unroll
  for (int i = 1; i < NW; ++i) m = fmaxf(m, p[i][0]);
  const float ref = finite_ref(m);
  s = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i) s += p[i][1] * exp2_fast((p[i][0] - ref) * mul);
}

// Which of a token's entries share their index with another.  Up to kSearch entries: each one's p is
// summed over all of them.  With more, the indices go into an open table in the LDS of at least
// two slots per entry (so a free one ends every walk) whose top bit marks an index that came twice,
// and only marked ones are summed over: the same terms in the same order, as p + 0 = p.  A table
// costs two short walks and its clearing for each entry.  2048 x
// 32000 bf16, loss and gradient: 62.5 us for 68.1 us at 256 entries, 123 for 213 us at 1024; 8192 x
// 2000 at 128 entries 27.0 for 33.4 us; at 32 entries (no table) 20.1 for 21.4 us, at 64 equal.
constexpr int kSearch = 64;
__host__ __device__ constexpr int entry_slots(int top) {
  int n = 4 * kSearch;
  while (n < 2 * top) n *= 2;
  return top <= kSearch ? 0 : n;
}
__device__ __forceinline__ int first_slot(int i, int slots) {  // multiplicative hash, top bits
  return (int)(((uint32_t)i * 2654435769u) >> (__clz(slots) + 1));
}
__device__ __forceinline__ void enter(int* key, int slots, int i) {
  for (int at = first_slot(i, slots);; at = (at + 1) & (slots - 1)) {
    const int was = atomicCAS(key + at, -1, i);
    if (was == -1) return;
    if ((was & 0x7fffffff) == i) {
      atomicOr(key + at, (int)0x80000000u);
      return;
    }
  }
}
__device__ __forceinline__ bool entered_twice(const int* key, int slots, int i) {
  int at = first_slot(i, slots);
  while ((key[at] & 0x7fffffff) != i) at = (at + 1) & (slots - 1);
  return key[at] < 0;
}

enum Mode { kHeld, kStreamed, kParts };

// One token's row (kParts: the part blockIdx.y of it).
template <typename T, int NT, int CH, int MODE>
__global__
__launch_bounds__(NT, NT >= 512 && CH <= 4 ? 8 : NT == 512 && CH == 8 ? 6 : 4)
void distill_kernel(DistillArgs a) {
  constexpr int VEC = RowType<T>::VEC, NW = NT / 64;
  __shared__ float s_row[NW][2], s_tea[4][2], s_loss[NW];
  // t, then p [K]; logit [K]; index [K]; with many entries, a table of indices [slots]
  extern __shared__ __attribute__((aligned(16))) float s_top[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t tok = a.first + blockIdx.x;
  const int K = a.top;
  const float mul = a.inv_tau * kLog2e;
  const T* row = reinterpret_cast<const T*>(a.logits) + tok * a.ldl;
  T* out = reinterpret_cast<T*>(a.dlogits) + tok * a.ldd;
  const int Kp = (K + 3) & ~3;  // the entries are also read 4 at a time
  float* s_p = s_top;
  float* s_z = s_top + Kp;
  int* s_i = reinterpret_cast<int*>(s_top + 2 * Kp);
  int* s_key = s_i + Kp;
  const int slots = entry_slots(K);
  // This workgroup's elements [lo, hi): full chunks from base on, then fewer than VEC more, one per
  // thread.  A part's chunks start on 64 bytes (777 x 50257 fp32: 212 MB fetched for 156 MB of rows
  // where they start anywhere); the elements before the first part's also go one per thread.
  constexpr int SPAN = NT * CH * VEC;
  const int part = MODE == kParts ? (int)blockIdx.y : 0;
  const int to_line = (int)((-reinterpret_cast<uintptr_t>(row) & 63) / sizeof(T));
  const int head = MODE == kParts ? min(a.vocab, to_line) : 0;
  const int base = head + part * SPAN;
  const int n = MODE == kParts ? max(0, min(a.vocab - base, SPAN)) : a.vocab;
  const int lo = part == 0 ? 0 : base, hi = base + n;
  const int whole = n / VEC, tail = n - whole * VEC;
  const int lone = tid < tail ? base + whole * VEC + tid
                   : part == 0 && tid - tail < head ? tid - tail : -1;
  const T* in = row + base;
  const bool grad = a.dlogits != nullptr;
  const float dl = a.dloss ? a.dloss[tok] : 0.f;

  if (MODE == kParts && dl == 0.f) {  // a token that takes no part
    const float z[VEC] = {};
    for (int c = tid; c < whole; c += NT) store16u_nt(out + base + c * VEC, pack16<T>(z));
    if (lone >= 0) elem_store<T>(out + lone, 0.f);
    return;
  }

  // the teacher's first entries are asked for before the row, so that the loads of their logits
  // need not wait for it
  constexpr int TT = NT < 256 ? NT : 256;  // threads that reduce the teacher's entries
  const int32_t* idx = a.idx + tok * a.ldi;
  auto teacher = [&](int k) {
    return a.t_bf16 ? elem_f32(reinterpret_cast<const uint16_t*>(a.tlogits) + tok * a.ldt + k)
                    : reinterpret_cast<const float*>(a.tlogits)[tok * a.ldt + k];
  };
  const bool mine = tid < TT && tid < K;
  const int i0 = mine ? idx[tid] : -1;
  const float t0 = mine ? teacher(tid) : 0.f;

  uint4 raw[MODE == kStreamed ? 1 : CH];
  if constexpr (MODE != kStreamed) {
    if (whole > 0) {  // chunks past the row read its first one
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = j * NT + tid;
        raw[j] = load16u_nt(in + (c < whole ? c : 0) * VEC);
      }
    } else {
#pragma unroll
      for (int j = 0; j < CH; ++j) raw[j] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  const float rest = lone >= 0 ? elem_f32<T>(row + lone) : -__builtin_inff();

  // the teacher's entries: kept in LDS, and their (maximum, sum)
  if (tid < TT) {
    float tm = -__builtin_inff();
    auto keep = [&](int k, int i, float t, float z) __attribute__((always_inline)) {
      const bool there = i >= 0 && i < a.vocab;
      t = there ? t : -__builtin_inff();
      s_i[k] = there ? i : -1;
      s_z[k] = there ? z : 0.f;
      s_p[k] = t;
      tm = fmaxf(tm, t != t ? __builtin_inff() : t);  // a NaN entry keeps the token in, as NaN
    };
    // a part takes the logits of its own entries, the others' of the row's first element
    const int from = MODE == kParts ? lo : 0, to = MODE == kParts ? hi : a.vocab;
    auto logit = [&](int i) { return elem_f32<T>(row + (i >= from && i < to ? i : 0)); };
    if (mine) keep(tid, i0, t0, logit(i0));
    // DEEP entries in flight.  4 where many fall on a thread (8192 x 2000 bf16 with 512 entries:
    // 53 us, 68 us with 1) and for parts; 1 beside a longer row in registers (4096 x 131072 with 64
    // entries: 398 us, 418 us with 4).
    constexpr int DEEP = NT <= 64 || MODE == kParts ? 4 : 1;
    for (int k0 = tid + TT; k0 < K; k0 += DEEP * TT) {
      int i[DEEP];
      float t[DEEP], z[DEEP];
#pragma unroll
      for (int j = 0; j < DEEP; ++j) {
        const int k = min(k0 + j * TT, K - 1);
        i[j] = idx[k];
        t[j] = teacher(k);
      }
#pragma unroll
      for (int j = 0; j < DEEP; ++j) z[j] = logit(i[j]);
#pragma unroll
      for (int j = 0; j < DEEP; ++j)
        if (k0 + j * TT < K) keep(k0 + j * TT, i[j], t[j], z[j]);
    }
    if (tid < Kp - K) {
      s_i[K + tid] = -1;
      s_p[K + tid] = 0.f;
    }
    float ts = 0.f;
    const float ref = finite_ref(tm);
    for (int k = tid; k < K; k += TT) ts += exp2_fast((s_p[k] - ref) * mul);
    wave_pair(tm, ts, mul);
    if (lane == 0) {
      s_tea[wave][0] = tm;
      s_tea[wave][1] = ts;
    }
  }

  for (int k = tid; k < slots; k += NT) s_key[k] = -1;

  // the row's (maximum, sum)
  if constexpr (MODE != kParts) {
    float m = rest, sum = 0.f;
    if (lone >= 0) sum = exp2_fast((rest - finite_ref(m)) * mul);
    // chunks c0, c0 + NT, .. (4 of them): their maximum first, then the running sum moves to it
    auto group = [&](const uint4* w, int c0) __attribute__((always_inline)) {
      float top = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[VEC], t = -__builtin_inff();
        unpack16<T>(w[j], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) t = fmaxf(t, v[e]);
        if (c0 + j * NT < whole) top = fmaxf(top, t);
      }
      top = fmaxf(m, top);
      const float ref = finite_ref(top);
      sum *= exp2_fast((m - ref) * mul);
      m = top;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[VEC], part = 0.f;
        unpack16<T>(w[j], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) part += exp2_fast((v[e] - ref) * mul);
        sum += c0 + j * NT < whole ? part : 0.f;
      }
    };
    if constexpr (MODE == kHeld) {
#pragma unroll
      for (int j = 0; j < CH; j += 4) group(&raw[j], j * NT + tid);
      keep_raw(raw);
    } else {
      for (int c0 = tid; c0 < whole; c0 += NT * 4) {
        uint4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + j * NT;
          w[j] = load16u_nt(in + (c < whole ? c : c0) * VEC);
        }
        group(w, c0);
      }
    }
    wave_pair(m, sum, mul);
    if (lane == 0) {
      s_row[wave][0] = m;
      s_row[wave][1] = sum;
    }
  }
  __syncthreads();
  float tm, ts, lse, m = 0.f, logsum = 0.f;
  bool none;  // every logit is -inf; lse alone may also be below the range of fp32
  pair_of<TT / 64>(s_tea, mul, tm, ts);
  if (MODE == kParts) {
    lse = a.lse_in[tok];
    none = lse == -__builtin_inff();
  } else {
    float sum;
    pair_of<NW>(s_row, mul, m, sum);
    logsum = logf(sum);
    none = sum == 0.f;
    lse = none ? -__builtin_inff() : __builtin_fmaf(m, a.inv_tau, logsum);
    if (a.lse && tid == 0) a.lse[tok] = lse;
  }
  const bool empty = tm == -__builtin_inff() || none;

  // each entry's p, and the loss
  float l = 0.f;
  const float logts = logf(ts);
  for (int k = tid; k < K; k += NT) {
    const float lp = __builtin_fmaf(s_p[k] - tm, a.inv_tau, -logts);
    const float p = empty ? 0.f : exp2_fast(lp * kLog2e);
    s_p[k] = p;
    if (p != 0.f) l += p * (lp - __builtin_fmaf(s_z[k] - m, a.inv_tau, -logsum));
    const int i = s_i[k];
    if (slots && grad && i >= lo && i < hi) enter(s_key, slots, i);
  }
  if (MODE != kParts) {
    l = wave_sum(l);
    if (lane == 0) s_loss[wave] = l;
  }
  const float by = empty ? 0.f : dl * a.tau;
  const bool zero = by == 0.f;
  const bool far = !(fabsf(lse) <= kFar);
  const Exponent<T> ex(a.inv_tau, lse);
  FarExponent exf{m, mul, logsum * kLog2e};
  if (MODE == kParts) {
    exf.ref = fmaxf(lse * a.tau, -__FLT_MAX__);
    exf.sub = lse == lse ? 0.f : lse;
  }
  auto write = [&](auto ex) __attribute__((always_inline)) {
    T* o = out + base;
    if constexpr (MODE == kStreamed) {
      for (int c = tid; c < whole; c += NT) {
        float v[VEC];
        unpack16<T>(load16u(in + c * VEC), v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = zero ? 0.f : by * ex(v[e]);
        store16u_nt(o + c * VEC, pack16<T>(v));
      }
    } else {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = j * NT + tid;
        float v[VEC];
        unpack16<T>(raw[j], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = zero ? 0.f : by * ex(v[e]);
        if (c < whole) store16u_nt(o + c * VEC, pack16<T>(v));
      }
    }
    if (lone >= 0) elem_store<T>(out + lone, zero ? 0.f : by * ex(rest));
  };
  if (grad) {
    if (far) write(exf);
    else write(ex);
  }
  __syncthreads();  // the losses and the p are in LDS; the row's stores come before the entries'
  if (MODE != kParts && tid == 0) {
    l = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) l += s_loss[i];
    a.loss[tok] = l * a.tau * a.tau;
  }
  if (!grad || zero) return;
  for (int k = tid; k < K; k += NT) {
    const int i = s_i[k];
    if (i < lo || i >= hi) continue;
    const float q = far ? exf(s_z[k]) : ex(s_z[k]);
    if (slots && !entered_twice(s_key, slots, i)) {
      elem_store<T>(out + i, by * (q - s_p[k]));
      continue;
    }
    float p = 0.f;
    for (int o = 0; o < Kp; o += 4) {
      const int4 oi = *reinterpret_cast<const int4*>(s_i + o);
      const float4 op = *reinterpret_cast<const float4*>(s_p + o);
      p += oi.x == i ? op.x : 0.f;
      p += oi.y == i ? op.y : 0.f;
      p += oi.z == i ? op.z : 0.f;
      p += oi.w == i ? op.w : 0.f;
    }
    elem_store<T>(out + i, by * (q - p));
  }
}

template <typename T, int NT, int CH, int MODE>
hipError_t run(DistillArgs a, hipStream_t st) {
  constexpr int64_t part = (int64_t)NT * CH * RowType<T>::VEC;
  const int64_t most = max_workgroups(NT);
  for (a.first = 0; a.first < a.tokens; a.first += most) {
    const int64_t left = a.tokens - a.first;
    const dim3 grid((unsigned)(left < most ? left : most),
                    MODE == kParts ? (unsigned)((a.vocab + part - 1) / part) : 1u);
    hipLaunchKernelGGL((distill_kernel<T, NT, CH, MODE>), grid, dim3(NT),
                       (size_t)((a.top + 3) & ~3) * 12 + (size_t)entry_slots(a.top) * 4, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Threads per token, by the vocabulary alone: so few that a compute unit holds several rows, one of
// which loads while another is reduced or stored, and so many that a row fits their registers.
// 8192 x 2000 bf16, loss and gradient: 17.8 us with a wave per token, 33.0 us with 256 threads;
// 4096 x 16000: 58 us with 512 threads, 69 us with 1024; 2048 x 65536: 95 and 107 us.
template <typename T>
hipError_t pick(const DistillArgs& a, hipStream_t st) {
  const int64_t chunks = a.vocab / RowType<T>::VEC;
  if (chunks <= 64 * 4) {
    if (a.lse_in) return run<T, 64, 4, kParts>(a, st);
    return a.dlogits ? run<T, 64, 4, kHeld>(a, st) : run<T, 64, 4, kStreamed>(a, st);
  }
  if (a.lse_in) return run<T, 256, 8, kParts>(a, st);
  if (chunks <= 256 * 4)
    return a.dlogits ? run<T, 256, 4, kHeld>(a, st) : run<T, 256, 4, kStreamed>(a, st);
  if (chunks <= 512 * 16) {
    if (!a.dlogits) return run<T, 512, 4, kStreamed>(a, st);
    return chunks <= 512 * 8 ? run<T, 512, 8, kHeld>(a, st) : run<T, 512, 16, kHeld>(a, st);
  }
  if (!a.dlogits) return run<T, 1024, 4, kStreamed>(a, st);
  if (chunks <= 1024 * 16) return run<T, 1024, 16, kHeld>(a, st);
  return run<T, 1024, 4, kStreamed>(a, st);
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, int in_bf16, hipStream_t st) {
  return in_bf16 ? pick<uint16_t>(a, st) : pick<float>(a, st);
}

}  // namespace halo
