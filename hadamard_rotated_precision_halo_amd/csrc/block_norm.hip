// block_norm.hip -- the join between two blocks of a model, forward and backward (gfx950).
//
// Forward.  A block's output y joins the residual stream r and the next block's input is
// normalised (every mean over the D elements of a token's row):
//   a = 1 / sqrt(mean(y^2) + eps),     r' = r + scale gate (y a post_weight)
//   b = 1 / sqrt(mean(r'^2) + eps),    h  = r' b pre_weight
// r' stays in fp32 between the two norms; each output is rounded once.
//
// Backward, with rhat = r' b, yhat = y a, u = dh pre_weight, c = scale gate post_weight:
//   G  = dr' + b (u - rhat mean(u rhat))              (dr = G)
//   dy = a (c G - yhat mean(c G yhat))
//   dgate = sum scale G yhat post_weight,  dpost = sum scale gate G yhat,  dpre = sum dh rhat
// The second mean is linear in the first: mean(c G yhat) = mean(c yhat (dr' + b u)) -
// mean(u rhat) mean(c yhat b rhat), so one pass over the row and one joint reduction of three
// sums give both, and a row is read once.
//
// Mapping.  Both directions are bound by memory: a row (or several) is held in registers as
// 16-byte chunks by a team of NW waves, CH chunks per lane, read once and written once.  A row
// whose length the chunk does not divide ends in a chunk that is moved back to end at the row's
// last element; the elements it shares with the chunk before are computed twice (the same
// values) and counted once.
// The backward's parameter gradients are sums over tokens: a team keeps its columns' sums in
// registers over its rows, a workgroup folds its teams through the LDS and writes one partial
// row per sum, and a second launch adds the partial rows in a fixed order (no atomics: the
// results do not change between runs).
#include "halo_kernels.h"
#include "rowops.h"

namespace halo {

namespace {

// One chunk's place in a row of d elements: chunk c starts at element min(c VEC, d - VEC) and
// counts its elements from c VEC on (`from`: elements below are the chunk before's).
template <int VEC>
struct Place {
  int at, from;
  bool in;
};
template <int VEC, bool ODD>
__device__ __forceinline__ Place<VEC> place_of(int c, int d) {
  Place<VEC> p;
  const int start = c * VEC;
  p.in = start < d;
  p.at = p.in ? (ODD ? min(start, d - VEC) : start) : 0;
  p.from = ODD ? start - p.at : 0;
  return p;
}

template <typename T, int VEC>
__device__ __forceinline__ uint4 get(const T* row, int at) {
  if constexpr (VEC == 1) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (sizeof(T) == 2) w.x = *reinterpret_cast<const uint16_t*>(row + at);
    else w.x = *reinterpret_cast<const uint32_t*>(row + at);
    return w;
  } else {
    return load16u(row + at);
  }
}
// A row that is read once and not again, past the caches (8192 x 4096 bf16: forward 49.1 us with,
// 51.7 us without; backward 80.7 and 91.1 us): not where rows start anywhere (ODD), whose boundary
// lines two rows share (2310 x 2049 fp32 backward: 36.8 us with, 34.1 us without).  The outputs
// are stored through the caches; past them, a chain of join, layer, layer and join at 8192 x 4096
// took 371 us for 379 us.
template <typename T, int VEC, bool ODD>
__device__ __forceinline__ uint4 get_once(const T* row, int at) {
  if constexpr (VEC == 1 || ODD) return get<T, VEC>(row, at);
  else return load16u_nt(row + at);
}

// 16 bytes at offset off of a row of row_bytes bytes (16-byte aligned, the same for the wave)
// through a buffer resource over the row: zeros past its end, and a store there is dropped.  Loads
// past the caches, as get_once.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* row, uint32_t row_bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(row), 0, (int)row_bytes, 0x00020000);
}
__device__ __forceinline__ uint4 buffer_load16(const void* row, uint32_t row_bytes, uint32_t off) {
  const auto w = __builtin_amdgcn_raw_buffer_load_b128(row_rsrc(row, row_bytes), (int)off, 0, 2);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void buffer_store16(void* row, uint32_t row_bytes, uint32_t off, uint4 v) {
  typedef unsigned v4u __attribute__((ext_vector_type(4)));
  const v4u w = {v.x, v.y, v.z, v.w};
  __builtin_amdgcn_raw_buffer_store_b128(w, row_rsrc(row, row_bytes), (int)off, 0, 0);
}

template <typename T, int VEC>
__device__ __forceinline__ void val(uint4 w, float* o) {
  if constexpr (VEC == 1) o[0] = sizeof(T) == 2 ? __uint_as_float(w.x << 16) : __uint_as_float(w.x);
  else unpack16<T>(w, o);
}
// Only the elements of a moved-back chunk that are its own (see place_of).
template <typename T, int VEC>
__device__ __forceinline__ void put_own(T* row, int at, int from, const float* v) {
  if (from == 0) {
    if constexpr (VEC == 1) elem_store<T>(row + at, v[0]);
    else store16u(row + at, pack16<T>(v));
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e >= from) elem_store<T>(row + at + e, v[e]);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void put(T* row, int at, const float* v) {
  if constexpr (VEC == 1) elem_store<T>(row + at, v[0]);
  else store16u(row + at, pack16<T>(v));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// Sum over the NW waves of a team (NW == 1: the wave).  `s` holds one float per wave of the
// workgroup; each call uses its own slot array, so one barrier per call is enough.
template <int NW>
__device__ __forceinline__ float team_sum(float v, float* s, int wave, int team) {
  v = wave_sum(v);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0) s[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) v += s[team * NW + i];
  }
  return v;
}

// NW waves per token; workgroups of at least 3 waves.
template <int NW>
struct FwdGeo {
  static constexpr int TEAMS = NW == 1 ? 4 : NW == 2 ? 2 : 1, WAVES = TEAMS * NW;
};
template <typename T, int VEC, bool ODD, int NW, int CH>
__global__ __launch_bounds__(64 * FwdGeo<NW>::WAVES) void norm_fwd_kernel(NormFwdArgs a) {
  constexpr int WAVES = FwdGeo<NW>::WAVES, TEAMS = FwdGeo<NW>::TEAMS;
  __shared__ float s_post[WAVES], s_pre[WAVES];
  const int wave = threadIdx.x >> 6, team = wave / NW;
  const int tl = threadIdx.x - team * NW * 64;  // thread within the team
  const int64_t tok = a.first + (int64_t)blockIdx.x * TEAMS + team;
  // a workgroup of several teams may end past the last token; a team of one wave meets no
  // barrier and leaves, one of more waves repeats the last token (its stores write the same)
  if (NW == 1 && tok >= a.tokens) return;
  const int64_t t = min(tok, a.tokens - 1);
  const int d = a.dim;
  const T* r = reinterpret_cast<const T*>(a.r) + t * a.ldr;
  const T* y = reinterpret_cast<const T*>(a.y) + t * a.ldy;
  Place<VEC> pl[CH];
  uint4 rr[CH], yr[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) pl[j] = place_of<VEC, ODD>(j * NW * 64 + tl, d);
  if (a.y) {
#pragma unroll
    for (int j = 0; j < CH; ++j) yr[j] = get_once<T, VEC, ODD>(y, pl[j].at);
  }
#pragma unroll
  for (int j = 0; j < CH; ++j) rr[j] = get_once<T, VEC, ODD>(r, pl[j].at);

  float x[CH][VEC];
  float inv_post = 1.f;
  if (a.y) {
    if (a.post) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        float v[VEC];
        val<T, VEC>(yr[j], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (pl[j].in && (!ODD || e >= pl[j].from)) ss = __builtin_fmaf(v[e], v[e], ss);
      }
      ss = team_sum<NW>(ss, s_post, wave, team);
      inv_post = 1.f / sqrtf(ss * a.inv_dim + a.eps);
      if (a.rstd_post && tl == 0) a.rstd_post[t] = inv_post;
    }
    const T* gate = reinterpret_cast<const T*>(a.gate) + (a.gate ? (t / a.group_len) * a.ldg : 0);
    const T* post = reinterpret_cast<const T*>(a.post);
    const float k = a.scale * inv_post;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float yv[VEC], rv[VEC], c[VEC];
      val<T, VEC>(yr[j], yv);
      val<T, VEC>(rr[j], rv);
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = k;
      if (post) {
        float w[VEC];
        val<T, VEC>(get<T, VEC>(post, pl[j].at), w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) c[e] *= w[e];
      }
      if (a.gate) {
        float w[VEC];
        val<T, VEC>(get<T, VEC>(gate, pl[j].at), w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) c[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[j][e] = __builtin_fmaf(c[e], yv[e], rv[e]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < CH; ++j) val<T, VEC>(rr[j], x[j]);
  }
  // with no norm on either side no reduction has ordered this row's loads before its stores,
  // which may overlap them (r_out may be r, and a moved-back chunk shares elements)
  if (NW > 1 && !a.pre && !a.post) __syncthreads();
  float inv_pre = 1.f;
  if (a.pre) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (pl[j].in && (!ODD || e >= pl[j].from)) ss = __builtin_fmaf(x[j][e], x[j][e], ss);
    ss = team_sum<NW>(ss, s_pre, wave, team);
    inv_pre = 1.f / sqrtf(ss * a.inv_dim + a.eps);
    if (a.rstd_pre && tl == 0) a.rstd_pre[t] = inv_pre;
  }
  if (a.y) {
    T* ro = reinterpret_cast<T*>(a.r_out) + t * a.ldro;
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (pl[j].in) put<T, VEC>(ro, pl[j].at, x[j]);
  }
  if (a.pre) {
    T* h = reinterpret_cast<T*>(a.h) + t * a.ldh;
    const T* pre = reinterpret_cast<const T*>(a.pre);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float w[VEC];
      val<T, VEC>(get<T, VEC>(pre, pl[j].at), w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] *= x[j][e] * inv_pre;
      if (pl[j].in) put<T, VEC>(h, pl[j].at, w);
    }
  }
}

template <typename T, int VEC, bool ODD, int NW, int CH>
hipError_t run_fwd(NormFwdArgs a, hipStream_t st) {
  constexpr int WAVES = FwdGeo<NW>::WAVES, TEAMS = FwdGeo<NW>::TEAMS;
  const int64_t grid = (a.tokens + TEAMS - 1) / TEAMS, most = max_workgroups(64 * WAVES);
  for (int64_t g = 0; g < grid; g += most) {
    a.first = g * TEAMS;
    hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, ODD, NW, CH>),
                       dim3((unsigned)(grid - g < most ? grid - g : most)), dim3(64 * WAVES), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Waves per token: so many that a lane holds at most two chunks of r and of y, since few registers
// leave many rows in flight (8192 x 4096 bf16, 268 MB: 48.5 us with 4 waves of 2 chunks, 55 us
// with 2 of 4, 72 us with 1 of 8); and up to one chunk where the tokens alone would not fill the
// device (8 x 4096: latency counts).
template <typename T, int VEC, bool ODD>
hipError_t pick_fwd(const NormFwdArgs& a, hipStream_t st) {
  const int64_t chunks = (a.dim + VEC - 1) / VEC;
  const int64_t per = (chunks + 63) / 64;  // chunks per lane of one wave
  if (per <= 1) return run_fwd<T, VEC, ODD, 1, 1>(a, st);
  if (a.tokens <= 1024) {
    if (per <= 4) return run_fwd<T, VEC, ODD, 4, 1>(a, st);
    if (per <= 16) return run_fwd<T, VEC, ODD, 16, 1>(a, st);
  }
  switch ((per + 1) / 2) {
    case 1: return run_fwd<T, VEC, ODD, 1, 2>(a, st);
    case 2: return run_fwd<T, VEC, ODD, 2, 2>(a, st);
    case 3: return run_fwd<T, VEC, ODD, 3, 2>(a, st);
    case 4: return run_fwd<T, VEC, ODD, 4, 2>(a, st);
    case 5: return run_fwd<T, VEC, ODD, 5, 2>(a, st);
    case 6: return run_fwd<T, VEC, ODD, 6, 2>(a, st);
    case 7: return run_fwd<T, VEC, ODD, 7, 2>(a, st);
    case 8: return run_fwd<T, VEC, ODD, 8, 2>(a, st);
  }
  if (per <= 32) return run_fwd<T, VEC, ODD, 16, 2>(a, st);
  if (per <= 64) return run_fwd<T, VEC, ODD, 16, 4>(a, st);
  return hipErrorInvalidValue;  // past norm_max_dim
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// Row plan of the backward: workgroup i handles rows_per_wg consecutive rows of one gate group
// (chunks_per_group workgroups per group), its teams taking rows in turn; or, where groups are
// shorter than a team's share (whole_groups > 0), whole_groups consecutive groups, its teams
// taking groups in turn and writing their gate gradients themselves.
struct NormPlan {
  int64_t wgs, rows_per_wg, chunks_per_group, whole_groups;
};

// Waves per token and chunks per lane of the backward for a row of `chunks` chunks: two chunks per
// lane and as many waves as that takes, so that few lanes idle whatever the width (one chunk per
// lane and twice the waves, in a form of the loop that had branches: as long at 8192 x 4096 bf16, 8 %
// longer at 6500 x 5120, which takes 87.7 us).
// bf16 lanes (256 registers, 8 waves) and fp32 lanes (160 registers, 12 waves) bound the row;
// longer rows (nw 0) go by column strips, see norm_strip_kernel.
void bwd_shape(int64_t chunks, int vec, int* nw, int* ch) {
  const int64_t per = (chunks + 63) / 64;
  *ch = per <= 1 ? 1 : 2;
  *nw = per <= 2 * (vec == 8 ? 8 : 12) ? (int)((per + 1) / 2) : 0;
}
// Teams of a workgroup, as many as its registers allow.
constexpr int bwd_teams(int nw, int vec) { return (vec == 8 ? 8 : 12) / nw; }
constexpr int kStripTeams = 4;

// wgs: the workgroups to aim at.
NormPlan plan_bwd(int64_t tokens, int64_t group_len, int teams, int64_t wgs) {
  NormPlan p{};
  // whole rows: one workgroup per compute unit, whose teams keep enough rows in flight (each
  // prefetches its next row), so that the partial sums, one row per workgroup, stay few (8192 x
  // 4096 bf16: 80.7 us with 256 workgroups, 88.1 us with 512; 2310 x 2049 fp32: 34.1 and 43.1 us)
  int64_t rows = (tokens + wgs - 1) / wgs;
  if (rows < teams) rows = teams;
  if (group_len * teams <= rows) {
    p.whole_groups = rows / group_len;
    const int64_t groups = tokens / group_len;
    p.rows_per_wg = p.whole_groups * group_len;
    p.wgs = (groups + p.whole_groups - 1) / p.whole_groups;
    p.chunks_per_group = 0;
    return p;
  }
  p.chunks_per_group = (group_len + rows - 1) / rows;
  p.rows_per_wg = (group_len + p.chunks_per_group - 1) / p.chunks_per_group;
  p.chunks_per_group = (group_len + p.rows_per_wg - 1) / p.rows_per_wg;
  p.wgs = p.chunks_per_group * (tokens / group_len);
  return p;
}

// The rows of a team in workgroup `wg`'s range (nrows from row0 on), one per iteration: whole
// groups: team q takes groups q, q + teams, ..; else rows q, q + teams, ...
struct TeamRows {
  int64_t row0, nrows, iters, row, in_group, group_len;
  int teams;
  bool whole;
  // token of the current row; the range's first where there is none
  __device__ __forceinline__ int64_t token() const { return row0 + (row < nrows ? row : 0); }
  __device__ __forceinline__ bool live() const { return row < nrows; }
  __device__ __forceinline__ bool first_of_group() const { return whole && in_group == 0; }
  __device__ __forceinline__ bool last_of_group() const { return whole && in_group == group_len - 1; }
  __device__ __forceinline__ void advance() {
    if (!whole) {
      row += teams;
    } else {
      const bool wrap = ++in_group == group_len;
      row += wrap ? (teams - 1) * group_len + 1 : 1;
      in_group = wrap ? 0 : in_group;
    }
  }
};
__device__ __forceinline__ TeamRows team_rows(const NormBwdArgs& a, const NormPlan& pn, int teams,
                                              int team, int64_t wg) {
  TeamRows r;
  r.group_len = a.group_len;
  r.teams = teams;
  r.whole = pn.whole_groups > 0;
  r.in_group = 0;
  if (r.whole) {
    const int64_t groups = a.tokens / a.group_len;
    const int64_t g0 = wg * pn.whole_groups, ng = min(pn.whole_groups, groups - g0);
    r.row0 = g0 * a.group_len;
    r.nrows = ng * a.group_len;
    r.iters = (ng + teams - 1) / teams * a.group_len;
    r.row = team * a.group_len;
  } else {
    const int64_t group = wg / pn.chunks_per_group, c = wg % pn.chunks_per_group;
    r.row0 = group * a.group_len + c * pn.rows_per_wg;
    r.nrows = min(pn.rows_per_wg, a.group_len - c * pn.rows_per_wg);
    r.iters = (r.nrows + teams - 1) / teams;
    r.row = team;
  }
  return r;
}

// FAST: every optional input is there (the gate may be missing: ones) and every row starts on 16
// bytes.  Loads and stores then go through buffer resources of one row, which give zeros (that add
// nothing) past its end and drop what is stored there, or of no bytes where a team has no row: the
// loop has no branch around a memory access, and no wait covers more than the row it needs.
// WHOLE: the plan's whole groups, whose gate rows are loaded with each row.
template <typename T, int VEC, bool ODD, int NW, int CH, bool FAST, bool WHOLE>
__global__ __launch_bounds__(64 * NW * bwd_teams(NW, VEC)) void norm_bwd_kernel(NormBwdArgs a,
                                                                           NormPlan pn) {
  constexpr int TEAMS = bwd_teams(NW, VEC), WAVES = NW * TEAMS;
  __shared__ float s_red[2][3][WAVES];
  extern __shared__ float s_fold[];  // TEAMS > 1: (TEAMS - 1) x (columns) x 3 floats, see below
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), team = wave / NW;
  const int tl = threadIdx.x - team * NW * 64;
  const int d = a.dim;
  const T* gate = reinterpret_cast<const T*>(a.gate);
  const T* post = reinterpret_cast<const T*>(a.post);
  const T* pre = reinterpret_cast<const T*>(a.pre);
  const bool has_in = FAST || a.dr_out, has_pre = FAST || pre, has_y = FAST || a.y,
             has_post = FAST || post;

  Place<VEC> pl[CH];
  uint32_t off[CH];  // byte offset of a chunk in its row (FAST; past the row for idle lanes)
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    pl[j] = place_of<VEC, ODD>(j * NW * 64 + tl, d);
    off[j] = (uint32_t)(j * NW * 64 + tl) * (uint32_t)(VEC * sizeof(T));
  }
  const uint32_t row_bytes = (uint32_t)d * (uint32_t)sizeof(T);
  // A lane keeps its weights in their stored form and has the next row's loads in flight while a
  // row is reduced and stored.
  const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
  const uint32_t one = sizeof(T) == 2 ? 0x3f803f80u : 0x3f800000u;
  const uint4 ones4 = make_uint4(one, one, one, one);
  uint4 wpost[CH], wpre[CH], wgate[CH];
  float spost[CH][VEC], spre[CH][VEC], sgate[CH][VEC];
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) spost[j][e] = spre[j][e] = sgate[j][e] = 0.f;

  TeamRows now = team_rows(a, pn, TEAMS, team, blockIdx.x);
  TeamRows then = now;  // one row ahead
  const int64_t iters = now.iters;
  struct Row {
    uint4 g, h, r, y, w;
  };
  auto part = [&](const void* base, int64_t ld, int64_t t, int j) __attribute__((always_inline)) {
    const T* row = reinterpret_cast<const T*>(base) + t * ld;
    if constexpr (FAST) return buffer_load16(row, then.live() ? row_bytes : 0u, off[j]);
    else return get_once<T, VEC, ODD>(row, pl[j].at);
  };
  Row cur[CH], nxt[CH];
  float nb = 0.f, na = 1.f;
  auto ahead = [&]() __attribute__((always_inline)) {
    const int64_t t = then.token();
    if (has_pre) nb = a.rstd_pre[t];
    if (has_post) na = a.rstd_post[t];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      nxt[j].g = has_in ? part(a.dr_out, a.lddro, t, j) : zero4;
      nxt[j].h = has_pre ? part(a.dh, a.lddh, t, j) : zero4;
      nxt[j].r = has_pre ? part(a.r_out, a.ldro, t, j) : zero4;
      nxt[j].y = has_y ? part(a.y, a.ldy, t, j) : zero4;
      if (WHOLE)
        nxt[j].w = gate ? get<T, VEC>(gate + t / a.group_len * a.ldg, pl[j].at) : ones4;
    }
    then.advance();
  };
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    wpost[j] = has_post ? get<T, VEC>(post, pl[j].at) : ones4;
    wpre[j] = has_pre ? get<T, VEC>(pre, pl[j].at) : ones4;
    wgate[j] = gate ? get<T, VEC>(gate + now.token() / a.group_len * a.ldg, pl[j].at) : ones4;
  }
  ahead();
  for (int64_t it = 0; it < iters; ++it) {
    const bool live = now.live();
    const int64_t t = now.token();
    keep_raw(wpost);
    keep_raw(wpre);
    keep_raw(wgate);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      cur[j] = nxt[j];
      if (WHOLE) wgate[j] = nxt[j].w;
      if (!FAST && !pl[j].in) cur[j].g = cur[j].h = cur[j].r = cur[j].y = zero4;
    }
    const float b = nb, ar = na;
    ahead();
    // the three sums: m1 = sum u rhat, A = sum c yhat (dr' + b u), B = sum c yhat b rhat
    float m1 = 0.f, sa = 0.f, sb = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float g[VEC], u[VEC], rv[VEC], yv[VEC], wp[VEC], wq[VEC], wg[VEC];
      val<T, VEC>(cur[j].g, g);
      val<T, VEC>(cur[j].h, u);
      val<T, VEC>(cur[j].r, rv);
      val<T, VEC>(cur[j].y, yv);
      val<T, VEC>(wpre[j], wq);
      val<T, VEC>(wpost[j], wp);
      val<T, VEC>(wgate[j], wg);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        u[e] *= wq[e];
        rv[e] *= b;
        const float cy = (wp[e] * wg[e]) * (yv[e] * ar);
        const bool own = !ODD || e >= pl[j].from;  // the chunk before counts the shared elements
        m1 = own ? __builtin_fmaf(u[e], rv[e], m1) : m1;
        sa = own ? __builtin_fmaf(cy, __builtin_fmaf(b, u[e], g[e]), sa) : sa;
        sb = own ? __builtin_fmaf(cy * b, rv[e], sb) : sb;
      }
    }
    m1 = wave_sum(m1);
    sa = wave_sum(sa);
    sb = wave_sum(sb);
    if constexpr (NW > 1) {
      float(*s)[WAVES] = s_red[it & 1];  // the other buffer is still being read
      if ((tl & 63) == 0) {
        s[0][wave] = m1;
        s[1][wave] = sa;
        s[2][wave] = sb;
      }
      __syncthreads();
      if constexpr (NW <= 4) {
        m1 = sa = sb = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          m1 += s[0][team * NW + i];
          sa += s[1][team * NW + i];
          sb += s[2][team * NW + i];
        }
      } else {  // a lane per wave's sum: few registers
        const int i = team * NW + min(tl & 63, NW - 1);
        const bool mine = (tl & 63) < NW;
        m1 = wave_sum(mine ? s[0][i] : 0.f);
        sa = wave_sum(mine ? s[1][i] : 0.f);
        sb = wave_sum(mine ? s[2][i] : 0.f);
      }
    }
    m1 *= a.inv_dim;
    const float bm = b * m1;
    const float m2 = has_post ? (sa - m1 * sb) * a.scale * a.inv_dim : 0.f;
    keep_raw(wpost);
    keep_raw(wpre);
    keep_raw(wgate);
    T* dr = reinterpret_cast<T*>(a.dr) + t * a.lddr;
    T* dy = reinterpret_cast<T*>(a.dy) + t * a.lddy;
    // Without a row (!live) the sums stay as they are: selected, not multiplied by zero, since the row
    // read in its place, its factors and the weights may hold infinities.
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      keep_raw1(cur[j].g);
      keep_raw1(cur[j].h);
      keep_raw1(cur[j].r);
      keep_raw1(cur[j].y);
      float g[VEC], u[VEC], rv[VEC], yv[VEC], wp[VEC], wq[VEC], wg[VEC], o[VEC];
      val<T, VEC>(cur[j].g, g);
      val<T, VEC>(cur[j].h, u);
      val<T, VEC>(cur[j].r, rv);
      val<T, VEC>(cur[j].y, yv);
      val<T, VEC>(wpre[j], wq);
      val<T, VEC>(wpost[j], wp);
      val<T, VEC>(wgate[j], wg);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float rhat = rv[e] * b, yhat = yv[e] * ar;
        g[e] = __builtin_fmaf(-bm, rhat, __builtin_fmaf(b, u[e] * wq[e], g[e]));
        const float sG = a.scale * g[e], gy = sG * yhat;
        spre[j][e] = live ? __builtin_fmaf(u[e], rhat, spre[j][e]) : spre[j][e];
        sgate[j][e] = live ? __builtin_fmaf(gy, wp[e], sgate[j][e]) : sgate[j][e];
        spost[j][e] = live ? __builtin_fmaf(gy, wg[e], spost[j][e]) : spost[j][e];
        o[e] = ar * __builtin_fmaf(-m2, yhat, sG * wg[e] * wp[e]);
      }
      if constexpr (FAST) {
        buffer_store16(dr, live ? row_bytes : 0u, off[j], pack16<T>(g));
        buffer_store16(dy, live ? row_bytes : 0u, off[j], pack16<T>(o));
      } else if (live && pl[j].in) {
        put<T, VEC>(dr, pl[j].at, g);
        if (has_y) put<T, VEC>(dy, pl[j].at, o);
      }
    }
    if (WHOLE) {  // the group's last row writes its gate gradient
      const bool last = now.last_of_group();
      const bool put_gate = last && live && a.dgate;
      T* dg = reinterpret_cast<T*>(a.dgate) + t / a.group_len * (int64_t)d;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if constexpr (FAST)
          buffer_store16(dg, put_gate ? row_bytes : 0u, off[j], pack16<T>(sgate[j]));
        else if (put_gate && pl[j].in)
          put<T, VEC>(dg, pl[j].at, sgate[j]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) sgate[j][e] = last ? 0.f : sgate[j][e];
      }
    }
    now.advance();
  }
  // fold the teams: team q's sums are added in team order, one sum at a time, through
  // (TEAMS - 1) x 64 NW CH VEC floats of LDS, and the workgroup's partial rows are written
  constexpr int COLS = NW * 64 * CH * VEC;
  const bool want[3] = {a.part_post != nullptr, a.part_pre != nullptr,
                        a.part_gate != nullptr};
  float* out[3] = {a.part_post, a.part_pre, a.part_gate};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (!want[k]) continue;
    float(*s)[VEC] = k == 0 ? spost : k == 1 ? spre : sgate;
    if constexpr (TEAMS > 1) {
      __syncthreads();
      if (team > 0) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            s_fold[(team - 1) * COLS + (j * VEC + e) * NW * 64 + tl] = s[j][e];
      }
      __syncthreads();
    }
    if (team == 0) {
      float* o = out[k] + (int64_t)blockIdx.x * d;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float v = s[j][e];
          for (int q = 0; q < TEAMS - 1; ++q) v += s_fold[q * COLS + (j * VEC + e) * NW * 64 + tl];
          if (pl[j].in && (!ODD || e >= pl[j].from)) o[pl[j].at + e] = v;
        }
      }
    }
  }
}

// Second launch of the backward: the partial rows of each sum, added in a fixed order.  Sum
// rows: 0 dpost and 1 dpre over all workgroups, then the gate groups over their chunks.  A
// workgroup takes 64 columns of one sum row; its 16 waves take the partial rows in turn and are
// added in wave order.
template <typename T>
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormBwdArgs a, NormPlan pn) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  int64_t which = blockIdx.y;
  const float* p;
  T* o;
  int64_t n;
  const int nw = (a.part_post ? 1 : 0) + (a.part_pre ? 1 : 0);
  if (which < nw) {
    const bool is_post = a.part_post && which == 0;
    p = is_post ? a.part_post : a.part_pre;
    o = reinterpret_cast<T*>(is_post ? a.dpost : a.dpre);
    n = pn.wgs;
  } else {
    const int64_t g = which - nw;
    p = a.part_gate + g * pn.chunks_per_group * (int64_t)a.dim;
    o = reinterpret_cast<T*>(a.dgate) + g * (int64_t)a.dim;
    n = pn.chunks_per_group;
  }
  float v = 0.f;
  if (col < a.dim) {
#pragma unroll 16
    for (int64_t i = w; i < n; i += 16) v += p[i * a.dim + col];
  }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && col < a.dim) {
    v = s[0][lane];
#pragma unroll
    for (int i = 1; i < 16; ++i) v += s[i][lane];
    elem_store<T>(o + col, v);
  }
}

struct BwdLayout {
  NormPlan plan;
  int nw, ch, vec;
  size_t post, pre, gate, stats, total;  // byte offsets of the partial rows and row statistics
};

BwdLayout bwd_layout(int64_t tokens, int64_t dim, int64_t group_len, int in_bf16, bool post,
                     bool pre, bool gate) {
  BwdLayout l{};
  l.vec = in_bf16 ? 8 : 4;
  if (dim < l.vec) l.vec = 1;
  bwd_shape((dim + l.vec - 1) / l.vec, l.vec, &l.nw, &l.ch);
  if (l.nw > 0) {
    l.plan = plan_bwd(tokens, group_len, bwd_teams(l.nw, l.vec), 256);
  } else {
    const int64_t strips = (dim + 64 * l.vec - 1) / (64 * l.vec);
    l.plan = plan_bwd(tokens, group_len, kStripTeams, (1024 + strips - 1) / strips);
  }
  const size_t rows = (size_t)l.plan.wgs * (size_t)dim * 4;
  l.post = 0;
  l.pre = post ? rows : 0;
  l.gate = l.pre + (pre ? rows : 0);
  l.stats = l.gate + (gate && l.plan.whole_groups == 0 ? rows : 0);
  l.total = l.stats + (l.nw == 0 ? (size_t)tokens * 8 : 0);
  return l;
}

// The widest rows, which a workgroup's registers do not hold beside their columns' sums: a first
// launch reduces each row to the two numbers that its gradient needs, bm = b mean(u rhat) and the
// mean m2 of dy's formula; a second takes strips of 64 chunks, a wave per row of a strip, and does
// the rest (2048 x 16384 bf16: 138 us, everything being read twice; with the row held and registers
// spilled, more than twice that).  Only the second stores, so dr and dy may be
// inputs as before; a moved-back chunk's shared elements are another workgroup's and not stored.
template <typename T, int VEC, bool ODD>
__global__ __launch_bounds__(512) void norm_stats_kernel(NormBwdArgs a) {
  constexpr int WAVES = 8;
  __shared__ float s_red[3][WAVES];
  const int64_t t = a.first + blockIdx.x;
  const T* dr_out = reinterpret_cast<const T*>(a.dr_out) + t * a.lddro;
  const T* dh = reinterpret_cast<const T*>(a.dh) + t * a.lddh;
  const T* r = reinterpret_cast<const T*>(a.r_out) + t * a.ldro;
  const T* y = reinterpret_cast<const T*>(a.y) + t * a.ldy;
  const T* gate = reinterpret_cast<const T*>(a.gate) + (a.gate ? t / a.group_len * a.ldg : 0);
  const T* post = reinterpret_cast<const T*>(a.post);
  const T* pre = reinterpret_cast<const T*>(a.pre);
  const float b = a.pre ? a.rstd_pre[t] : 0.f, ar = a.post ? a.rstd_post[t] : 1.f;
  float m1 = 0.f, sa = 0.f, sb = 0.f;
  for (int c = threadIdx.x; c * VEC < a.dim; c += 64 * WAVES) {
    const Place<VEC> p = place_of<VEC, ODD>(c, a.dim);
    float g[VEC] = {}, u[VEC] = {}, rv[VEC] = {}, cy[VEC] = {}, w[VEC];
    if (a.dr_out) val<T, VEC>(get<T, VEC>(dr_out, p.at), g);
    if (a.pre) {
      val<T, VEC>(get<T, VEC>(dh, p.at), u);
      val<T, VEC>(get<T, VEC>(r, p.at), rv);
      val<T, VEC>(get<T, VEC>(pre, p.at), w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[e] *= w[e];
    }
    if (a.post) {
      val<T, VEC>(get<T, VEC>(y, p.at), cy);
      val<T, VEC>(get<T, VEC>(post, p.at), w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) cy[e] *= ar * w[e];
      if (a.gate) {
        val<T, VEC>(get<T, VEC>(gate, p.at), w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) cy[e] *= w[e];
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (ODD && e < p.from) continue;
      const float rhat = rv[e] * b;
      m1 = __builtin_fmaf(u[e], rhat, m1);
      sa = __builtin_fmaf(cy[e], __builtin_fmaf(b, u[e], g[e]), sa);
      sb = __builtin_fmaf(cy[e] * b, rhat, sb);
    }
  }
  const float s[3] = {wave_sum(m1), wave_sum(sa), wave_sum(sb)};
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < 3; ++k) s_red[k][threadIdx.x >> 6] = s[k];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float v[3] = {};
#pragma unroll
    for (int i = 0; i < WAVES; ++i)
#pragma unroll
      for (int k = 0; k < 3; ++k) v[k] += s_red[k][i];
    m1 = v[0] * a.inv_dim;
    a.stats[2 * t] = b * m1;
    a.stats[2 * t + 1] = a.post ? (v[1] - m1 * v[2]) * a.scale * a.inv_dim : 0.f;
  }
}

template <typename T, int VEC, bool ODD>
__global__ __launch_bounds__(64 * kStripTeams) void norm_strip_kernel(NormBwdArgs a, NormPlan pn) {
  constexpr int TEAMS = kStripTeams;
  __shared__ float s_fold[TEAMS - 1][VEC][64];
  const int lane = threadIdx.x & 63;
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const T* gate = reinterpret_cast<const T*>(a.gate);
  const Place<VEC> pl = place_of<VEC, ODD>((int)blockIdx.x * 64 + lane, a.dim);
  const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
  const uint32_t one = sizeof(T) == 2 ? 0x3f803f80u : 0x3f800000u;
  const uint4 ones4 = make_uint4(one, one, one, one);
  const uint4 wpost = a.post ? get<T, VEC>(reinterpret_cast<const T*>(a.post), pl.at) : ones4;
  const uint4 wpre = a.pre ? get<T, VEC>(reinterpret_cast<const T*>(a.pre), pl.at) : ones4;
  uint4 wgate = ones4;
  float sums[3][VEC] = {};  // post, pre, gate
  TeamRows now = team_rows(a, pn, TEAMS, team, blockIdx.y);
  TeamRows then = now;
  const int64_t iters = now.iters;
  struct Row {
    uint4 g, h, r, y;
    float b, a, bm, m2;
  } nxt;
  auto ahead = [&]() __attribute__((always_inline)) {
    const int64_t t = then.token();
    then.advance();
    auto part = [&](const void* base, int64_t ld) {
      return get_once<T, VEC, ODD>(reinterpret_cast<const T*>(base) + t * ld, pl.at);
    };
    nxt.b = a.pre ? a.rstd_pre[t] : 0.f;
    nxt.a = a.post ? a.rstd_post[t] : 1.f;
    nxt.bm = a.stats[2 * t];
    nxt.m2 = a.stats[2 * t + 1];
    nxt.g = a.dr_out ? part(a.dr_out, a.lddro) : zero4;
    nxt.h = a.pre ? part(a.dh, a.lddh) : zero4;
    nxt.r = a.pre ? part(a.r_out, a.ldro) : zero4;
    nxt.y = a.y ? part(a.y, a.ldy) : zero4;
  };
  if (gate) wgate = get<T, VEC>(gate + now.token() / a.group_len * a.ldg, pl.at);
  ahead();
  for (int64_t it = 0; it < iters; ++it) {
    const bool live = now.live();
    const int64_t t = now.token();
    if (gate && now.first_of_group())
      wgate = get<T, VEC>(gate + t / a.group_len * a.ldg, pl.at);
    const Row cur = nxt;
    ahead();
    float g[VEC], u[VEC], rv[VEC], yv[VEC], wp[VEC], wq[VEC], wg[VEC], o[VEC];
    val<T, VEC>(cur.g, g);
    val<T, VEC>(cur.h, u);
    val<T, VEC>(cur.r, rv);
    val<T, VEC>(cur.y, yv);
    val<T, VEC>(wpre, wq);
    val<T, VEC>(wpost, wp);
    val<T, VEC>(wgate, wg);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {  // !live: see norm_bwd_kernel
      const float rhat = rv[e] * cur.b, yhat = yv[e] * cur.a;
      g[e] = __builtin_fmaf(-cur.bm, rhat, __builtin_fmaf(cur.b, u[e] * wq[e], g[e]));
      const float sG = a.scale * g[e], gy = sG * yhat;
      sums[1][e] = live ? __builtin_fmaf(u[e], rhat, sums[1][e]) : sums[1][e];
      sums[2][e] = live ? __builtin_fmaf(gy, wp[e], sums[2][e]) : sums[2][e];
      sums[0][e] = live ? __builtin_fmaf(gy, wg[e], sums[0][e]) : sums[0][e];
      o[e] = cur.a * __builtin_fmaf(-cur.m2, yhat, sG * wg[e] * wp[e]);
    }
    if (live && pl.in) {
      put_own<T, VEC>(reinterpret_cast<T*>(a.dr) + t * a.lddr, pl.at, pl.from, g);
      if (a.y) put_own<T, VEC>(reinterpret_cast<T*>(a.dy) + t * a.lddy, pl.at, pl.from, o);
    }
    if (now.last_of_group()) {  // whole groups: this wave's own gate row
      if (a.dgate && live && pl.in)
        put_own<T, VEC>(reinterpret_cast<T*>(a.dgate) + t / a.group_len * (int64_t)a.dim, pl.at,
                        pl.from, sums[2]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) sums[2][e] = 0.f;
    }
    now.advance();
  }
  float* out[3] = {a.part_post, a.part_pre, a.part_gate};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (!out[k]) continue;
    __syncthreads();
    if (team > 0) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) s_fold[team - 1][e][lane] = sums[k][e];
    }
    __syncthreads();
    if (team == 0 && pl.in) {
      float* o = out[k] + (int64_t)blockIdx.y * a.dim;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float v = sums[k][e];
#pragma unroll
        for (int q = 0; q < TEAMS - 1; ++q) v += s_fold[q][e][lane];
        if (e >= pl.from) o[pl.at + e] = v;
      }
    }
  }
}

template <typename T, int VEC, bool ODD>
hipError_t run_strips(NormBwdArgs a, const NormPlan& pn, hipStream_t st) {
  const int64_t most = max_workgroups(512);
  for (a.first = 0; a.first < a.tokens; a.first += most) {
    const int64_t left = a.tokens - a.first;
    hipLaunchKernelGGL((norm_stats_kernel<T, VEC, ODD>), dim3((unsigned)(left < most ? left : most)),
                       dim3(512), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const unsigned strips = (unsigned)((a.dim + 64 * VEC - 1) / (64 * VEC));
  hipLaunchKernelGGL((norm_strip_kernel<T, VEC, ODD>), dim3(strips, (unsigned)pn.wgs),
                     dim3(64 * kStripTeams), 0, st, a, pn);
  return hipGetLastError();
}

template <typename T, int VEC, bool ODD, int NW, int CH>
hipError_t run_bwd(const NormBwdArgs& a, const NormPlan& pn, hipStream_t st) {
  constexpr int TEAMS = bwd_teams(NW, VEC);
  constexpr int LDS = (TEAMS - 1) * NW * 64 * CH * VEC * 4;
  static_assert(LDS < 60000, "the fold's LDS fits a workgroup's default limit");
  const dim3 grid((unsigned)pn.wgs), block(64 * NW * TEAMS);
  const bool whole = pn.whole_groups > 0;
  if constexpr (!ODD && VEC > 1) {
    auto on16 = [](const void* p, int64_t ld) {
      return ((reinterpret_cast<uintptr_t>(p) | (uint64_t)ld * sizeof(T)) & 15) == 0;
    };
    if (a.dr_out && a.pre && a.y && a.post && on16(a.dr_out, a.lddro) && on16(a.dh, a.lddh) &&
        on16(a.r_out, a.ldro) && on16(a.y, a.ldy) && on16(a.dr, a.lddr) && on16(a.dy, a.lddy) &&
        on16(a.dgate, a.dim)) {
      if (whole)
        hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, ODD, NW, CH, true, true>), grid, block,
                           LDS, st, a, pn);
      else
        hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, ODD, NW, CH, true, false>), grid, block,
                           LDS, st, a, pn);
      return hipGetLastError();
    }
  }
  if (whole)
    hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, ODD, NW, CH, false, true>), grid, block,
                           LDS, st, a, pn);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, ODD, NW, CH, false, false>), grid, block,
                           LDS, st, a, pn);
  return hipGetLastError();
}

template <typename T, int VEC, bool ODD>
hipError_t pick_bwd(const NormBwdArgs& a, const BwdLayout& l, hipStream_t st) {
  if (l.nw == 0) return run_strips<T, VEC, ODD>(a, l.plan, st);
  if (l.ch == 1) return run_bwd<T, VEC, ODD, 1, 1>(a, l.plan, st);
  switch (l.nw) {
    case 1: return run_bwd<T, VEC, ODD, 1, 2>(a, l.plan, st);
    case 2: return run_bwd<T, VEC, ODD, 2, 2>(a, l.plan, st);
    case 3: return run_bwd<T, VEC, ODD, 3, 2>(a, l.plan, st);
    case 4: return run_bwd<T, VEC, ODD, 4, 2>(a, l.plan, st);
    case 5: return run_bwd<T, VEC, ODD, 5, 2>(a, l.plan, st);
    case 6: return run_bwd<T, VEC, ODD, 6, 2>(a, l.plan, st);
    case 7: return run_bwd<T, VEC, ODD, 7, 2>(a, l.plan, st);
    case 8: return run_bwd<T, VEC, ODD, 8, 2>(a, l.plan, st);
  }
  if constexpr (VEC == 4) {
    switch (l.nw) {
      case 9: return run_bwd<T, VEC, ODD, 9, 2>(a, l.plan, st);
      case 10: return run_bwd<T, VEC, ODD, 10, 2>(a, l.plan, st);
      case 11: return run_bwd<T, VEC, ODD, 11, 2>(a, l.plan, st);
      case 12: return run_bwd<T, VEC, ODD, 12, 2>(a, l.plan, st);
    }
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t bwd_type(NormBwdArgs a, const BwdLayout& l, hipStream_t st) {
  constexpr int VEC = RowType<T>::VEC;
  hipError_t e = l.vec == 1          ? run_bwd<T, 1, false, 1, 1>(a, l.plan, st)
                 : a.dim % VEC == 0 ? pick_bwd<T, VEC, false>(a, l, st)
                                    : pick_bwd<T, VEC, true>(a, l, st);
  if (e != hipSuccess) return e;
  const int64_t sums = (a.part_post ? 1 : 0) + (a.part_pre ? 1 : 0) +
                       (a.part_gate ? a.tokens / a.group_len : 0);
  if (sums == 0) return hipSuccess;
  hipLaunchKernelGGL((norm_sum_kernel<T>), dim3((unsigned)((a.dim + 63) / 64), (unsigned)sums),
                     dim3(1024), 0, st, a, l.plan);
  return hipGetLastError();
}

}  // namespace

int64_t norm_max_dim(int in_bf16) { return in_bf16 ? 32768 : 16384; }

hipError_t launch_norm_fwd(const NormFwdArgs& a, int in_bf16, hipStream_t st) {
  if (in_bf16) {
    if (a.dim < 8) return run_fwd<uint16_t, 1, false, 1, 1>(a, st);
    return a.dim % 8 == 0 ? pick_fwd<uint16_t, 8, false>(a, st) : pick_fwd<uint16_t, 8, true>(a, st);
  }
  if (a.dim < 4) return run_fwd<float, 1, false, 1, 1>(a, st);
  return a.dim % 4 == 0 ? pick_fwd<float, 4, false>(a, st) : pick_fwd<float, 4, true>(a, st);
}

size_t norm_bwd_ws_bytes(int64_t tokens, int64_t dim, int64_t group_len, int in_bf16, bool post,
                         bool pre, bool gate) {
  return bwd_layout(tokens, dim, group_len, in_bf16, post, pre, gate).total;
}

hipError_t launch_norm_bwd(NormBwdArgs a, int in_bf16, void* ws, hipStream_t st) {
  const BwdLayout l = bwd_layout(a.tokens, a.dim, a.group_len, in_bf16, a.dpost != nullptr,
                                 a.dpre != nullptr, a.dgate != nullptr);
  char* base = static_cast<char*>(ws);
  a.part_post = a.dpost ? reinterpret_cast<float*>(base + l.post) : nullptr;
  a.part_pre = a.dpre ? reinterpret_cast<float*>(base + l.pre) : nullptr;
  a.part_gate = a.dgate && l.plan.whole_groups == 0 ? reinterpret_cast<float*>(base + l.gate) : nullptr;
  a.stats = reinterpret_cast<float*>(base + l.stats);
  return in_bf16 ? bwd_type<uint16_t>(a, l, st) : bwd_type<float>(a, l, st);
}

}  // namespace halo
