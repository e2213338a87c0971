// halo_kernels.h -- internal launch interface between the C ABI layer and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace halo {

// Arguments of one fused rotation + quantisation pass.
struct FqArgs {
  const void* x;       // input, row-major [rows x cols], leading dim ldx (elements)
  int64_t ldx;
  int64_t nvec;        // number of vectors (rows for the rows axis, cols for the cols axis)
  int64_t len;         // rotated length L
  void* q;             // codes [nvec x L], leading dim ldq (elements)
  int64_t ldq;
  float* scale;        // [nvec]
  int64_t vec_per_wg;  // rows kernel: vectors per workgroup (set by the launcher)
  int block;
  float qmax;          // 127, 448, 57344
  float denom;         // fl32(qmax * sqrt(block)): scale = max|b| / denom
  float inv_sqrt_b;    // fl32(1 / sqrt(block)) for the fp32 test mode
  int64_t in_len;      // input elements per vector (<= len); positions [in_len, len) are the
                       // zero padding and are not read
  const uint32_t* signs;  // randomised transform: bit i set negates element i (NULL: none)
  int sr;                 // 1: stochastic rounding of the codes (code types only)
  uint32_t key0, key1;    // Philox4x32-10 key
  uint32_t ctr2, ctr3;    // Philox counter words 2 and 3 (word 0: position / 4, word 1: vector)
  uint32_t polls;         // columns passes that exchange maxima: polls of a waiting task
                          // before it stops waiting (0: the default, 2^20)
  // activation-gradient passes only (launch_fq_*_act): the input is dy = x and the vectors rotated
  // are those of dz = dy act'(z), z [rows x cols] with x's leading dimension (bf16); db_part: the
  // columns pass's sums of dz over each task's rows, [parts x nvec] fp32, or, where a task holds
  // whole columns and db is not NULL, db [nvec] bf16 itself
  const void* z;
  int act;
  float* db_part;
  uint16_t* db;
  // the general form of these passes (launch_fq_*_kept): z's form (zk: a Kept of checkpoint.h) and
  // its powers
  int zk;
  const uint8_t* zw;
  // x itself kept in 8 bits (columns passes of launch_fq_batch_kept): its form and powers
  int xk;
  const uint8_t* xw;
};

// in_bf16: 1 for bf16 input, 0 for fp32.  qt: 0 INT8, 1 E4M3, 2 E5M2, 3 fp32 values.
// axis: 0 rows, 1 cols.  ws / ws_bytes: scratch for the single-read columns kernel (may be
// NULL / 0: the columns pass then reads its input twice).
hipError_t launch_fwht_quant(const FqArgs& a, int in_bf16, int qt, int axis, void* ws,
                             size_t ws_bytes, hipStream_t st);

// Scratch bytes the single-read columns kernel needs for columns of `rows` elements (0 when
// it needs none or does not cover the shape), for bf16 and fp32 input alike.
size_t fq_cols2_ws_bytes(int64_t rows, int64_t cols, int block);
// Whether the single-read columns kernel takes the pass (bf16 or fp32 input; fp32 with
// stochastic rounding is not covered) given ws_bytes of scratch.
bool fq_cols2_supported(int64_t rows, int64_t cols, int block, int in_bf16, bool sr,
                        size_t ws_bytes);
hipError_t launch_fq_cols2(const FqArgs& a, int in_bf16, int qt, void* ws, hipStream_t st);

// What a layer backward's dY passes take: dY as it is, dz = dY act'(z) of a bf16 z or of a z in any
// kept form, or a dz that is stored in fp32 (columns passes, which then sum it over the rows too).
enum DyForm { kDyPlain = 0, kDyAct = 1, kDyKept = 2, kDyStored = 3 };

// The rotation passes of a layer backward in one launch (bf16 input): the rows of dY (codes
// qg; may be NULL, else fq_batch_rows_ok(len) must hold) and the single-read column passes of
// W (qw), dY (qg) and X (qw), whose scratch must be zero at launch.  Code type pairs (qg, qw):
// (0, 0), (2, 1), (1, 1).
bool fq_batch_rows_ok(int64_t len);
hipError_t launch_fq_batch(const FqArgs* rows, const FqArgs& cw, void* ws_w, const FqArgs& cdy,
                           void* ws_dy, const FqArgs& cx, void* ws_x, int qg, int qw,
                           hipStream_t st);

// The same with dY's passes taken from dy and z (see FqArgs::z), nearest rounding, blocks
// fq_act_block_ok: the rows of dz (NULL, or fq_batch_rows_ok(len)) and the columns of W, dz and X
// in one launch; and the rows of dz alone.  fq_act_parts: rows of db_part (1: whole columns).
bool fq_act_block_ok(int block);
int64_t fq_act_parts(int64_t rows, int block);
hipError_t launch_fq_batch_act(const FqArgs* rows, const FqArgs& cw, void* ws_w, const FqArgs& cdy,
                               void* ws_dy, const FqArgs& cx, void* ws_x, int qg, int qw,
                               hipStream_t st);

// The same from kept activations: x (cx.xk) and z (zk) in any form; form: what dY's passes take (a
// DyForm; a stored dz is fp32, and its rows are another pass's).
hipError_t launch_fq_batch_kept(const FqArgs* rows, const FqArgs& cw, void* ws_w, const FqArgs& cdy,
                                void* ws_dy, const FqArgs& cx, void* ws_x, int qg, int qw, int form,
                                hipStream_t st);

// The rows pass of the gated layer's gradient (glu_rows.hip): dz = [dy u act'(g), dy act(g)] formed in
// fp32, stored, rotated and quantised in one pass.  dy [rows x n] and z [2 rows x n] (any kept form);
// n as glu_rows_ok; nearest rounding.
struct GluRowsArgs {
  const uint16_t* dy;
  const void* z;
  const uint8_t* zw;
  int zk, act;
  int64_t rows, n;
  float* dz;             // [rows x 2 n]
  uint8_t* q;            // codes [rows x nq], nq = 2 n padded to a multiple of the block
  int64_t nq;
  float* scale;          // [rows]
  int block;
  float qmax, denom;     // as FqArgs
  const uint32_t* signs; // along 2 n, or NULL
  uint32_t* zero;        // words to clear beside the pass (may be NULL)
  int64_t nzero;
};
bool glu_rows_ok(int64_t n, int block);
hipError_t launch_glu_rows(const GluRowsArgs& a, int qt, hipStream_t st);

// Both passes of one bf16 matrix from a single read (fwht_dual.hip): the rows pass ar and
// the columns pass ac of the same x (same block and code type qt), with one scratch whose
// size fq_dual_ws_bytes gives (0: the shape is not covered: rows and cols multiples of 256,
// block <= 256).  fq_dual_supported also asks that all 256 x 256 tiles fit on the device at
// once and that both passes round to nearest.
size_t fq_dual_ws_bytes(int64_t rows, int64_t cols, int block, int in_bf16);
bool fq_dual_supported(int64_t rows, int64_t cols, int block, int in_bf16, int qt, bool sr_rows,
                       bool sr_cols, size_t ws_bytes);
hipError_t launch_fq_dual(const FqArgs& ar, const FqArgs& ac, void* ws, int qt, int prezeroed,
                          hipStream_t st);

// Zero n floats (also used for 32-bit counters).
hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t st);

// Wave-per-slice rows kernel: rows of L = 64 j elements, L <= 65536.
bool fq_rows2_supported(int64_t len, int block);
hipError_t launch_fq_rows2(const FqArgs& a, int in_bf16, int qt, hipStream_t st);

// Two rows passes of the same row length, block, input and code type in one launch (p1 is
// used when has1 != 0), which also clears `nzero` 32-bit words at `zero` (may be NULL).
struct FqPair {
  FqArgs p0, p1;
  int has1;
  int64_t split, first;  // set by the launcher
  uint32_t* zero;
  int64_t nzero;
};
hipError_t launch_fq_rows2_pair(const FqPair& a, int in_bf16, int qt, hipStream_t st);
hipError_t launch_fq_rows2_act(const FqPair& a, int qt, hipStream_t st);
hipError_t launch_fq_rows2_kept(const FqPair& a, int qt, hipStream_t st);

// Up to two single-read column passes over columns of the same length, block, input type
// (in_bf16) and code type in one launch (a1 may be NULL).  prezeroed: the scratch of both was
// cleared earlier on st.
hipError_t launch_fq_cols2_pair(const FqArgs& a0, void* ws0, const FqArgs* a1, void* ws1,
                                int in_bf16, int qt, int prezeroed, hipStream_t st);

// Longest row the single-pass rows kernel takes for this block size.
int64_t fq_rows_max_len(int block);

struct GemmArgs {
  const void* a;  // [m x k], lda (bytes = elements)
  int64_t lda;
  const void* b;  // [n x k], ldb
  int64_t ldb;
  const float* sa;
  const float* sb;
  void* c;        // [m x n], ldc (elements)
  int64_t ldc;
  int64_t m, n, k;
  // the layer's epilogue (launch_gemm_act only): bias [n], residual and z [m x n] (ldc), of the
  // output's type, each may be NULL; act: an Act of epilogue.h
  const void* bias = nullptr;
  const void* res = nullptr;
  void* z = nullptr;
  int act = 0;
  // glu: the gated layer: b holds 2 n rows (gate, then up), sb and bias 2 n entries, y = act(zg) zu
  // is [m x n] and z [m x 2 n]; no residual
  int glu = 0;
  // kept: z's form (a Kept of checkpoint.h); its codes go to z and its powers to zp (the gated
  // layer's z as 2 m rows of n)
  int kept = 0;
  uint8_t* zp = nullptr;
};

// kind: 0 INT8, 1 FP8.  afmt/bfmt (FP8 only): 0 E4M3, 1 E5M2.  out: 0 int32, 1 fp32, 2 bf16.
hipError_t launch_gemm(const GemmArgs& g, int kind, int afmt, int bfmt, int out, hipStream_t st);
// Two products of the same kind, formats and output type in one launch (g1 may be NULL).
hipError_t launch_gemm_pair(const GemmArgs& g, const GemmArgs* g1, int kind, int afmt, int bfmt,
                            int out, hipStream_t st);

// One product with the layer's epilogue: y = act(z) + residual, z = (acc sa) sb + bias.  kind: 0
// INT8, 1 FP8 (E4M3 both).  out: 1 fp32, 2 bf16.  c, res and z rows and bias 16-byte aligned.
hipError_t launch_gemm_act(const GemmArgs& g, int kind, int out, hipStream_t st);
// The same with the contraction split over a workgroup's waves, for few tiles (gemm_ksplit.hip).
hipError_t launch_gemm_ksplit(const GemmArgs& g, int kind, int out, hipStream_t st);
// The same for up to kSkinnyRows rows of a (gemm_skinny.hip).  From 5 rows on wide layers would be faster
// on the 64 tiles (INT8, 2 x 11008 x 4096, 16 rows 29.0 us a call, 23.6 there; 11008 x 4096 18.4, 18.0;
// 4096 x 4096 11.3, 15.4), whose z is rounded once and not twice: the fewest rows, quantised inside, and the
// forward of the same rows would then differ in last bits.
constexpr int kSkinnyRows = 16;
hipError_t launch_gemm_skinny(const GemmArgs& g, int kind, int out, hipStream_t st);
// The same with the rows pass f (its codes and scales stay inside) of m rows in one launch.
bool skinny_fused_ok(int64_t m, int64_t kq, int block);
hipError_t launch_skinny_fused(const GemmArgs& g, const FqArgs& f, int in_bf16, int kind, int out,
                               hipStream_t st);

// Rows of partial sums that launch_dz makes for its db.
int64_t act_grad_parts(int64_t m, int64_t n);
// db (bf16) = the sum of `parts` rows of part, in order.
hipError_t launch_part_sum(const float* part, int64_t parts, int64_t n, uint16_t* db,
                           hipStream_t st);

// dz = dy act'(z) in fp32 of a layer whose z is plain (kept 0) or a checkpoint (kept: a Kept of
// checkpoint.h, zp its powers), or of the gated layer (glu: z is 2 m rows of n, dz [m x 2 n], db [2 n]),
// and its sums db over the rows (bias type: that of dy).  n is a multiple of 8.
struct DzArgs {
  const void *dy, *z;  // z is not read without an activation or a gate
  const uint8_t* zp;
  int kept, act, glu;
  int64_t m, n;
  float* dz;           // or NULL
  void* db;            // or NULL
  float* part;         // scratch of db: act_grad_parts(m, n) x (glu ? 2 n : n)
};
hipError_t launch_dz(const DzArgs& a, int in_bf16, hipStream_t st);

// Rows to 8-bit checkpoints (pack: x is read) and back (x_out is written); see checkpoint.h.  qt: 0
// INT8, 1 E4M3.  Any leading dimension of at least a row, any alignment of whole elements.
struct KeepArgs {
  const void* x;
  void* x_out;
  void* codes;      // [rows x cols], ldc
  uint8_t* powers;  // [rows x ceil(cols / 32)], ldp
  int64_t ldx, ldc, ldp, rows, cols;
  int chunks;  // set by the launcher: chunks of 8 a row, whole groups
};
hipError_t launch_keep(const KeepArgs& a, int in_bf16, int qt, bool pack, hipStream_t st);

// Workgroups of `threads` along x that one launch may hold: HIP counts a launch's threads along an
// axis in 32 bits, and what passes them is dropped without an error.  The row operators, whose
// grids have a team of threads for every token, launch longer calls in pieces.
constexpr int64_t max_workgroups(int threads) { return (int64_t(1) << 31) / threads; }

// The join between two blocks (block_norm.hip).  Optional tensors are NULL; leading dimensions
// in elements; group_len = tokens / gate rows.
struct NormFwdArgs {
  const void *r, *y, *gate, *post, *pre;
  void *r_out, *h;
  float *rstd_post, *rstd_pre;
  int64_t ldr, ldy, ldg, ldro, ldh;
  int64_t tokens, group_len;
  int64_t first;  // set by the launcher: the launch's first token
  int dim;
  float scale, eps, inv_dim;
};
struct NormBwdArgs {
  const void *dr_out, *dh, *r_out, *y, *gate, *post, *pre;
  const float *rstd_post, *rstd_pre;
  void *dr, *dy, *dgate, *dpost, *dpre;
  int64_t lddro, lddh, ldro, ldy, ldg, lddr, lddy;
  int64_t tokens, group_len;
  int dim;
  float scale, inv_dim;
  // set by the launcher: partial sums, and the widest rows' statistics [tokens x 2], of the tokens
  // from `first` on in a launch
  float *part_post, *part_pre, *part_gate, *stats;
  int64_t first;
};
int64_t norm_max_dim(int in_bf16);
hipError_t launch_norm_fwd(const NormFwdArgs& a, int in_bf16, hipStream_t st);
size_t norm_bwd_ws_bytes(int64_t tokens, int64_t dim, int64_t group_len, int in_bf16, bool post,
                         bool pre, bool gate);
hipError_t launch_norm_bwd(NormBwdArgs a, int in_bf16, void* ws, hipStream_t st);

// Distillation loss over a teacher's top logits (distill.hip).
constexpr int kDistillMaxTop = 1024;
struct DistillArgs {
  const void* logits;    // [tokens x vocab], ldl
  const int32_t* idx;    // [tokens x top], ldi
  const void* tlogits;   // [tokens x top], ldt
  const float* dloss;    // NULL: no gradient
  const float* lse_in;   // NULL: computed
  float *loss, *lse;     // NULL: not written
  void* dlogits;         // [tokens x vocab], ldd; may be logits
  int64_t ldl, ldi, ldt, ldd;
  int64_t tokens;
  int64_t first;         // set by the launcher: the launch's first token
  int vocab, top;
  int t_bf16;            // tlogits are bf16
  float tau, inv_tau;
};
hipError_t launch_distill(const DistillArgs& a, int in_bf16, hipStream_t st);

// Matrix-core rate probe (mfma_probe.hip): kind 0 INT8 32x32x32, 1 FP8 32x32x64, 2 FP8
// 16x16x128; mfma_probe_ops gives the operations one launch performs.
hipError_t launch_mfma_probe(int kind, int iters, hipStream_t st);
int64_t mfma_probe_ops(int kind, int iters);

// Let `Kernel` launch with `bytes` of dynamic LDS on the current device.  The attribute belongs
// to one kernel on one device, so it is set once per kernel and device (concurrent first calls
// may both set it); a failure is returned, and tried again on the next call.
template <auto Kernel>
hipError_t allow_dynamic_lds(int bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const bool cached = dev >= 0 && dev < 64;
  if (cached && done[dev].load(std::memory_order_acquire)) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(Kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && cached) done[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace halo
