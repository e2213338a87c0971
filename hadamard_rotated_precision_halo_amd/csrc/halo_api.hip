// halo_api.hip -- the C ABI of libhalo.so (declared in include/halo.h).
//
// Host side only: argument validation (every check runs before any HIP call, so invalid
// calls launch nothing and touch no output), workspace carving, and stream-ordered launches
// of the rotation (fwht_quant.hip) and GEMM (gemm.hip) kernels.  The layer entry points
// compose them exactly as the HALO page places the rotations ("HALO: Hadamard-Assisted
// Lower-Precision Optimization for LLMs", abstract: forward and backward, every large
// product in low precision): each product's two operands are rotated and quantised along
// that product's contraction dimension.
#include "../../include/halo.h"
#include "halo_kernels.h"

#include <atomic>
#include <cmath>
#include <cstring>

using namespace halo;

// Scratch of halo_fwht_quant_noalloc: a fixed device array, one copy per device, held until
// the process ends.  In host code its name stands for a host-side shadow, not a device
// address: the device address comes from hipGetSymbolAddress, once per device.
static __device__ __align__(256) unsigned char scratch[HALO_NOALLOC_SCRATCH_BYTES];

namespace {

// Device address of `scratch` on the current device, looked up once per device (concurrent
// first calls may both look it up and store the same address).  NULL on a HIP error.
void* noalloc_scratch() {
  static std::atomic<void*> addr[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return nullptr;
  void* p = addr[dev].load(std::memory_order_acquire);
  if (p) return p;
  if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return nullptr;
  addr[dev].store(p, std::memory_order_release);
  return p;
}

// Whether an enum argument holds a value in [lo, hi].  A C caller may pass any int in an enum
// parameter, and in C++ loading an enum object whose value lies outside the enum's range is
// undefined, so the value is read through its object representation, before any other use.
// (The argument is taken by reference: passing it by value would itself be such a load.)
template <typename E>
bool enum_in(const E& e, int lo, int hi) {
  static_assert(sizeof(E) == sizeof(int), "C enums are int-sized");
  int v;
  std::memcpy(&v, &e, sizeof v);
  return v >= lo && v <= hi;
}
bool dtype_ok(const halo_dtype& t) { return enum_in(t, HALO_F32, HALO_I32); }
bool axis_ok(const halo_axis& a) { return enum_in(a, HALO_ALONG_ROWS, HALO_ALONG_COLS); }

constexpr int64_t kMaxDim = int64_t(1) << 31;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int esize(halo_dtype t) {
  switch (t) {
    case HALO_F32: return 4;
    case HALO_BF16: return 2;
    case HALO_I8: case HALO_E4M3: case HALO_E5M2: return 1;
    case HALO_I32: return 4;
  }
  return 0;
}

bool valid_block(int32_t b) { return b >= 1 && b <= 4096 && (b & (b - 1)) == 0; }

int qt_index(halo_dtype q) {
  switch (q) {
    case HALO_I8: return 0;
    case HALO_E4M3: return 1;
    case HALO_E5M2: return 2;
    case HALO_F32: return 3;
    default: return -1;
  }
}

float qmax_of(halo_dtype q) {
  return q == HALO_I8 ? 127.f : (q == HALO_E4M3 ? 448.f : (q == HALO_E5M2 ? 57344.f : 1.f));
}

halo_status from_hip(hipError_t e) { return e == hipSuccess ? HALO_OK : HALO_ERR_HIP; }

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Padded (rotated) length of a vector of L elements: a multiple of the block (the zero
// padding of the QWHA page, s5).
int64_t padded_len(int64_t L, int32_t block) { return round_up(L, block); }

// Contraction length of a layer product: the dimension zero-padded to a multiple of the block
// and of 32 (the FP8 matrix cores' k step); blocks past the padded length are all zero and
// get zero codes, so the product equals the one over the padded operands.
int64_t contraction_len(int64_t d, int32_t block) { return round_up(d, block > 32 ? block : 32); }

halo_status check_signs(const uint32_t* signs) {
  return signs && !aligned16(signs) ? HALO_ERR_ALIGN : HALO_OK;
}

// Whether a rows pass over vectors of Lp rotated positions has a kernel: the wave kernel
// (Lp a multiple of 64, one wave per 4096 positions and up to 16 per row; its stochastic
// rounding takes bf16 input), else the older kernel, whose workgroup holds a whole row of up
// to fq_rows_max_len(block) positions.
bool rows_len_ok(int64_t Lp, int32_t block, bool in_bf16, bool sr) {
  return (fq_rows2_supported(Lp, block) && (in_bf16 || !sr)) || Lp <= fq_rows_max_len(block);
}

// Validation of one rotation pass; shared by halo_fwht_quant and the layer calls.
halo_status check_fq(const void* x, halo_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                     halo_axis axis, int32_t block, halo_dtype qt, const void* q, int64_t ldq,
                     const float* scale, const halo_quant_opts* o) {
  if (rows < 0 || cols < 0) return HALO_ERR_SHAPE;
  const bool any = rows > 0 && cols > 0;  // empty matrices may come with NULL pointers
  if ((any && (!x || !q)) || (!scale && (axis == HALO_ALONG_ROWS ? rows : cols) > 0))
    return HALO_ERR_NULL;
  if (xt != HALO_F32 && xt != HALO_BF16) return HALO_ERR_DTYPE;
  if (qt_index(qt) < 0) return HALO_ERR_DTYPE;
  if (axis != HALO_ALONG_ROWS && axis != HALO_ALONG_COLS) return HALO_ERR_SHAPE;
  if (rows >= kMaxDim || cols >= kMaxDim) return HALO_ERR_SHAPE;
  if (ldx < cols || ldx < 1) return HALO_ERR_SHAPE;
  if (!valid_block(block)) return HALO_ERR_BLOCK;
  const int64_t L = axis == HALO_ALONG_ROWS ? cols : rows;
  const int64_t Lp = padded_len(L, block);
  const int64_t nvec = axis == HALO_ALONG_ROWS ? rows : cols;
  if (ldq < Lp || ldq < 1) return HALO_ERR_SHAPE;
  if (Lp % 8 != 0) return HALO_ERR_SHAPE;
  if (axis == HALO_ALONG_ROWS && L % 8 != 0) return HALO_ERR_SHAPE;
  if (axis == HALO_ALONG_COLS && nvec % 8 != 0) return HALO_ERR_SHAPE;
  const bool sr = o && o->rounding == HALO_ROUND_STOCHASTIC;
  if (axis == HALO_ALONG_ROWS && !rows_len_ok(Lp, block, xt == HALO_BF16, sr))
    return HALO_ERR_SHAPE;
  if (o) {
    if (o->rounding != HALO_ROUND_NEAREST_EVEN && o->rounding != HALO_ROUND_STOCHASTIC)
      return HALO_ERR_OPTION;
    if (o->rounding == HALO_ROUND_STOCHASTIC && qt == HALO_F32) return HALO_ERR_OPTION;
  }
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale)) return HALO_ERR_ALIGN;
  if ((ldx * esize(xt)) % 16 != 0 || (ldq * esize(qt)) % 16 != 0) return HALO_ERR_ALIGN;
  if (o && check_signs(o->signs) != HALO_OK) return HALO_ERR_ALIGN;
  return HALO_OK;
}

// Options of one pass: the transform's signs and the rounding of its codes.
struct PassOpts {
  const uint32_t* signs = nullptr;
  int sr = 0;
  uint32_t key0 = 0, key1 = 0, ctr2 = 0, ctr3 = 0;
  uint32_t polls = 0;
};

PassOpts pass_opts(const halo_quant_opts* o) {
  PassOpts p;
  if (!o) return p;
  p.signs = o->signs;
  p.sr = o->rounding == HALO_ROUND_STOCHASTIC ? 1 : 0;
  p.key0 = o->seed[0];
  p.key1 = o->seed[1];
  p.ctr2 = o->counter[0];
  p.ctr3 = o->counter[1];
  p.polls = o->exchange_polls;
  return p;
}

// Arguments of one pass over x[rows x cols]; len: the rotated (padded) length, 0 = the
// vector length padded to a multiple of the block.
FqArgs make_fq(const void* x, int64_t rows, int64_t cols, int64_t ldx, halo_axis axis,
               int32_t block, halo_dtype qt, void* q, int64_t ldq, float* scale,
               const PassOpts& po = PassOpts(), int64_t len = 0) {
  FqArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.nvec = axis == HALO_ALONG_ROWS ? rows : cols;
  a.in_len = axis == HALO_ALONG_ROWS ? cols : rows;
  a.len = len > 0 ? len : padded_len(a.in_len, block);
  a.q = q;
  a.ldq = ldq;
  a.scale = scale;
  a.block = block;
  a.qmax = qmax_of(qt);
  a.denom = (float)((double)a.qmax * std::sqrt((double)block));
  a.inv_sqrt_b = (float)(1.0 / std::sqrt((double)block));
  a.signs = po.signs;
  a.sr = po.sr;
  a.key0 = po.key0;
  a.key1 = po.key1;
  a.ctr2 = po.ctr2;
  a.ctr3 = po.ctr3;
  a.polls = po.polls;
  return a;
}

halo_status run_fa(const FqArgs& a, halo_dtype xt, halo_axis axis, halo_dtype qt, void* ws,
                   size_t ws_bytes, hipStream_t st) {
  return from_hip(launch_fwht_quant(a, xt == HALO_BF16 ? 1 : 0, qt_index(qt), (int)axis, ws,
                                    ws ? ws_bytes : 0, st));
}

halo_status run_fq(const void* x, halo_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                   halo_axis axis, int32_t block, halo_dtype qt, void* q, int64_t ldq,
                   float* scale, void* ws, size_t ws_bytes, hipStream_t st,
                   const PassOpts& po = PassOpts(), int64_t len = 0) {
  const FqArgs a = make_fq(x, rows, cols, ldx, axis, block, qt, q, ldq, scale, po, len);
  return run_fa(a, xt, axis, qt, ws, ws_bytes, st);
}

// Scratch of one rotation pass (the single-read columns kernel's partial maxima and counters);
// len: the rotated (padded) length.
// The same for bf16 and fp32 input.
size_t fq_ws_bytes_len(int64_t len, int64_t nvec, halo_axis axis, int32_t block) {
  if (axis != HALO_ALONG_COLS) return 0;
  return fq_cols2_ws_bytes(len, nvec, block);
}

// The GEMM kernel loads each code operand through a buffer resource of 2^32 - 1 bytes with
// 32-bit byte offsets: an operand of `rows` rows (leading dimension ld bytes, k bytes used per
// row) must end below byte 2^32 - 1 of its base (a load reaching past the resource's size would
// read zeros).  Both ld and k are multiples of 16, so the span is at most 2^32 - 16.
bool operand_fits(int64_t rows, int64_t ld, int64_t k) {
  return rows <= 0 || (rows - 1) * ld + k < (int64_t(1) << 32);
}

halo_status check_gemm(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t m,
                       int64_t n, int64_t k, const void* c, halo_dtype ct, int64_t ldc,
                       const float* sa, const float* sb, int kmult) {
  if (m < 0 || n < 0 || k <= 0 || m >= kMaxDim || n >= kMaxDim || k >= kMaxDim)
    return HALO_ERR_SHAPE;
  // empty operands may come with NULL pointers
  if ((m > 0 && !a) || (n > 0 && !b) || (m > 0 && n > 0 && !c)) return HALO_ERR_NULL;
  if (ct != HALO_I32 && ((m > 0 && !sa) || (n > 0 && !sb))) return HALO_ERR_NULL;
  if (k % kmult != 0) return HALO_ERR_SHAPE;
  if (lda < k || ldb < k || ldc < n || ldc < 1) return HALO_ERR_SHAPE;
  if (!operand_fits(m, lda, k) || !operand_fits(n, ldb, k)) return HALO_ERR_SHAPE;
  if (!aligned16(a) || !aligned16(b) || !aligned16(c)) return HALO_ERR_ALIGN;
  if (lda % 16 != 0 || ldb % 16 != 0 || (ldc * esize(ct)) % 16 != 0) return HALO_ERR_ALIGN;
  return HALO_OK;
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }


// Region sizes of the layer workspace, in carve order; the backward's last region is the
// scratch of its three column passes (W, dY, X: one sub-region each, cleared together by the
// first kernel of the call).
struct WsPlan {
  size_t off[9];
  size_t total;
  size_t scratch_off, scratch_bytes;
  size_t scr_w, scr_dy, scr_x;  // sub-region sizes, in this order
};

WsPlan plan_ws(int64_t m, int64_t n, int64_t k, int backward, int32_t block) {
  WsPlan p{};
  size_t sizes[9];
  int cnt = 0;
  const int64_t kq = contraction_len(k, block), nq = contraction_len(n, block),
                mq = contraction_len(m, block);
  if (!backward) {
    sizes[cnt++] = (size_t)m * kq;     // X codes   [m x kq]
    sizes[cnt++] = (size_t)m * 4;      // X scales
    sizes[cnt++] = (size_t)n * kq;     // W codes   [n x kq]
    sizes[cnt++] = (size_t)n * 4;      // W scales
  } else {
    sizes[cnt++] = (size_t)m * nq;     // dY row codes     [m x nq]
    sizes[cnt++] = (size_t)m * 4;
    sizes[cnt++] = (size_t)k * nq;     // W column codes   [k x nq]
    sizes[cnt++] = (size_t)k * 4;
    sizes[cnt++] = (size_t)n * mq;     // dY column codes  [n x mq]
    sizes[cnt++] = (size_t)n * 4;
    sizes[cnt++] = (size_t)k * mq;     // X column codes   [k x mq]
    sizes[cnt++] = (size_t)k * 4;
  }
  size_t o = 0;
  for (int i = 0; i < cnt; ++i) {
    p.off[i] = o;
    o += round256(sizes[i]);
  }
  if (backward) {
    p.scr_w = round256(fq_ws_bytes_len(nq, k, HALO_ALONG_COLS, block));   // W columns along n
    p.scr_dy = round256(fq_ws_bytes_len(mq, n, HALO_ALONG_COLS, block));  // dY columns along m
    p.scr_x = round256(fq_ws_bytes_len(mq, k, HALO_ALONG_COLS, block));   // X columns along m
  }
  p.scratch_off = o;
  p.scratch_bytes = p.scr_w + p.scr_dy + p.scr_x;
  p.total = o + p.scratch_bytes;
  return p;
}

int gemm_kind_fmt(halo_dtype t) { return t == HALO_E5M2 ? 1 : 0; }

halo_status gemm_any(const void* a, halo_dtype at, int64_t lda, const float* sa, const void* b,
                     halo_dtype bt, int64_t ldb, const float* sb, int64_t m, int64_t n, int64_t k,
                     void* c, halo_dtype ct, int64_t ldc, hipStream_t st) {
  GemmArgs g{a, lda, b, ldb, sa, sb, c, ldc, m, n, k};
  const int out = ct == HALO_I32 ? 0 : (ct == HALO_F32 ? 1 : 2);
  if (at == HALO_I8) return from_hip(launch_gemm(g, 0, 0, 0, out, st));
  return from_hip(launch_gemm(g, 1, gemm_kind_fmt(at), gemm_kind_fmt(bt), out, st));
}

bool layer_dims_ok(int64_t m, int64_t n, int64_t k) {
  return m >= 0 && n >= 0 && k >= 0 && m < kMaxDim && n < kMaxDim && k < kMaxDim;
}

halo_status check_epilogue(const halo_epilogue* ep) {
  if (!ep) return HALO_OK;
  if (ep->activation < HALO_ACT_NONE || ep->activation > HALO_ACT_GELU_ERF) return HALO_ERR_OPTION;
  if (!aligned16(ep->bias) || !aligned16(ep->residual) || !aligned16(ep->z)) return HALO_ERR_ALIGN;
  return HALO_OK;
}

GemmArgs act_args(const void* a, int64_t lda, const float* sa, const void* b, int64_t ldb,
                  const float* sb, int64_t m, int64_t n, int64_t k, void* y,
                  const halo_epilogue* ep) {
  GemmArgs g{a, lda, b, ldb, sa, sb, y, n, m, n, k};
  g.bias = ep->bias;
  g.res = ep->residual;
  g.z = ep->z;
  g.act = ep->activation;
  return g;
}

// The product with its epilogue.
halo_status act_product(const void* a, int64_t lda, const float* sa, const void* b, int64_t ldb,
                        const float* sb, int64_t m, int64_t n, int64_t k, halo_dtype qt, void* y,
                        halo_dtype yt, const halo_epilogue* ep, hipStream_t st) {
  return from_hip(launch_gemm_act(act_args(a, lda, sa, b, ldb, sb, m, n, k, y, ep),
                                  qt == HALO_I8 ? 0 : 1, yt == HALO_F32 ? 1 : 2, st));
}

// Validation of a layer forward.
halo_status check_fwd(const void* x, const void* w, halo_dtype io_type, int64_t m, int64_t n,
                      int64_t k, int32_t block, halo_dtype q_type, const void* y,
                      halo_dtype y_type, const halo_linear_opts* opts) {
  if (!layer_dims_ok(m, n, k) || k == 0) return HALO_ERR_SHAPE;
  if ((m > 0 && !x) || (n > 0 && !w) || (m > 0 && n > 0 && !y)) return HALO_ERR_NULL;
  if (io_type != HALO_F32 && io_type != HALO_BF16) return HALO_ERR_DTYPE;
  if (q_type != HALO_I8 && q_type != HALO_E4M3) return HALO_ERR_DTYPE;
  if (y_type != HALO_F32 && y_type != HALO_BF16) return HALO_ERR_DTYPE;
  if (!valid_block(block)) return HALO_ERR_BLOCK;
  const int64_t kq = contraction_len(k, block);
  if (k % 8 != 0 || !rows_len_ok(kq, block, io_type == HALO_BF16, false)) return HALO_ERR_SHAPE;
  if (!operand_fits(m, kq, kq) || !operand_fits(n, kq, kq)) return HALO_ERR_SHAPE;
  if (opts && (opts->grad_rounding != HALO_ROUND_NEAREST_EVEN &&
               opts->grad_rounding != HALO_ROUND_STOCHASTIC))
    return HALO_ERR_OPTION;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y)) return HALO_ERR_ALIGN;
  if ((n * esize(y_type)) % 16 != 0) return HALO_ERR_ALIGN;
  if (opts && check_signs(opts->signs_k) != HALO_OK) return HALO_ERR_ALIGN;
  return HALO_OK;
}

// The layer forward on validated arguments; ep: the epilogue's part of the product's arguments
// (NULL: the bare product).  ws holds plan_ws(m, n, k, 0, block).total bytes.
halo_status run_fwd(const void* x, const void* w, halo_dtype io_type, int64_t m, int64_t n,
                    int64_t k, int32_t block, halo_dtype q_type, void* y, halo_dtype y_type,
                    const halo_epilogue* ep, const halo_linear_opts* opts, void* ws,
                    hipStream_t st) {
  const WsPlan p = plan_ws(m, n, k, 0, block);
  const int64_t kq = contraction_len(k, block);
  char* base = static_cast<char*>(ws);
  void* qx = base + p.off[0];
  float* sx = reinterpret_cast<float*>(base + p.off[1]);
  void* qw = base + p.off[2];
  float* sw = reinterpret_cast<float*>(base + p.off[3]);
  PassOpts po;  // X and W: the signs along k, nearest-even codes
  if (opts) po.signs = opts->signs_k;
  const FqArgs ax = make_fq(x, m, k, k, HALO_ALONG_ROWS, block, q_type, qx, kq, sx, po, kq);
  const FqArgs aw = make_fq(w, n, k, k, HALO_ALONG_ROWS, block, q_type, qw, kq, sw, po, kq);
  halo_status s = HALO_OK;
  if (fq_rows2_supported(kq, block)) {  // X and W rows in one launch
    FqPair pp{};
    pp.p0 = ax;
    pp.p1 = aw;
    pp.has1 = 1;
    s = from_hip(launch_fq_rows2_pair(pp, io_type == HALO_BF16 ? 1 : 0, qt_index(q_type), st));
  } else {
    s = run_fa(ax, io_type, HALO_ALONG_ROWS, q_type, nullptr, 0, st);
    if (s == HALO_OK) s = run_fa(aw, io_type, HALO_ALONG_ROWS, q_type, nullptr, 0, st);
  }
  if (s == HALO_OK && ep)
    return act_product(qx, kq, sx, qw, kq, sw, m, n, kq, q_type, y, y_type, ep, st);
  if (s == HALO_OK)
    s = gemm_any(qx, q_type, kq, sx, qw, q_type, kq, sw, m, n, kq, y, y_type, n, st);
  return s;
}

// Validation of a layer backward; rot_type: the type dY's rows are rotated in.
halo_status check_bwd(const void* dy, halo_dtype rot_type, const void* x, const void* w,
                      halo_dtype io_type, int64_t m, int64_t n, int64_t k, int32_t block,
                      halo_dtype q_type, halo_dtype grad_q_type, const void* dx, const void* dw,
                      const halo_linear_opts* opts) {
  if (!dy || !x || !w) return HALO_ERR_NULL;
  if (io_type != HALO_F32 && io_type != HALO_BF16) return HALO_ERR_DTYPE;
  if (q_type == HALO_I8) {
    if (grad_q_type != HALO_I8) return HALO_ERR_DTYPE;
  } else if (q_type == HALO_E4M3) {
    if (grad_q_type != HALO_E5M2 && grad_q_type != HALO_E4M3) return HALO_ERR_DTYPE;
  } else {
    return HALO_ERR_DTYPE;
  }
  if (!layer_dims_ok(m, n, k) || m == 0 || n == 0 || k == 0) return HALO_ERR_SHAPE;
  if (!valid_block(block)) return HALO_ERR_BLOCK;
  const int64_t nq = contraction_len(n, block), mq = contraction_len(m, block);
  if (n % 8 != 0 || k % 8 != 0) return HALO_ERR_SHAPE;
  const bool sr_dy = opts && opts->grad_rounding == HALO_ROUND_STOCHASTIC;
  if (dx && !rows_len_ok(nq, block, rot_type == HALO_BF16, sr_dy)) return HALO_ERR_SHAPE;
  if (!operand_fits(m, nq, nq) || !operand_fits(k, nq, nq) || !operand_fits(n, mq, mq) ||
      !operand_fits(k, mq, mq))
    return HALO_ERR_SHAPE;
  if (opts && (opts->grad_rounding != HALO_ROUND_NEAREST_EVEN &&
               opts->grad_rounding != HALO_ROUND_STOCHASTIC))
    return HALO_ERR_OPTION;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(w)) return HALO_ERR_ALIGN;
  if ((dx && !aligned16(dx)) || (dw && !aligned16(dw))) return HALO_ERR_ALIGN;
  if (opts && (check_signs(opts->signs_n) != HALO_OK || check_signs(opts->signs_m) != HALO_OK))
    return HALO_ERR_ALIGN;
  return HALO_OK;
}

// The activation whose gradient the backward's dY passes take in (fused into their loads).
struct ActGrad {
  const void* z = nullptr;
  int act = 0;
  void* db = nullptr;    // bf16 [n] or NULL
  float* part = nullptr; // scratch of its partial sums
};

// Whether the backward forms dz = dy act'(z) inside its rotation passes: the one-launch batch of
// bf16 passes, both products, nearest rounding.
bool act_fused_ok(halo_dtype io_type, int64_t m, int64_t n, int64_t k, int32_t block, bool dx,
                  bool dw, bool stochastic) {
  const int64_t nq = contraction_len(n, block), mq = contraction_len(m, block);
  const WsPlan p = plan_ws(m, n, k, 1, block);
  return dx && dw && io_type == HALO_BF16 && fq_act_block_ok(block) &&
         !stochastic &&
         fq_rows2_supported(nq, block) && fq_cols2_supported(nq, k, block, 1, false, p.scr_w) &&
         fq_cols2_supported(mq, n, block, 1, false, p.scr_dy) &&
         fq_cols2_supported(mq, k, block, 1, false, p.scr_x) &&
         act_grad_parts(m, n) >= (fq_act_parts(mq, block) > 1 ? fq_act_parts(mq, block) : 1);
}

// Workspace of a layer backward with its activation: the layer's, then a stored dz (where the
// rotation passes do not form it) and the bias gradient's partial rows.
struct ActBwdWs {
  bool fused;
  size_t dz, part, total;  // byte offsets, and the whole
};

ActBwdWs act_bwd_ws(halo_dtype io_type, int64_t m, int64_t n, int64_t k, int32_t block, bool act,
                    bool dx, bool dw, bool db, bool stochastic) {
  ActBwdWs w{};
  w.fused = act && act_fused_ok(io_type, m, n, k, block, dx, dw, stochastic);
  w.dz = plan_ws(m, n, k, 1, block).total;
  w.part = w.dz + (act && !w.fused ? round256((size_t)m * n * 4) : 0);
  w.total = w.part + (db ? round256((size_t)act_grad_parts(m, n) * n * 4) : 0);
  return w;
}

// The layer backward on validated arguments: the rotation passes of dY (of type dy_type), W and X
// (io_type), then the products.  ws holds plan_ws(m, n, k, 1, block).total bytes.
// act: NULL, or the activation dY's passes take in (act_fused_ok).
halo_status run_bwd(const void* dy, halo_dtype dy_type, const void* x, const void* w,
                    halo_dtype io_type, int64_t m, int64_t n, int64_t k, int32_t block,
                    halo_dtype q_type, halo_dtype grad_q_type, void* dx, void* dw,
                    const halo_linear_opts* opts, void* ws, hipStream_t st,
                    const ActGrad* act = nullptr) {
  const WsPlan p = plan_ws(m, n, k, 1, block);
  const int64_t nq = contraction_len(n, block), mq = contraction_len(m, block);
  char* base = static_cast<char*>(ws);
  char* scr = base + p.scratch_off;
  void* scr_w = scr;
  void* scr_dy = scr + p.scr_w;
  void* scr_x = scr + p.scr_w + p.scr_dy;
  const int inb = io_type == HALO_BF16 ? 1 : 0, inb_dy = dy_type == HALO_BF16 ? 1 : 0;
  halo_status s = HALO_OK;

  // pass options: the signs along each contraction dimension; the dY codes' rounding (its
  // columns pass draws at counter word 3 ^ 2^31)
  PassOpts on, om, gn, gm;
  if (opts) {
    on.signs = gn.signs = opts->signs_n;
    om.signs = gm.signs = opts->signs_m;
    gn.sr = gm.sr = opts->grad_rounding == HALO_ROUND_STOCHASTIC ? 1 : 0;
    gn.key0 = gm.key0 = opts->seed[0];
    gn.key1 = gm.key1 = opts->seed[1];
    gn.ctr2 = gm.ctr2 = opts->counter[0];
    gn.ctr3 = opts->counter[1];
    gm.ctr3 = opts->counter[1] ^ 0x80000000u;
    on.polls = om.polls = gn.polls = gm.polls = opts->exchange_polls;
  }
  void* qdy = base + p.off[0];
  float* sdy = reinterpret_cast<float*>(base + p.off[1]);
  void* qwt = base + p.off[2];
  float* swt = reinterpret_cast<float*>(base + p.off[3]);
  void* qdyt = base + p.off[4];
  float* sdyt = reinterpret_cast<float*>(base + p.off[5]);
  void* qxt = base + p.off[6];
  float* sxt = reinterpret_cast<float*>(base + p.off[7]);
  // dX = dY W: rows of dY and columns of W along n; dW = dY^T X: columns of dY and X along m
  FqArgs rows = make_fq(dy, m, n, n, HALO_ALONG_ROWS, block, grad_q_type, qdy, nq, sdy, gn, nq);
  const FqArgs cw = make_fq(w, n, k, k, HALO_ALONG_COLS, block, q_type, qwt, nq, swt, on, nq);
  FqArgs cdy = make_fq(dy, m, n, n, HALO_ALONG_COLS, block, grad_q_type, qdyt, mq, sdyt, gm, mq);
  const FqArgs cx = make_fq(x, m, k, k, HALO_ALONG_COLS, block, q_type, qxt, mq, sxt, om, mq);

  const int64_t db_parts = act ? fq_act_parts(mq, block) : 0;
  if (act) {
    rows.z = cdy.z = static_cast<const uint16_t*>(act->z);
    rows.act = cdy.act = act->act;
    if (act->db && db_parts == 1) cdy.db = static_cast<uint16_t*>(act->db);
    if (act->db && db_parts > 1) cdy.db_part = act->part;
  }

  // the single-read column passes need their scratch cleared: folded into the first kernel
  // when that is a rows pass, else one fill
  bool zero_pending = p.scratch_bytes > 0;
  auto clear_scratch = [&]() {
    if (!zero_pending || s != HALO_OK) return;
    s = from_hip(launch_fill_zero(reinterpret_cast<float*>(scr), (int64_t)(p.scratch_bytes / 4), st));
    zero_pending = false;
  };
  // one column pass: single-read when covered (its scratch already clear), else two reads
  auto cols_pass = [&](const FqArgs& a, halo_dtype at, halo_dtype qt, void* sws, size_t sbytes) {
    if (s != HALO_OK) return;
    const int ib = at == HALO_BF16 ? 1 : 0;
    if (fq_cols2_supported(a.len, a.nvec, block, ib, a.sr != 0, sbytes))
      s = from_hip(launch_fq_cols2_pair(a, sws, nullptr, nullptr, ib, qt_index(qt), 1, st));
    else
      s = run_fa(a, at, HALO_ALONG_COLS, qt, nullptr, 0, st);
  };
  // the rows pass of dY, clearing the scratch as a side job when it runs as the wave kernel
  auto rows_pass = [&]() {
    if (s != HALO_OK) return;
    if (fq_rows2_supported(nq, block) && (inb_dy || !rows.sr)) {
      FqPair pp{};
      pp.p0 = rows;
      if (zero_pending) {
        pp.zero = reinterpret_cast<uint32_t*>(scr);
        pp.nzero = (int64_t)(p.scratch_bytes / 4);
        zero_pending = false;
      }
      s = from_hip(act ? launch_fq_rows2_act(pp, qt_index(grad_q_type), st)
                       : launch_fq_rows2_pair(pp, inb_dy, qt_index(grad_q_type), st));
    } else {
      s = run_fa(rows, dy_type, HALO_ALONG_ROWS, grad_q_type, nullptr, 0, st);
    }
  };
  const int qg = qt_index(grad_q_type), qw = qt_index(q_type);
  const bool pair_ok = (qg == 0 && qw == 0) || (qg == 2 && qw == 1) || (qg == 1 && qw == 1);
  if (dx && dw && inb && inb_dy && pair_ok && fq_cols2_supported(nq, k, block, 1, false, p.scr_w) &&
      fq_cols2_supported(mq, n, block, 1, cdy.sr != 0, p.scr_dy) &&
      fq_cols2_supported(mq, k, block, 1, false, p.scr_x)) {
    // every rotation pass of the backward in one launch (or two, when the dY rows are long):
    // the passes overlap on the device, then the two products
    const bool rows_in = fq_batch_rows_ok(nq);
    if (rows_in) {
      clear_scratch();
    } else {
      rows_pass();
      clear_scratch();
    }
    if (s == HALO_OK)
      s = from_hip((act ? launch_fq_batch_act : launch_fq_batch)(
          rows_in ? &rows : nullptr, cw, scr_w, cdy, scr_dy, cx, scr_x, qg, qw, st));
    if (s == HALO_OK && cdy.db_part)
      s = from_hip(launch_part_sum(cdy.db_part, db_parts, n, static_cast<uint16_t*>(act->db), st));
  } else {
    if (dx) rows_pass();
    clear_scratch();
    if (dx) cols_pass(cw, io_type, q_type, scr_w, p.scr_w);
    if (dw) {
      const bool c1 = fq_cols2_supported(mq, n, block, inb_dy, cdy.sr != 0, p.scr_dy);
      const bool c2 = fq_cols2_supported(mq, k, block, inb, cx.sr != 0, p.scr_x);
      if (s == HALO_OK && c1 && c2 && inb == inb_dy && grad_q_type == q_type && cdy.sr == cx.sr) {
        // dY and X columns in one launch
        s = from_hip(launch_fq_cols2_pair(cdy, scr_dy, &cx, scr_x, inb, qt_index(q_type), 1, st));
      } else {
        cols_pass(cdy, dy_type, grad_q_type, scr_dy, p.scr_dy);
        cols_pass(cx, io_type, q_type, scr_x, p.scr_x);
      }
    }
  }
  if (s == HALO_OK && dx && dw) {  // both products in one launch
    const GemmArgs gx{qdy, nq, qwt, nq, sdy, swt, dx, k, m, k, nq};
    const GemmArgs gw{qdyt, mq, qxt, mq, sdyt, sxt, dw, k, n, k, mq};
    const int out = io_type == HALO_F32 ? 1 : 2;
    if (grad_q_type == HALO_I8)
      s = from_hip(launch_gemm_pair(gx, &gw, 0, 0, 0, out, st));
    else
      s = from_hip(launch_gemm_pair(gx, &gw, 1, gemm_kind_fmt(grad_q_type), gemm_kind_fmt(q_type),
                                    out, st));
    return s;
  }
  if (s == HALO_OK && dx)
    s = gemm_any(qdy, grad_q_type, nq, sdy, qwt, q_type, nq, swt, m, k, nq, dx, io_type, k, st);
  if (s == HALO_OK && dw)
    s = gemm_any(qdyt, grad_q_type, mq, sdyt, qxt, q_type, mq, sxt, n, k, mq, dw, io_type, k, st);
  return s;
}

// Row operators take any stride and any alignment of whole elements.
bool aligned_to(const void* p, int e) { return (reinterpret_cast<uintptr_t>(p) & (e - 1)) == 0; }

bool norm_dims_ok(int64_t tokens, int64_t dim, int64_t groups, halo_dtype io) {
  return tokens >= 0 && tokens < kMaxDim && dim > 0 && dim <= norm_max_dim(io == HALO_BF16) &&
         groups > 0 && (tokens == 0 || groups <= tokens) && tokens % groups == 0;
}

halo_status check_distill(const void* logits, const halo_dtype& lt, int64_t ldl,
                          const int32_t* idx, int64_t ldi, const void* tlogits,
                          const halo_dtype& tt, int64_t ldt, int64_t tokens, int64_t vocab,
                          int64_t top, float temperature) {
  if (!dtype_ok(lt) || !dtype_ok(tt)) return HALO_ERR_DTYPE;
  if ((lt != HALO_F32 && lt != HALO_BF16) || (tt != HALO_F32 && tt != HALO_BF16))
    return HALO_ERR_DTYPE;
  if (tokens < 0 || tokens >= kMaxDim || vocab <= 0 || vocab >= kMaxDim || top <= 0 ||
      top > kDistillMaxTop)
    return HALO_ERR_SHAPE;
  if (ldl < vocab || ldi < top || ldt < top) return HALO_ERR_SHAPE;
  if (!(temperature > 0.f) || std::isinf(temperature) || std::isinf(1.f / temperature))
    return HALO_ERR_OPTION;
  if (tokens > 0 && (!logits || !idx || !tlogits)) return HALO_ERR_NULL;
  if (!aligned_to(logits, esize(lt)) || !aligned_to(idx, 4) || !aligned_to(tlogits, esize(tt)))
    return HALO_ERR_ALIGN;
  return HALO_OK;
}

DistillArgs make_distill(const void* logits, int64_t ldl, const int32_t* idx, int64_t ldi,
                         const void* tlogits, halo_dtype tt, int64_t ldt, int64_t tokens,
                         int64_t vocab, int64_t top, float temperature) {
  DistillArgs a{};
  a.logits = logits;
  a.idx = idx;
  a.tlogits = tlogits;
  a.ldl = ldl;
  a.ldi = ldi;
  a.ldt = ldt;
  a.tokens = tokens;
  a.vocab = (int)vocab;
  a.top = (int)top;
  a.t_bf16 = tt == HALO_BF16 ? 1 : 0;
  a.tau = temperature;
  a.inv_tau = 1.f / temperature;
  return a;
}

}  // namespace

extern "C" {

halo_status halo_mfma_rate_probe(int32_t kind, int32_t iters, int64_t* ops, void* stream) {
  if (!ops) return HALO_ERR_NULL;
  if (kind < 0 || kind > 2 || iters < 2 || iters > (1 << 20)) return HALO_ERR_SHAPE;
  const hipError_t e = launch_mfma_probe(kind, iters, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return HALO_ERR_HIP;
  *ops = mfma_probe_ops(kind, iters);
  return HALO_OK;
}

const char* halo_status_str(halo_status s) {
  if (!enum_in(s, HALO_OK, HALO_ERR_OPTION)) return "unknown status";
  switch (s) {
    case HALO_OK: return "ok";
    case HALO_ERR_NULL: return "a required pointer is NULL";
    case HALO_ERR_SHAPE: return "unsupported or inconsistent sizes";
    case HALO_ERR_BLOCK: return "block must be a power of two in [1, 4096]";
    case HALO_ERR_DTYPE: return "unsupported element type";
    case HALO_ERR_ALIGN: return "pointer or leading dimension not aligned (16 bytes; row operators: the element)";
    case HALO_ERR_WORKSPACE: return "workspace missing or too small";
    case HALO_ERR_HIP: return "HIP launch failed";
    case HALO_ERR_OPTION: return "invalid option (rounding mode, activation, eps or temperature)";
  }
  return "unknown status";
}

// ---- block norms ------------------------------------------------------------------------

size_t halo_block_norm_bwd_workspace_bytes(int64_t tokens, int64_t dim, int64_t groups,
                                           halo_dtype io_type) {
  if (!dtype_ok(io_type) || (io_type != HALO_F32 && io_type != HALO_BF16)) return 0;
  if (tokens <= 0 || dim <= 0 || groups <= 0 || tokens >= kMaxDim || tokens % groups != 0 ||
      dim > norm_max_dim(io_type == HALO_BF16))
    return 0;
  return norm_bwd_ws_bytes(tokens, dim, tokens / groups, io_type == HALO_BF16, true, true, true);
}

halo_status halo_block_norm_fwd(const void* r, int64_t ldr, const void* y, int64_t ldy,
                                const void* gate, int64_t ldg, int64_t groups,
                                const void* post_weight, const void* pre_weight,
                                halo_dtype io_type, int64_t tokens, int64_t dim, float scale,
                                float eps, void* r_out, int64_t ldr_out, void* h, int64_t ldh,
                                float* rstd_post, float* rstd_pre, void* stream) {
  if (!dtype_ok(io_type)) return HALO_ERR_DTYPE;
  if (io_type != HALO_F32 && io_type != HALO_BF16) return HALO_ERR_DTYPE;
  if (!norm_dims_ok(tokens, dim, groups, io_type)) return HALO_ERR_SHAPE;
  if (!(eps >= 0.f)) return HALO_ERR_OPTION;
  if (tokens == 0) return HALO_OK;  // empty tensors may come with NULL pointers
  if ((gate || post_weight || r_out || rstd_post) && !y) return HALO_ERR_NULL;
  if (rstd_post && !post_weight) return HALO_ERR_NULL;
  if ((h || rstd_pre) && !pre_weight) return HALO_ERR_NULL;
  if (!r || (y && !r_out) || (pre_weight && !h) || (!y && !pre_weight)) return HALO_ERR_NULL;
  if (ldr < dim || (y && (ldy < dim || ldr_out < dim)) || (pre_weight && ldh < dim) ||
      (gate && ldg < dim))
    return HALO_ERR_SHAPE;
  const int e = esize(io_type);
  if (!aligned_to(r, e) || !aligned_to(y, e) || !aligned_to(gate, e) ||
      !aligned_to(post_weight, e) || !aligned_to(pre_weight, e) || !aligned_to(r_out, e) ||
      !aligned_to(h, e) || !aligned_to(rstd_post, 4) || !aligned_to(rstd_pre, 4))
    return HALO_ERR_ALIGN;
  NormFwdArgs a{};
  a.r = r; a.y = y; a.gate = gate; a.post = post_weight; a.pre = pre_weight;
  a.r_out = r_out; a.h = h; a.rstd_post = rstd_post; a.rstd_pre = rstd_pre;
  a.ldr = ldr; a.ldy = ldy; a.ldg = ldg; a.ldro = ldr_out; a.ldh = ldh;
  a.tokens = tokens; a.group_len = tokens / groups; a.dim = (int)dim;
  a.scale = scale; a.eps = eps; a.inv_dim = (float)(1.0 / (double)dim);
  return from_hip(launch_norm_fwd(a, io_type == HALO_BF16 ? 1 : 0, (hipStream_t)stream));
}

halo_status halo_block_norm_bwd(const void* dr_out, int64_t lddr_out, const void* dh,
                                int64_t lddh, const void* r_out, int64_t ldr_out, const void* y,
                                int64_t ldy, const void* gate, int64_t ldg, int64_t groups,
                                const void* post_weight, const void* pre_weight,
                                const float* rstd_post, const float* rstd_pre,
                                halo_dtype io_type, int64_t tokens, int64_t dim, float scale,
                                void* dr, int64_t lddr, void* dy, int64_t lddy, void* dgate,
                                void* dpost_weight, void* dpre_weight, void* ws,
                                size_t ws_bytes, void* stream) {
  if (!dtype_ok(io_type)) return HALO_ERR_DTYPE;
  if (io_type != HALO_F32 && io_type != HALO_BF16) return HALO_ERR_DTYPE;
  if (!norm_dims_ok(tokens, dim, groups, io_type) || tokens == 0) return HALO_ERR_SHAPE;
  if (!dr || (!dr_out && !dh)) return HALO_ERR_NULL;
  if (pre_weight ? (!dh || !r_out || !rstd_pre) : (dh || dpre_weight)) return HALO_ERR_NULL;
  if ((gate || post_weight || dy || dgate || dpost_weight) && !y) return HALO_ERR_NULL;
  if (y && !dy) return HALO_ERR_NULL;
  if (post_weight ? !rstd_post : dpost_weight != nullptr) return HALO_ERR_NULL;
  if (dgate && !gate) return HALO_ERR_NULL;
  if ((dr_out && lddr_out < dim) || (pre_weight && (lddh < dim || ldr_out < dim)) ||
      (y && (ldy < dim || lddy < dim)) || (gate && ldg < dim) || lddr < dim)
    return HALO_ERR_SHAPE;
  const int e = esize(io_type);
  if (!aligned_to(dr_out, e) || !aligned_to(dh, e) || !aligned_to(r_out, e) ||
      !aligned_to(y, e) || !aligned_to(gate, e) || !aligned_to(post_weight, e) ||
      !aligned_to(pre_weight, e) || !aligned_to(rstd_post, 4) || !aligned_to(rstd_pre, 4) ||
      !aligned_to(dr, e) || !aligned_to(dy, e) || !aligned_to(dgate, e) ||
      !aligned_to(dpost_weight, e) || !aligned_to(dpre_weight, e))
    return HALO_ERR_ALIGN;
  const size_t need =
      norm_bwd_ws_bytes(tokens, dim, tokens / groups, io_type == HALO_BF16,
                        dpost_weight != nullptr, dpre_weight != nullptr, dgate != nullptr);
  if (need > 0 && (!ws || ws_bytes < need)) return HALO_ERR_WORKSPACE;
  if (!aligned16(ws)) return HALO_ERR_ALIGN;
  NormBwdArgs a{};
  a.dr_out = dr_out; a.dh = dh; a.r_out = r_out; a.y = y;
  a.gate = gate; a.post = post_weight; a.pre = pre_weight;
  a.rstd_post = rstd_post; a.rstd_pre = rstd_pre;
  a.dr = dr; a.dy = dy; a.dgate = dgate; a.dpost = dpost_weight; a.dpre = dpre_weight;
  a.lddro = lddr_out; a.lddh = lddh; a.ldro = ldr_out; a.ldy = ldy; a.ldg = ldg;
  a.lddr = lddr; a.lddy = lddy;
  a.tokens = tokens; a.group_len = tokens / groups; a.dim = (int)dim;
  a.scale = scale; a.inv_dim = (float)(1.0 / (double)dim);
  return from_hip(launch_norm_bwd(a, io_type == HALO_BF16 ? 1 : 0, ws, (hipStream_t)stream));
}

// ---- distillation -----------------------------------------------------------------------

halo_status halo_distill_fwd(const void* logits, halo_dtype logits_type, int64_t ldl,
                             const int32_t* idx, int64_t ldi, const void* tlogits,
                             halo_dtype t_type, int64_t ldt, int64_t tokens, int64_t vocab,
                             int64_t top, float temperature, float* loss, float* lse,
                             void* stream) {
  halo_status s = check_distill(logits, logits_type, ldl, idx, ldi, tlogits, t_type, ldt, tokens,
                                vocab, top, temperature);
  if (s != HALO_OK) return s;
  if (tokens > 0 && !loss) return HALO_ERR_NULL;
  if (!aligned_to(loss, 4) || !aligned_to(lse, 4)) return HALO_ERR_ALIGN;
  if (tokens == 0) return HALO_OK;
  DistillArgs a = make_distill(logits, ldl, idx, ldi, tlogits, t_type, ldt, tokens, vocab, top,
                               temperature);
  a.loss = loss;
  a.lse = lse;
  return from_hip(launch_distill(a, logits_type == HALO_BF16 ? 1 : 0, (hipStream_t)stream));
}

halo_status halo_distill_bwd(const float* dloss, const void* logits, halo_dtype logits_type,
                             int64_t ldl, const float* lse, const int32_t* idx, int64_t ldi,
                             const void* tlogits, halo_dtype t_type, int64_t ldt, int64_t tokens,
                             int64_t vocab, int64_t top, float temperature, void* dlogits,
                             int64_t ldd, void* stream) {
  halo_status s = check_distill(logits, logits_type, ldl, idx, ldi, tlogits, t_type, ldt, tokens,
                                vocab, top, temperature);
  if (s != HALO_OK) return s;
  if (tokens > 0 && (!dloss || !lse || !dlogits)) return HALO_ERR_NULL;
  if (ldd < vocab || (dlogits == logits && ldd != ldl)) return HALO_ERR_SHAPE;
  if (!aligned_to(dloss, 4) || !aligned_to(lse, 4) || !aligned_to(dlogits, esize(logits_type)))
    return HALO_ERR_ALIGN;
  if (tokens == 0) return HALO_OK;
  DistillArgs a = make_distill(logits, ldl, idx, ldi, tlogits, t_type, ldt, tokens, vocab, top,
                               temperature);
  a.dloss = dloss;
  a.lse_in = lse;
  a.dlogits = dlogits;
  a.ldd = ldd;
  return from_hip(launch_distill(a, logits_type == HALO_BF16 ? 1 : 0, (hipStream_t)stream));
}

halo_status halo_distill_fwd_bwd(const void* logits, halo_dtype logits_type, int64_t ldl,
                                 const int32_t* idx, int64_t ldi, const void* tlogits,
                                 halo_dtype t_type, int64_t ldt, const float* dloss,
                                 int64_t tokens, int64_t vocab, int64_t top, float temperature,
                                 float* loss, float* lse, void* dlogits, int64_t ldd,
                                 void* stream) {
  halo_status s = check_distill(logits, logits_type, ldl, idx, ldi, tlogits, t_type, ldt, tokens,
                                vocab, top, temperature);
  if (s != HALO_OK) return s;
  if (tokens > 0 && (!dloss || !loss || !dlogits)) return HALO_ERR_NULL;
  if (ldd < vocab || (dlogits == logits && ldd != ldl)) return HALO_ERR_SHAPE;
  if (!aligned_to(dloss, 4) || !aligned_to(loss, 4) || !aligned_to(lse, 4) ||
      !aligned_to(dlogits, esize(logits_type)))
    return HALO_ERR_ALIGN;
  if (tokens == 0) return HALO_OK;
  DistillArgs a = make_distill(logits, ldl, idx, ldi, tlogits, t_type, ldt, tokens, vocab, top,
                               temperature);
  a.dloss = dloss;
  a.loss = loss;
  a.lse = lse;
  a.dlogits = dlogits;
  a.ldd = ldd;
  return from_hip(launch_distill(a, logits_type == HALO_BF16 ? 1 : 0, (hipStream_t)stream));
}

size_t halo_fwht_quant_workspace_bytes(int64_t rows, int64_t cols, halo_axis axis,
                                       int32_t block, halo_dtype x_type) {
  if (!axis_ok(axis) || !dtype_ok(x_type)) return 0;
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim || !valid_block(block))
    return 0;
  if (axis != HALO_ALONG_COLS) return 0;
  return fq_ws_bytes_len(padded_len(rows, block), cols, axis, block);
}

halo_status halo_fwht_quant_ex(const void* x, halo_dtype x_type, int64_t rows, int64_t cols,
                               int64_t ldx, halo_axis axis, int32_t block, halo_dtype q_type,
                               void* q, int64_t ldq, float* scale, const halo_quant_opts* opts,
                               void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(x_type) || !dtype_ok(q_type)) return HALO_ERR_DTYPE;
  if (!axis_ok(axis)) return HALO_ERR_SHAPE;
  halo_status s = check_fq(x, x_type, rows, cols, ldx, axis, block, q_type, q, ldq, scale, opts);
  if (s != HALO_OK) return s;
  if (ws && !aligned16(ws)) return HALO_ERR_ALIGN;
  return run_fq(x, x_type, rows, cols, ldx, axis, block, q_type, q, ldq, scale, ws, ws_bytes,
                (hipStream_t)stream, pass_opts(opts));
}

halo_status halo_fwht_quant(const void* x, halo_dtype x_type, int64_t rows, int64_t cols,
                            int64_t ldx, halo_axis axis, int32_t block, halo_dtype q_type,
                            void* q, int64_t ldq, float* scale, void* ws, size_t ws_bytes,
                            void* stream) {
  if (!dtype_ok(x_type) || !dtype_ok(q_type)) return HALO_ERR_DTYPE;
  if (!axis_ok(axis)) return HALO_ERR_SHAPE;
  return halo_fwht_quant_ex(x, x_type, rows, cols, ldx, axis, block, q_type, q, ldq, scale,
                            nullptr, ws, ws_bytes, stream);
}

halo_status halo_fwht_quant_noalloc(const void* x, halo_dtype x_type, int64_t rows, int64_t cols,
                                    int64_t ldx, halo_axis axis, int32_t block,
                                    halo_dtype q_type, void* q, int64_t ldq, float* scale,
                                    const halo_quant_opts* opts, void* stream) {
  if (!dtype_ok(x_type) || !dtype_ok(q_type)) return HALO_ERR_DTYPE;
  if (!axis_ok(axis)) return HALO_ERR_SHAPE;
  halo_status s = check_fq(x, x_type, rows, cols, ldx, axis, block, q_type, q, ldq, scale, opts);
  if (s != HALO_OK) return s;
  const size_t need = halo_fwht_quant_workspace_bytes(rows, cols, axis, block, x_type);
  if (need > HALO_NOALLOC_SCRATCH_BYTES) return HALO_ERR_WORKSPACE;
  void* ws = nullptr;
  if (need > 0 && !(ws = noalloc_scratch())) return HALO_ERR_HIP;
  return run_fq(x, x_type, rows, cols, ldx, axis, block, q_type, q, ldq, scale, ws,
                ws ? HALO_NOALLOC_SCRATCH_BYTES : 0, (hipStream_t)stream, pass_opts(opts));
}

size_t halo_fwht_quant_dual_workspace_bytes(int64_t rows, int64_t cols, int32_t block,
                                            halo_dtype x_type) {
  if (!dtype_ok(x_type)) return 0;
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim || !valid_block(block))
    return 0;
  // the single-read launch's scratch, or, for shapes it does not take, the columns pass's
  const size_t dual = fq_dual_ws_bytes(rows, cols, block, x_type == HALO_BF16 ? 1 : 0);
  const size_t cols_ws = fq_ws_bytes_len(padded_len(rows, block), cols, HALO_ALONG_COLS, block);
  return dual > cols_ws ? dual : cols_ws;
}

halo_status halo_fwht_quant_dual(const void* x, halo_dtype x_type, int64_t rows, int64_t cols,
                                 int64_t ldx, int32_t block, halo_dtype q_type, void* qr,
                                 int64_t ldqr, float* scale_r, void* qc, int64_t ldqc,
                                 float* scale_c, const halo_quant_opts* row_opts,
                                 const halo_quant_opts* col_opts, void* ws, size_t ws_bytes,
                                 void* stream) {
  if (!dtype_ok(x_type) || !dtype_ok(q_type)) return HALO_ERR_DTYPE;
  halo_status s = check_fq(x, x_type, rows, cols, ldx, HALO_ALONG_ROWS, block, q_type, qr, ldqr,
                           scale_r, row_opts);
  if (s != HALO_OK) return s;
  s = check_fq(x, x_type, rows, cols, ldx, HALO_ALONG_COLS, block, q_type, qc, ldqc, scale_c,
               col_opts);
  if (s != HALO_OK) return s;
  if (ws && !aligned16(ws)) return HALO_ERR_ALIGN;
  const hipStream_t st = (hipStream_t)stream;
  const FqArgs ar = make_fq(x, rows, cols, ldx, HALO_ALONG_ROWS, block, q_type, qr, ldqr, scale_r,
                            pass_opts(row_opts));
  const FqArgs ac = make_fq(x, rows, cols, ldx, HALO_ALONG_COLS, block, q_type, qc, ldqc, scale_c,
                            pass_opts(col_opts));
  const int inb = x_type == HALO_BF16 ? 1 : 0;
  if (ws && fq_dual_supported(rows, cols, block, inb, qt_index(q_type), ar.sr != 0, ac.sr != 0,
                              ws_bytes))
    return from_hip(launch_fq_dual(ar, ac, ws, qt_index(q_type), 0, st));
  s = run_fa(ar, x_type, HALO_ALONG_ROWS, q_type, nullptr, 0, st);
  if (s != HALO_OK) return s;
  return run_fa(ac, x_type, HALO_ALONG_COLS, q_type, ws, ws ? ws_bytes : 0, st);
}

halo_status halo_gemm_i8(const int8_t* a, int64_t lda, const float* sa, const int8_t* b,
                         int64_t ldb, const float* sb, int64_t m, int64_t n, int64_t k, void* c,
                         halo_dtype c_type, int64_t ldc, void* stream) {
  if (!dtype_ok(c_type)) return HALO_ERR_DTYPE;
  if (c_type != HALO_I32 && c_type != HALO_F32 && c_type != HALO_BF16) return HALO_ERR_DTYPE;
  halo_status s = check_gemm(a, lda, b, ldb, m, n, k, c, c_type, ldc, sa, sb, 16);
  if (s != HALO_OK) return s;
  if (c_type != HALO_I32 && (!aligned16(sa) || !aligned16(sb))) return HALO_ERR_ALIGN;
  return gemm_any(a, HALO_I8, lda, sa, b, HALO_I8, ldb, sb, m, n, k, c, c_type, ldc,
                  (hipStream_t)stream);
}

halo_status halo_gemm_fp8(const void* a, halo_dtype a_type, int64_t lda, const float* sa,
                          const void* b, halo_dtype b_type, int64_t ldb, const float* sb,
                          int64_t m, int64_t n, int64_t k, void* c, halo_dtype c_type,
                          int64_t ldc, void* stream) {
  if (!dtype_ok(a_type) || !dtype_ok(b_type) || !dtype_ok(c_type)) return HALO_ERR_DTYPE;
  if ((a_type != HALO_E4M3 && a_type != HALO_E5M2) || (b_type != HALO_E4M3 && b_type != HALO_E5M2))
    return HALO_ERR_DTYPE;
  if (c_type != HALO_F32 && c_type != HALO_BF16) return HALO_ERR_DTYPE;
  halo_status s = check_gemm(a, lda, b, ldb, m, n, k, c, c_type, ldc, sa, sb, 32);
  if (s != HALO_OK) return s;
  if (!aligned16(sa) || !aligned16(sb)) return HALO_ERR_ALIGN;
  return gemm_any(a, a_type, lda, sa, b, b_type, ldb, sb, m, n, k, c, c_type, ldc,
                  (hipStream_t)stream);
}


size_t halo_linear_workspace_bytes_ex(int64_t m, int64_t n, int64_t k, int32_t block,
                                      halo_dtype q_type, int backward) {
  if (!dtype_ok(q_type)) return 0;
  if (!layer_dims_ok(m, n, k) || !valid_block(block)) return 0;
  if (q_type != HALO_I8 && q_type != HALO_E4M3) return 0;
  return plan_ws(m, n, k, backward ? 1 : 0, block).total;
}

size_t halo_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, halo_dtype q_type,
                                   int backward) {
  if (!dtype_ok(q_type)) return 0;
  size_t most = 0;
  for (int32_t b = 1; b <= 4096; b *= 2) {
    const size_t t = halo_linear_workspace_bytes_ex(m, n, k, b, q_type, backward);
    if (t > most) most = t;
  }
  return most;
}

halo_status halo_linear_fwd_ex(const void* x, const void* w, halo_dtype io_type, int64_t m,
                               int64_t n, int64_t k, int32_t block, halo_dtype q_type, void* y,
                               halo_dtype y_type, const halo_linear_opts* opts, void* ws,
                               size_t ws_bytes, void* stream) {
  if (!dtype_ok(io_type) || !dtype_ok(q_type) || !dtype_ok(y_type)) return HALO_ERR_DTYPE;
  const halo_status s = check_fwd(x, w, io_type, m, n, k, block, q_type, y, y_type, opts);
  if (s != HALO_OK) return s;
  if (!ws || ws_bytes < plan_ws(m, n, k, 0, block).total) return HALO_ERR_WORKSPACE;
  if (!aligned16(ws)) return HALO_ERR_ALIGN;
  return run_fwd(x, w, io_type, m, n, k, block, q_type, y, y_type, nullptr, opts, ws,
                 (hipStream_t)stream);
}

halo_status halo_linear_fwd(const void* x, const void* w, halo_dtype io_type, int64_t m,
                            int64_t n, int64_t k, int32_t block, halo_dtype q_type, void* y,
                            halo_dtype y_type, void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(io_type) || !dtype_ok(q_type) || !dtype_ok(y_type)) return HALO_ERR_DTYPE;
  return halo_linear_fwd_ex(x, w, io_type, m, n, k, block, q_type, y, y_type, nullptr, ws,
                            ws_bytes, stream);
}

halo_status halo_linear_bwd_ex(const void* dy, const void* x, const void* w, halo_dtype io_type,
                               int64_t m, int64_t n, int64_t k, int32_t block, halo_dtype q_type,
                               halo_dtype grad_q_type, void* dx, void* dw,
                               const halo_linear_opts* opts, void* ws, size_t ws_bytes,
                               void* stream) {
  if (!dtype_ok(io_type) || !dtype_ok(q_type) || !dtype_ok(grad_q_type)) return HALO_ERR_DTYPE;
  const halo_status s = check_bwd(dy, io_type, x, w, io_type, m, n, k, block, q_type, grad_q_type,
                                  dx, dw, opts);
  if (s != HALO_OK) return s;
  if (!ws || ws_bytes < plan_ws(m, n, k, 1, block).total) return HALO_ERR_WORKSPACE;
  if (!aligned16(ws)) return HALO_ERR_ALIGN;
  return run_bwd(dy, io_type, x, w, io_type, m, n, k, block, q_type, grad_q_type, dx, dw, opts, ws,
                 (hipStream_t)stream);
}

halo_status halo_linear_bwd(const void* dy, const void* x, const void* w, halo_dtype io_type,
                            int64_t m, int64_t n, int64_t k, int32_t block, halo_dtype q_type,
                            halo_dtype grad_q_type, void* dx, void* dw, void* ws,
                            size_t ws_bytes, void* stream) {
  if (!dtype_ok(io_type) || !dtype_ok(q_type) || !dtype_ok(grad_q_type)) return HALO_ERR_DTYPE;
  return halo_linear_bwd_ex(dy, x, w, io_type, m, n, k, block, q_type, grad_q_type, dx, dw,
                            nullptr, ws, ws_bytes, stream);
}

// ---- the layer with its epilogue ------------------------------------------------------------

halo_status halo_linear_act_fwd(const void* x, const void* w, halo_dtype io_type, int64_t m,
                                int64_t n, int64_t k, int32_t block, halo_dtype q_type, void* y,
                                halo_dtype y_type, const halo_epilogue* ep,
                                const halo_linear_opts* opts, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!dtype_ok(io_type) || !dtype_ok(q_type) || !dtype_ok(y_type)) return HALO_ERR_DTYPE;
  halo_status s = check_fwd(x, w, io_type, m, n, k, block, q_type, y, y_type, opts);
  if (s == HALO_OK) s = check_epilogue(ep);
  if (s != HALO_OK) return s;
  if (!ws || ws_bytes < plan_ws(m, n, k, 0, block).total) return HALO_ERR_WORKSPACE;
  if (!aligned16(ws)) return HALO_ERR_ALIGN;
  const halo_epilogue none{};
  return run_fwd(x, w, io_type, m, n, k, block, q_type, y, y_type, ep ? ep : &none, opts, ws,
                 (hipStream_t)stream);
}

size_t halo_linear_act_q_workspace_bytes(int64_t m, int64_t k, int32_t block) {
  if (!layer_dims_ok(m, 0, k) || !valid_block(block)) return 0;
  if (skinny_fused_ok(m, contraction_len(k, block), block)) return 0;
  return round256((size_t)m * contraction_len(k, block)) + round256((size_t)m * 4);
}

halo_status halo_linear_act_q(const void* x, halo_dtype io_type, const void* qw, halo_dtype q_type,
                              const float* sw, int64_t m, int64_t n, int64_t k, int32_t block,
                              void* y, halo_dtype y_type, const halo_epilogue* ep,
                              const uint32_t* signs_k, void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(io_type) || !dtype_ok(q_type) || !dtype_ok(y_type)) return HALO_ERR_DTYPE;
  halo_status s = check_fwd(x, qw, io_type, m, n, k, block, q_type, y, y_type, nullptr);
  if (s == HALO_OK) s = check_epilogue(ep);
  if (s != HALO_OK) return s;
  const int64_t kq = contraction_len(k, block);
  if (kq != padded_len(k, block)) return HALO_ERR_SHAPE;
  if (n > 0 && !sw) return HALO_ERR_NULL;
  if (!aligned16(sw) || check_signs(signs_k) != HALO_OK) return HALO_ERR_ALIGN;
  if (m == 0 || n == 0) return HALO_OK;
  const size_t need = halo_linear_act_q_workspace_bytes(m, k, block);
  if (need > 0 && (!ws || ws_bytes < need)) return HALO_ERR_WORKSPACE;
  if (!aligned16(ws)) return HALO_ERR_ALIGN;
  const hipStream_t st = (hipStream_t)stream;
  char* base = static_cast<char*>(ws);
  float* sx = reinterpret_cast<float*>(need > 0 ? base + round256((size_t)m * kq) : nullptr);
  PassOpts po;
  po.signs = signs_k;
  const FqArgs ax = make_fq(x, m, k, k, HALO_ALONG_ROWS, block, q_type, base, kq, sx, po, kq);
  const halo_epilogue none{};
  if (need == 0) {
    const GemmArgs g = act_args(nullptr, kq, nullptr, qw, kq, sw, m, n, kq, y, ep ? ep : &none);
    return from_hip(launch_skinny_fused(g, ax, io_type == HALO_BF16 ? 1 : 0, q_type == HALO_I8 ? 0 : 1,
                                        y_type == HALO_F32 ? 1 : 2, st));
  }
  s = run_fa(ax, io_type, HALO_ALONG_ROWS, q_type, nullptr, 0, st);
  if (s != HALO_OK) return s;
  return act_product(base, kq, sx, qw, kq, sw, m, n, kq, q_type, y, y_type, ep ? ep : &none, st);
}

size_t halo_linear_act_bwd_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t block,
                                           halo_dtype q_type) {
  const size_t layer = halo_linear_workspace_bytes_ex(m, n, k, block, q_type, 1);
  if (layer == 0) return 0;
  return layer + round256((size_t)m * n * 4) + round256((size_t)act_grad_parts(m, n) * n * 4);
}

size_t halo_linear_act_bwd_workspace_bytes_ex(int64_t m, int64_t n, int64_t k, int32_t block,
                                              halo_dtype io_type, halo_dtype q_type,
                                              halo_activation activation, int32_t gradients,
                                              halo_rounding grad_rounding) {
  if (!dtype_ok(io_type) || (io_type != HALO_F32 && io_type != HALO_BF16)) return 0;
  if (!enum_in(activation, HALO_ACT_NONE, HALO_ACT_GELU_ERF)) return 0;
  if (!enum_in(grad_rounding, HALO_ROUND_NEAREST_EVEN, HALO_ROUND_STOCHASTIC)) return 0;
  if (gradients & ~(HALO_GRAD_DX | HALO_GRAD_DW | HALO_GRAD_DB)) return 0;
  if (halo_linear_workspace_bytes_ex(m, n, k, block, q_type, 1) == 0) return 0;
  return act_bwd_ws(io_type, m, n, k, block, activation != HALO_ACT_NONE, gradients & HALO_GRAD_DX,
                    gradients & HALO_GRAD_DW, gradients & HALO_GRAD_DB,
                    grad_rounding == HALO_ROUND_STOCHASTIC)
      .total;
}

halo_status halo_linear_act_bwd(const void* dy, const void* z, halo_activation activation,
                                const void* x, const void* w, halo_dtype io_type, int64_t m,
                                int64_t n, int64_t k, int32_t block, halo_dtype q_type,
                                halo_dtype grad_q_type, void* dx, void* dw, void* db,
                                const halo_linear_opts* opts, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!dtype_ok(io_type) || !dtype_ok(q_type) || !dtype_ok(grad_q_type)) return HALO_ERR_DTYPE;
  if (!enum_in(activation, HALO_ACT_NONE, HALO_ACT_GELU_ERF)) return HALO_ERR_OPTION;
  const bool act = activation != HALO_ACT_NONE;
  halo_status s = check_bwd(dy, act ? HALO_F32 : io_type, x, w, io_type, m, n, k, block, q_type,
                            grad_q_type, dx, dw, opts);
  if (s != HALO_OK) return s;
  if (act && !z) return HALO_ERR_NULL;
  if (!aligned16(z) || !aligned16(db)) return HALO_ERR_ALIGN;
  const ActBwdWs wl = act_bwd_ws(io_type, m, n, k, block, act, dx, dw, db,
                                 opts && opts->grad_rounding == HALO_ROUND_STOCHASTIC);
  if (!ws || ws_bytes < wl.total) return HALO_ERR_WORKSPACE;
  if (!aligned16(ws)) return HALO_ERR_ALIGN;
  const hipStream_t st = (hipStream_t)stream;
  float* dz = reinterpret_cast<float*>(static_cast<char*>(ws) + wl.dz);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + wl.part);
  if (wl.fused) {
    ActGrad ag;
    ag.z = z;
    ag.act = (int)activation;
    ag.db = db;
    ag.part = part;
    return run_bwd(dy, io_type, x, w, io_type, m, n, k, block, q_type, grad_q_type, dx, dw, opts, ws,
                   st, &ag);
  }
  if (act || db) {
    const hipError_t e = launch_act_grad(dy, z, (int)activation, io_type == HALO_BF16 ? 1 : 0, m, n,
                                         act ? dz : nullptr, db, part, st);
    if (e != hipSuccess) return HALO_ERR_HIP;
  }
  return run_bwd(act ? dz : dy, act ? HALO_F32 : io_type, x, w, io_type, m, n, k, block, q_type,
                 grad_q_type, dx, dw, opts, ws, st);
}

}  // extern "C"
