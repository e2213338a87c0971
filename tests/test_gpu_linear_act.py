"""The layer with its epilogue (linear_act_fwd, linear_act_q, linear_act_bwd).

Forward.  The codes are those of fwht_quant (held to the oracle by its own tests), so the product
has an exact value in 64 bits.  INT8 sums are exact integers: z carries at most 5 roundings of
2^-24 of |product| + |bias| (or of a subnormal unit); FP8 sums carry the matrix core's documented bound on top.  An
activation passes an error of z on by at most its largest slope (1.13) and adds 2^-24 (16 + 4 |z|)
of |z| (exponent scaled to base 2, two units in the last place of exp and rcp, erf).  y and z are
rounded once (2^-8 for bf16).

Backward.  With no activation the products are linear_bwd's, bit for bit.  With one, they are
linear_bwd's on a dz that torch computes in 64 bits and rounds to fp32: the two dz differ by some
2^-24, which moves a code in about 2^-20 of the places by one step of absmax / 127 (about 3 % of
the rms; FP8 less), 1e-4 of the result in norm, beside the output's rounding."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I8, E4M3, E5M2 = (torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn,
                             torch.float8_e5m2)
ROUND = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24
ETA = 2.0 ** -149   # a rounding in the subnormal range, where no relative bound holds
ACTS = ["none", "relu", "silu", "gelu_tanh", "gelu_erf"]


def rnd(shape, dt, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def act64(z, act):
    if act == "none":
        return z.clone()
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu_erf":
        return z * torch.special.ndtr(z)
    return z * torch.special.expit(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))


def slope64(z, act):
    z = z.detach().clone().requires_grad_(True)
    act64(z, act).sum().backward()
    return z.grad


def kq_of(k, block):
    return H.contraction_len(k, block)


def codes(t, block, q):
    """Row codes and scales padded to the layer's contraction length."""
    kq = kq_of(t.shape[1], block)
    full = torch.zeros((t.shape[0], kq), dtype=t.dtype, device=DEV)
    full[:, :t.shape[1]] = t
    return H.fwht_quant(full, H.ROWS, block, q)


def check_fwd(x, w, block, q, act, bias, res, y, z, yt):
    (qx, sx), (qw, sw) = codes(x, block, q), codes(w, block, q)
    a, b = qx.double(), qw.double()
    s = sx.double()[:, None] * sw.double()[None, :]
    prod = (a @ b.t()) * s
    bz = bias.double() if bias is not None else torch.zeros(w.shape[0], dtype=torch.float64, device=DEV)
    ref_z = prod + bz
    err = 5 * U * (prod.abs() + bz.abs()) + 5 * ETA
    if q != I8:
        n = a.shape[1] / 8 + 2
        err = err + (2.0 ** -10 + n * U / (1 - n * U)) * (a.abs() @ b.abs().t()) * s
    if z is not None:
        bad = (z.double() - ref_z).abs() > err + ROUND[yt] * (ref_z.abs() + err)
        assert not bad.any(), ("z", int(bad.sum()))
    ref_y = act64(ref_z, act)
    err = 1.13 * err + (U * (16 + 4 * ref_z.abs()) * ref_z.abs() if act not in ("none", "relu") else 0)
    if res is not None:
        ref_y = ref_y + res.double()
        err = err + U * ref_y.abs()
    bad = (y.double() - ref_y).abs() > err + ROUND[yt] * (ref_y.abs() + err)
    assert not bad.any(), ("y", int(bad.sum()), int(torch.nonzero(bad)[0][0]))


# rows, columns, contraction, block: up to 16 rows, waves that split the contraction, 128 and 256
# tiles (64 ones: see the small tiles below), whole and ragged tiles, whole and ragged contractions
SHAPES = [(1, 8, 32, 32), (1, 264, 4096, 256), (5, 40, 96, 32), (16, 512, 1000, 8), (17, 1000, 640, 64),
          (33, 72, 2048, 1024), (64, 136, 4128, 32), (65, 200, 512, 128), (203, 520, 1376, 32),
          (700, 1000, 256, 64), (1800, 2000, 160, 32), (1800, 2000, 256, 64),
          (3800, 3848, 128, 64), (3840, 3840, 224, 32)]


@pytest.mark.parametrize("q", [I8, E4M3])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("m,n,k,block", SHAPES)
def test_forward(m, n, k, block, dt, q):
    print(f"m {m} n {n} k {k} block {block} {dt} {q}", flush=True)
    x, w = rnd((m, k), dt, 1), rnd((n, k), dt, 2, 2.0 * k ** -0.5)
    bias, res = rnd((n,), dt, 3), rnd((m, n), dt, 4)
    act = ACTS[(m + n) % 5]
    y, z = H.linear_act_fwd(x, w, block, q, bias=bias, activation=act, residual=res, want_z=True)
    check_fwd(x, w, block, q, act, bias, res, y, z, dt)
    y2 = H.linear_act_fwd(x, w, block, q, bias=bias, activation=act, residual=res)
    assert torch.equal(y, y2)
    if kq_of(k, block) == H.padded_len(k, block):
        qw, sw = H.fwht_quant(w, H.ROWS, block, q)
        z3 = torch.empty_like(z)
        y3, z3 = H.linear_act_q(x, qw, sw, block, bias=bias, activation=act, residual=res, z=z3)
        assert torch.equal(y3, y) and torch.equal(z3, z)


@pytest.mark.parametrize("m", [3, 70, 2000])
@pytest.mark.parametrize("act", ACTS)
def test_parts_of_the_epilogue(m, act):
    n, k, block = 1928, 128, 64
    x, w = rnd((m, k), BF16, 1), rnd((n, k), BF16, 2, 0.3)
    for bias, res in ((None, None), (rnd((n,), BF16, 3), None), (None, rnd((m, n), BF16, 4))):
        y = H.linear_act_fwd(x, w, block, bias=bias, activation=act, residual=res)
        check_fwd(x, w, block, I8, act, bias, res, y, None, BF16)
    if act == "none":   # the bare product is the layer's
        y = H.linear_act_fwd(x, w, block)
        assert torch.equal(y, H.linear_fwd(x, w, block))
    # fp32 output of bf16 operands; the residual may be the output
    y32 = H.linear_act_fwd(x, w, block, activation=act, y_dtype=F32)
    check_fwd(x, w, block, I8, act, None, None, y32, None, F32)
    res = rnd((m, n), BF16, 5)
    want = H.linear_act_fwd(x, w, block, activation=act, residual=res)
    got = H.linear_act_fwd(x, w, block, activation=act, residual=res, y=res)
    assert got is res and torch.equal(got, want)


@pytest.mark.parametrize("m", [2, 130])
def test_extreme_values_and_signs(m):
    n, k, block = 64, 256, 64
    x, w = rnd((m, k), BF16, 1, 300.0), rnd((n, k), BF16, 2, 300.0)   # z of 1e6: exp overflows
    x[1] = 0                                                          # a row of zero codes
    signs = H.hadamard_signs(k, 5, DEV)
    for act in ACTS:
        y, z = H.linear_act_fwd(x, w, block, activation=act, want_z=True, signs_k=signs)
        assert torch.isfinite(y).all() and (y[1] == 0).all()
        big = z.double().abs() > 100
        assert big.any()
        want = z.double() if act == "none" else z.double().clamp(min=0)
        assert ((y.double() - want).abs()[big] <= 2.0 ** -7 * want.abs()[big]).all()
        qw, sw = H.fwht_quant(w, H.ROWS, block, signs=signs)
        assert torch.equal(H.linear_act_q(x, qw, sw, block, activation=act, signs_k=signs), y)


BWD = [(1, 8, 8, 8), (40, 64, 96, 32), (300, 520, 264, 64), (1000, 640, 512, 256),
       (4500, 256, 136, 128), (130, 4608, 256, 512)]


@pytest.mark.parametrize("q,gq", [(I8, I8), (E4M3, E5M2), (E4M3, E4M3)])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("m,n,k,block", BWD)
def test_backward(m, n, k, block, dt, q, gq):
    print(f"m {m} n {n} k {k} block {block} {dt} {q} {gq}", flush=True)
    x, w = rnd((m, k), dt, 1), rnd((n, k), dt, 2, k ** -0.5)
    z, dy = rnd((m, n), dt, 3, 1.5), rnd((m, n), dt, 4, 1e-3)
    act = ACTS[1 + (m + n + k // 8) % 4]
    dx, dw, db = H.linear_act_bwd(dy, z, x, w, block, q, gq, activation=act)
    dz = dy.double() * slope64(z.double(), act)
    # db: fp32 sums in a chain of at most 16 + 2048 additions (rows of a wave, partial rows)
    tol = ROUND[dt] * 1.01 * dz.sum(0).abs() + 2100 * U * dz.abs().sum(0)
    assert ((db.double() - dz.sum(0)).abs() <= tol).all()
    rx, rw = H.linear_bwd(dz.float(), x.float(), w.float(), block, q, gq)
    for got, ref, name in ((dx, rx, "dx"), (dw, rw, "dw")):
        rel = float((got.double() - ref.double()).norm() / ref.double().norm())
        assert rel <= ROUND[dt] / 3 ** 0.5 + 1e-3, (name, rel)
    again = H.linear_act_bwd(dy, z, x, w, block, q, gq, activation=act)
    for u, v in zip(again, (dx, dw, db)):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_backward_without_activation(dt):
    m, n, k, block = 520, 264, 384, 128
    x, w, dy = rnd((m, k), dt, 1), rnd((n, k), dt, 2), rnd((m, n), dt, 3)
    rx, rw = H.linear_bwd(dy, x, w, block)
    dx, dw, db = H.linear_act_bwd(dy, None, x, w, block)
    assert torch.equal(dx, rx) and torch.equal(dw, rw)
    s = dy.double().sum(0)
    assert ((db.double() - s).abs() <= ROUND[dt] * 1.01 * s.abs() + 600 * U * dy.double().abs().sum(0)).all()
    z = rnd((m, n), dt, 4)
    for want in ((True, False, False), (False, True, False), (False, False, True)):
        got = H.linear_act_bwd(dy, z, x, w, block, activation="silu", want_dx=want[0],
                               want_dw=want[1], want_db=want[2])
        assert tuple(v is not None for v in got) == want
    full = H.linear_act_bwd(dy, z, x, w, block, activation="silu")
    assert torch.equal(got[2], full[2])


def test_backward_options():
    # stochastic codes and random signs, against linear_bwd on the same dz
    m, n, k, block = 256, 512, 256, 128
    x, w, z, dy = rnd((m, k), F32, 1), rnd((n, k), F32, 2), rnd((m, n), F32, 3), rnd((m, n), F32, 4)
    kw = dict(signs_n=H.hadamard_signs(n, 1, DEV), signs_m=H.hadamard_signs(m, 2, DEV),
              grad_rounding="stochastic", seed=9, counter=4)
    dz = (dy.double() * (z > 0)).float()     # relu's slope is exact
    rx, rw = H.linear_bwd(dz, x, w, block, **kw)
    dx, dw, _ = H.linear_act_bwd(dy, z, x, w, block, activation="relu", **kw)
    assert torch.equal(dx, rx) and torch.equal(dw, rw)


@pytest.mark.parametrize("act", ACTS[1:])
def test_slope_against_differences(act):
    # db of a single row is dy act'(z): against central differences of the 64-bit activation
    n = 4096
    z = torch.linspace(-12, 12, n, device=DEV).to(F32)[None]
    dy, x, w = torch.ones((1, n), device=DEV), rnd((1, 8), F32, 1), rnd((n, 8), F32, 2)
    db = H.linear_act_bwd(dy, z, x, w, 8, activation=act, want_dx=False, want_dw=False)[2].double()
    h = 1e-5
    num = ((act64(z.double() + h, act) - act64(z.double() - h, act)) / (2 * h))[0]
    away = z[0].abs() > 1e-3 if act == "relu" else torch.ones_like(z[0], dtype=torch.bool)
    assert ((db - num).abs()[away] <= 1e-5).all()


def test_streams_graph_and_empty():
    m, n, k, block = 48, 256, 512, 64
    x, w, bias = rnd((m, k), BF16, 1), rnd((n, k), BF16, 2, 0.05), rnd((n,), BF16, 3)
    z, dy = rnd((m, n), BF16, 4), rnd((m, n), BF16, 5)
    qw, sw = H.fwht_quant(w, H.ROWS, block)

    def step():
        return (H.linear_act_q(x, qw, sw, block, bias=bias, activation="silu"),
                H.linear_act_fwd(x, w, block, bias=bias, activation="gelu_tanh"),
                *H.linear_act_bwd(dy, z, x, w, block, activation="gelu_erf"))

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        x.copy_(rnd((m, k), BF16, 10 + i))
        dy.copy_(rnd((m, n), BF16, 20 + i))
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, step()):
            assert torch.equal(u, v)
    e = torch.empty((0, k), dtype=BF16, device=DEV)
    assert H.linear_act_fwd(e, w, block, bias=bias).shape == (0, n)
    assert H.linear_act_q(e, qw, sw, block).shape == (0, n)


# rows, columns, contraction, block: rows quantised inside the product's kernel (up to 16 rows, 32
# slices of 512), and the shapes just past it
INSIDE = [(1, 16, 512, 512), (1, 40, 544, 32), (1, 4096, 4096, 256), (2, 24, 4064, 32),
          (3, 1000, 1536, 8), (4, 136, 4096, 2), (8, 80, 2048, 128), (16, 264, 992, 16),
          (1, 56, 16384, 64), (1, 48, 16448, 32), (16, 40, 1056, 32), (2, 32, 1024, 1024),
          (1, 64, 5504, 1)]


@pytest.mark.parametrize("q", [I8, E4M3])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("m,n,k,block", INSIDE)
def test_serving_form_equals_the_forward(m, n, k, block, dt, q):
    print(f"m {m} n {n} k {k} block {block} {dt} {q}", flush=True)
    x, w = rnd((m, k), dt, 1), rnd((n, k), dt, 2, k ** -0.5)
    x[:, 3] *= 40
    if m > 1:
        x[1] = 0                       # zero codes
    if m > 2 and dt == F32:
        x[2] *= 1e-40                  # so small that the quantiser's multiplier overflows
    bias, res = rnd((n,), dt, 3), rnd((m, n), dt, 4)
    for signs in (None, H.hadamard_signs(kq_of(k, block), 3, DEV)):
        qw, sw = H.fwht_quant(w, H.ROWS, block, q, signs=signs)
        y, z = H.linear_act_fwd(x, w, block, q, bias=bias, activation="silu", residual=res,
                                want_z=True, signs_k=signs)
        z2 = torch.empty_like(z)
        y2, _ = H.linear_act_q(x, qw, sw, block, bias=bias, activation="silu", residual=res, z=z2,
                               signs_k=signs)
        assert torch.equal(y2, y) and torch.equal(z2, z)
    if signs is not None:
        y = H.linear_act_fwd(x, w, block, q, activation="relu")
        check_fwd(x, w, block, q, "relu", None, None, y, None, dt)


@pytest.mark.parametrize("q,gq", [(I8, I8), (E4M3, E5M2)])
@pytest.mark.parametrize("act", ["silu", "gelu_erf"])
@pytest.mark.parametrize("m,n,k,block", [(256, 512, 256, 64), (4096, 64, 72, 1024), (128, 4096, 64, 128),
                                         (8192, 200, 64, 256), (5120, 520, 136, 512),
                                         (2000, 8192, 128, 128), (64, 12288, 64, 64),
                                         (448, 640, 64, 64), (1000, 1000, 256, 256)])
def test_backward_inside_the_rotations(m, n, k, block, act, q, gq):
    # shapes whose dz is formed as the rotation passes load it (whole columns, columns split over
    # workgroups, rows of one and of several waves, padded ends) against the same passes of an fp32
    # dz, and against the form that stores dz (random signs of a zero word: the same transform)
    print(f"m {m} n {n} k {k} block {block} {act} {q}", flush=True)
    x, w = rnd((m, k), BF16, 1), rnd((n, k), BF16, 2, k ** -0.5)
    z, dy = rnd((m, n), BF16, 3, 1.5), rnd((m, n), BF16, 4, 1e-3)
    z[0, :4], dy[-1] = 30.0, 0.0
    sn = torch.randint(-2 ** 31, 2 ** 31, (-(-H.contraction_len(n, block) // 32),), dtype=torch.int32).to(DEV)
    sm = torch.randint(-2 ** 31, 2 ** 31, (-(-H.contraction_len(m, block) // 32),), dtype=torch.int32).to(DEV)
    dz = dy.double() * slope64(z.double(), act)
    for kw in ({}, {"signs_n": sn, "signs_m": sm}):
        dx, dw, db = H.linear_act_bwd(dy, z, x, w, block, q, gq, activation=act, **kw)
        tol = ROUND[BF16] * 1.01 * dz.sum(0).abs() + 2100 * U * dz.abs().sum(0)
        assert ((db.double() - dz.sum(0)).abs() <= tol).all()
        rx, rw = H.linear_bwd(dz.float(), x.float(), w.float(), block, q, gq, **kw)
        for got, ref, name in ((dx, rx, "dx"), (dw, rw, "dw")):
            rel = float((got.double() - ref.double()).norm() / ref.double().norm())
            assert rel <= ROUND[BF16] / 3 ** 0.5 + 1e-3, (name, rel)
        again = H.linear_act_bwd(dy, z, x, w, block, q, gq, activation=act, **kw)
        only = H.linear_act_bwd(dy, z, x, w, block, q, gq, activation=act, want_dx=False, **kw)
        for u, v in zip(again, (dx, dw, db)):
            assert torch.equal(u, v)
        rel = float((only[1].double() - dw.double()).norm() / dw.double().norm())
        assert rel <= 1e-3   # the stored dz: the same fp32 values, the same codes


def tiles(m, n, t):
    return -(-m // t) * -(-n // t)


@pytest.mark.parametrize("q", [I8, E4M3])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("m,n,k,block", [(400, 4096, 512, 64), (1000, 1096, 160, 32), (333, 4104, 96, 32),
                                         (450, 2400, 256, 64), (257, 4096, 384, 128), (700, 1928, 1152, 128),
                                         (520, 2056, 1376, 32)])
def test_forward_on_the_small_tiles(m, n, k, block, dt, q):
    # more 64 x 64 tiles than compute units and too few 128 x 128 ones: the 64 x 64 tile kernel;
    # contractions of one to eleven 128-byte slabs (its ring holds four), whole and ragged
    assert tiles(m, n, 64) > 256 and tiles(m, n, 128) < 224
    test_forward(m, n, k, block, dt, q)


@pytest.mark.parametrize("act", ACTS)
def test_parts_of_the_epilogue_on_the_small_tiles(act):
    assert tiles(700, 1928, 64) > 256 and tiles(700, 1928, 128) < 224
    test_parts_of_the_epilogue(700, act)


# finite z whose square, cube or exponential passes the type's range
FAR = [30.0, 1e4, 1e10, 1.9e19, 1e20, 1e30, 3e38]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("act", ACTS[1:])
def test_activations_and_slopes_far_out(act, dt):
    """z so large that every activation is z or 0 and every slope 1 or 0, to the last bit: the nearest,
    gelu at -30, is 30 exp(-450)."""
    v = torch.tensor(FAR + [-f for f in FAR], dtype=torch.float64, device=DEV).to(dt)
    n, k, block = v.numel() + 2, 64, 64
    bias = torch.zeros(n, dtype=dt, device=DEV)
    bias[:v.numel()] = v
    w = rnd((n, k), dt, 1)
    for m in (1, 40):                      # rows of zeros: z is the bias
        x = torch.zeros((m, k), dtype=dt, device=DEV)
        y, z = H.linear_act_fwd(x, w, block, bias=bias, activation=act, want_z=True)
        assert torch.equal(z, bias.expand(m, n))
        assert ((y.double() - z.double().clamp(min=0)).abs() <= 1e-11).all()
    want = (v > 0).to(dt)
    for m in (1, 128):                     # 128 rows: dz inside the rotations (bf16)
        z = bias.expand(m, n).contiguous()
        dy = torch.zeros((m, n), dtype=dt, device=DEV)
        dy[0] = 1
        dx, dw, db = H.linear_act_bwd(dy, z, rnd((m, k), dt, 2), w, block, activation=act)
        assert ((db[:v.numel()] - want).abs() <= 1e-9).all()
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
        only = H.linear_act_bwd(dy, z, rnd((m, k), dt, 2), w, block, activation=act, want_dw=False)
        assert torch.equal(only[2], db) and torch.isfinite(only[0]).all()


@pytest.mark.parametrize("kw,dt", [(dict(activation="silu"), BF16), (dict(activation="silu"), F32),
                                   (dict(activation="silu", want_db=False), BF16),
                                   (dict(activation="gelu_erf", want_dw=False), BF16),
                                   (dict(activation="gelu_erf", want_dx=False, want_db=False), BF16),
                                   (dict(activation="relu", want_dx=False, want_dw=False), F32),
                                   (dict(), BF16), (dict(want_db=False), F32),
                                   (dict(activation="gelu_tanh", grad_rounding="stochastic"), BF16)])
@pytest.mark.parametrize("m,n,k,block", [(300, 520, 264, 64), (4500, 256, 136, 128), (64, 128, 64, 32)])
def test_backward_in_its_own_workspace(m, n, k, block, kw, dt):
    x, w = rnd((m, k), dt, 1), rnd((n, k), dt, 2, k ** -0.5)
    z, dy = rnd((m, n), dt, 3, 1.5), rnd((m, n), dt, 4, 1e-3)
    need = H.linear_act_bwd_workspace_bytes(m, n, k, block, torch.int8, dt, **kw)
    assert need <= H.linear_act_bwd_workspace_bytes(m, n, k, block)
    room = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    want = H.linear_act_bwd(dy, z, x, w, block, **kw)
    got = H.linear_act_bwd(dy, z, x, w, block, workspace=room[:need], **kw)
    for u, v in zip(got, want):
        assert (u is None and v is None) or torch.equal(u, v)
    assert (room[need:] == 77).all()
    with pytest.raises(H.HaloError, match="WORKSPACE"):
        H.linear_act_bwd(dy, z, x, w, block, workspace=room[:need - 1], **kw)


@pytest.mark.parametrize("m", [1, 40, 300, 1100, 3900])
def test_gelu_in_fp32_keeps_its_tail(m):
    """gelu by its distribution in fp32 outputs, relative to its own value down to z = -12.  With x = 0
    z is the bias.  The distribution's argument carries two roundings, which move it by at most
    2 u (z^2 + 1) of itself, the library's erfc 4 units in the last place, the two products around it
    one rounding each: u (16 + 2 (z^2 + 1)) of |y|."""
    n, k, block = 4096 if m > 40 else 4000, 64, 64
    bias = torch.linspace(-12, 12, n, device=DEV)
    x, w = torch.zeros((m, k), device=DEV), rnd((n, k), F32, 1)
    y, z = H.linear_act_fwd(x, w, block, bias=bias, activation="gelu_erf", want_z=True)
    assert torch.equal(z, bias.expand(m, n))
    want = bias.double() * torch.special.erfc(-bias.double() * 0.5 ** 0.5) / 2
    assert ((y.double() - want).abs() <= U * (16 + 2 * (bias.double() ** 2 + 1)) * want.abs()).all()
    qw, sw = H.fwht_quant(w, H.ROWS, block)
    assert torch.equal(H.linear_act_q(x, qw, sw, block, bias=bias, activation="gelu_erf"), y)
    # bf16 operands with fp32 outputs alike
    y = H.linear_act_fwd(x.bfloat16(), w.bfloat16(), block, bias=bias, activation="gelu_erf", y_dtype=F32)
    assert ((y.double() - want).abs() <= U * (16 + 2 * (bias.double() ** 2 + 1)) * want.abs()).all()


@pytest.mark.parametrize("q,gq", [(I8, I8), (E4M3, E5M2)])
def test_backward_when_tasks_stop_waiting(q, gq):
    """Columns split over 48 workgroups that exchange their maxima, dz formed inside: with one poll of
    the bounded wait, tasks stop waiting and the launch behind stores their parts from dy and z again;
    the gradients are the same bits, and the bias gradient's sums are counted once."""
    m, n, k, block = 49152, 384, 64, 256
    x, w = rnd((m, k), BF16, 1), rnd((n, k), BF16, 2, k ** -0.5)
    z, dy = rnd((m, n), BF16, 3, 1.5), rnd((m, n), BF16, 4, 1e-3)
    want = H.linear_act_bwd(dy, z, x, w, block, q, gq, activation="silu")
    dz = dy.double() * slope64(z.double(), "silu")
    tol = ROUND[BF16] * 1.01 * dz.sum(0).abs() + 2100 * U * dz.abs().sum(0)
    assert ((want[2].double() - dz.sum(0)).abs() <= tol).all()
    for _ in range(4):
        got = H.linear_act_bwd(dy, z, x, w, block, q, gq, activation="silu", exchange_polls=1)
        for u, v in zip(got, want):
            assert torch.equal(u, v)
