"""The gated feed-forward layer (linear_glu_fwd, linear_glu_q, linear_glu_bwd).

Forward.  z is held as the layer's epilogue tests hold it: the codes are fwht_quant's, the product has
an exact value in 64 bits, INT8 sums are exact and z carries at most 5 roundings of 2^-24 of |product| +
|bias|; FP8 sums carry the matrix core's documented bound on top.  y = act(g) u: an error e of g passes
through the activation with at most its largest slope (1.13) and joins 2^-24 (16 + 4 |g|) |g| of the
activation itself (exponent scaled to base 2, units in the last place of exp and rcp, erf); with that sum
called a, y is off by a |u| + |act(g)| e_u + a e_u and one rounding.  y and z are rounded once on their
stores (2^-8 for bf16).

Backward.  The products are linear_bwd's on a dz that torch computes in 64 bits and rounds to fp32: the
two dz differ by some 2^-24, which moves a code in about 2^-20 of the places by one step of absmax / 127
(about 3 % of the rms; FP8 less), 1e-4 of the result in norm, beside the output's rounding."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I8, E4M3, E5M2 = (torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn,
                             torch.float8_e5m2)
ROUND = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24
ETA = 2.0 ** -149
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


def glu_grad64(dy, z, act):
    """dz of y = act(g) u in 64 bits, by autograd."""
    z = z.detach().double().clone().requires_grad_(True)
    g, u = z.split(dy.shape[1], 1)
    (act64(g, act) * u).backward(dy.double())
    return z.grad


def codes(t, block, q):
    full = torch.zeros((t.shape[0], H.contraction_len(t.shape[1], block)), dtype=t.dtype, device=DEV)
    full[:, :t.shape[1]] = t
    return H.fwht_quant(full, H.ROWS, block, q)


def z64(x, w, block, q, bias):
    """z and the bound of its error before its rounding."""
    (qx, sx), (qw, sw) = codes(x, block, q), codes(w, block, q)
    a, b = qx.double(), qw.double()
    s = sx.double()[:, None] * sw.double()[None, :]
    prod = (a @ b.t()) * s
    bz = bias.double() if bias is not None else torch.zeros(w.shape[0], dtype=torch.float64, device=DEV)
    err = 5 * U * (prod.abs() + bz.abs()) + 5 * ETA
    if q != I8:
        n = a.shape[1] / 8 + 2
        err = err + (2.0 ** -10 + n * U / (1 - n * U)) * (a.abs() @ b.abs().t()) * s
    return prod + bz, err


def check_fwd(x, w, block, q, act, bias, y, z, yt):
    ref, err = z64(x, w, block, q, bias)
    if z is not None:
        bad = (z.double() - ref).abs() > err + ROUND[yt] * (ref.abs() + err)
        assert not bad.any(), ("z", int(bad.sum()))
    n = y.shape[1]
    (g, u), (eg, eu) = ref.split(n, 1), err.split(n, 1)
    a = act64(g, act)
    ea = 1.13 * eg + (U * (16 + 4 * g.abs()) * g.abs() if act not in ("none", "relu") else 0)
    want = a * u
    e = ea * u.abs() + a.abs() * eu + ea * eu + U * want.abs()
    bad = (y.double() - want).abs() > e + ROUND[yt] * (want.abs() + e)
    assert not bad.any(), ("y", int(bad.sum()), torch.nonzero(bad)[0].tolist())


# rows, columns, contraction, block: up to 16 rows (quantised inside and not), waves that split the
# contraction, 64, 128 and 256 tiles, whole and ragged tiles and contractions
SHAPES = [(1, 8, 32, 32), (1, 264, 4096, 256), (5, 40, 96, 32), (16, 512, 1000, 8), (16, 136, 8192, 64),
          (17, 1000, 640, 64), (33, 72, 2048, 1024), (64, 136, 4128, 32), (65, 200, 512, 128),
          (203, 520, 1376, 32), (400, 2048, 512, 64), (333, 2056, 96, 32), (700, 1000, 256, 64),
          (1800, 1000, 160, 32), (1800, 1000, 256, 64), (3800, 1928, 128, 64), (3840, 1920, 224, 32)]


@pytest.mark.parametrize("q", [I8, E4M3])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("m,n,k,block", SHAPES)
def test_forward(m, n, k, block, dt, q):
    print(f"m {m} n {n} k {k} block {block} {dt} {q}", flush=True)
    x, w = rnd((m, k), dt, 1), rnd((2 * n, k), dt, 2, 2.0 * k ** -0.5)
    bias = rnd((2 * n,), dt, 3)
    act = ACTS[(m + n // 8) % 5]
    y, z = H.linear_glu_fwd(x, w, block, q, bias=bias, activation=act, want_z=True)
    check_fwd(x, w, block, q, act, bias, y, z, dt)
    err = z64(x, w, block, q, bias)[1].view(2 * m, n)
    assert torch.equal(y, H.linear_glu_fwd(x, w, block, q, bias=bias, activation=act))
    if H.contraction_len(k, block) == H.padded_len(k, block):
        qw, sw = H.fwht_quant(w, H.ROWS, block, q)
        assert torch.equal(H.linear_glu_q(x, qw, sw, block, bias=bias, activation=act), y)
    for kept in (I8, E4M3):
        y8, z8 = H.linear_glu_fwd(x, w, block, q, bias=bias, activation=act, want_z=kept)
        assert z8.codes.shape == (2 * m, n)
        if m > 16:    # up to 16 rows another kernel writes a plain z (its product rounded before the bias)
            assert torch.equal(y8, y)
            if dt == F32:
                want = H.checkpoint_pack(z.view(2 * m, n), kept)
                assert torch.equal(z8.powers, want.powers)
                assert torch.equal(z8.codes.view(torch.uint8), want.codes.view(torch.uint8))
        else:
            check_fwd(x, w, block, q, act, bias, y8, None, dt)
        step = torch.exp2(z8.powers.double() - 127).repeat_interleave(32, 1)[:, :n]
        zz = z.double().view(2 * m, n)
        half = 0.5 * step if kept == I8 else (2.0 ** -4 * zz.abs() + 2.0 ** -10 * step)
        off = (H.checkpoint_unpack(z8, F32).double() - zz).abs()
        assert (off <= 1.001 * half + 1.1 * (ROUND[dt] * (zz.abs() + err) + 2 * err)).all()


@pytest.mark.parametrize("m", [3, 70, 700, 2000])
@pytest.mark.parametrize("act", ACTS)
def test_parts_of_the_epilogue(m, act):
    n, k, block = 968, 128, 64
    x, w = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, 0.3)
    y = H.linear_glu_fwd(x, w, block, activation=act)
    check_fwd(x, w, block, I8, act, None, y, None, BF16)
    y32, z32 = H.linear_glu_fwd(x, w, block, activation=act, y_dtype=F32, want_z=True)
    check_fwd(x, w, block, I8, act, None, y32, z32, F32)
    # the halves are the layer's own product
    z = H.linear_act_fwd(x, w, block, y_dtype=F32)
    assert torch.equal(z, z32)
    out, zo = torch.empty_like(y), torch.empty((m, 2 * n), dtype=BF16, device=DEV)
    got = H.linear_glu_fwd(x, w, block, activation=act, y=out, z=zo)
    assert got[0] is out and got[1] is zo and torch.equal(out, y)
    check_fwd(x, w, block, I8, act, None, out, zo, BF16)
    signs = H.hadamard_signs(k, 5, DEV)
    qw, sw = H.fwht_quant(w, H.ROWS, block, signs=signs)
    assert torch.equal(H.linear_glu_q(x, qw, sw, block, activation=act, signs_k=signs),
                       H.linear_glu_fwd(x, w, block, activation=act, signs_k=signs))


# rows quantised inside the product's kernel (up to 16 rows, 32 slices of 512), and just past it
INSIDE = [(1, 16, 512, 512), (1, 40, 544, 32), (1, 4096, 4096, 256), (2, 24, 4064, 32),
          (3, 1000, 1536, 8), (8, 80, 2048, 128), (16, 264, 992, 16), (1, 48, 16448, 32),
          (16, 40, 1056, 32), (2, 32, 1024, 1024)]


@pytest.mark.parametrize("q", [I8, E4M3])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("m,n,k,block", INSIDE)
def test_serving_form_equals_the_forward(m, n, k, block, dt, q):
    print(f"m {m} n {n} k {k} block {block} {dt} {q}", flush=True)
    x, w = rnd((m, k), dt, 1), rnd((2 * n, k), dt, 2, k ** -0.5)
    x[:, 3] *= 40
    if m > 1:
        x[1] = 0
    bias = rnd((2 * n,), dt, 3)
    qw, sw = H.fwht_quant(w, H.ROWS, block, q)
    y = H.linear_glu_fwd(x, w, block, q, bias=bias, activation="silu")
    check_fwd(x, w, block, q, "silu", bias, y, None, dt)
    assert torch.equal(H.linear_glu_q(x, qw, sw, block, bias=bias, activation="silu"), y)


def test_fp32_rows_of_a_multiple_of_four():
    # an fp32 y of 4, 12 .. columns: halves that end inside a lane's 8 columns
    for m in (2, 40, 300):
        for n in (4, 12, 36, 100):
            x, w, bias = rnd((m, 64), F32, 1), rnd((2 * n, 64), F32, 2, 0.2), rnd((2 * n,), F32, 3)
            y, z = H.linear_glu_fwd(x, w, 64, bias=bias, activation="gelu_tanh", want_z=True)
            check_fwd(x, w, 64, I8, "gelu_tanh", bias, y, z, F32)


BWD = [(1, 8, 8, 8), (40, 64, 96, 32), (300, 520, 264, 64), (1000, 640, 512, 256),
       (4500, 256, 136, 128), (130, 4608, 256, 512), (256, 256, 256, 64), (4096, 32, 72, 1024),
       (8192, 200, 64, 256), (2000, 4096, 128, 128), (64, 6144, 64, 64), (448, 328, 64, 64),
       (1000, 1048, 1056, 64), (1000, 504, 256, 256)]


def check_bwd(got, dy, zv, xv, w, block, q, gq, act, dt, **kw):
    dx, dw, db = got
    dz = glu_grad64(dy, zv, act)
    # db: fp32 sums in a chain of at most 16 + 2048 additions (rows of a wave, partial rows)
    tol = ROUND[dt] * 1.01 * dz.sum(0).abs() + 2100 * U * dz.abs().sum(0)
    assert ((db.double() - dz.sum(0)).abs() <= tol).all()
    rx, rw = H.linear_bwd(dz.float(), xv.float(), w.float(), block, q, gq, **kw)
    for g, ref, name in ((dx, rx, "dx"), (dw, rw, "dw")):
        rel = float((g.double() - ref.double()).norm() / ref.double().norm())
        assert rel <= ROUND[dt] / 3 ** 0.5 + 1e-3, (name, rel)


@pytest.mark.parametrize("q,gq", [(I8, I8), (E4M3, E5M2), (E4M3, E4M3)])
@pytest.mark.parametrize("m,n,k,block", BWD)
def test_backward(m, n, k, block, q, gq):
    print(f"m {m} n {n} k {k} block {block} {q} {gq}", flush=True)
    act = ACTS[(m + n // 8 + k // 8) % 5]
    for dt, kx, kz in ((BF16, None, None), (F32, None, None), (BF16, I8, E4M3), (BF16, E4M3, I8),
                       (BF16, None, I8), (F32, I8, I8)):
        x, w = rnd((m, k), dt, 1), rnd((2 * n, k), dt, 2, k ** -0.5)
        z, dy = rnd((m, 2 * n), dt, 3, 1.5), rnd((m, n), dt, 4, 1e-3)
        z[0, :4], dy[-1, 0] = 30.0, 0.0
        ck = H.checkpoint_pack(x, kx) if kx else x
        cz = H.checkpoint_pack(z.view(2 * m, n), kz) if kz else z
        xv = H.checkpoint_unpack(ck, dt) if kx else x
        zv = H.checkpoint_unpack(cz, dt).view(m, 2 * n) if kz else z
        got = H.linear_glu_bwd(dy, cz, ck, w, block, q, gq, activation=act)
        check_bwd(got, dy, zv, xv, w, block, q, gq, act, dt)
        again = H.linear_glu_bwd(dy, cz, ck, w, block, q, gq, activation=act)
        assert all(torch.equal(u, v) for u, v in zip(again, got))


@pytest.mark.parametrize("act", ACTS)
def test_backward_options_and_parts(act):
    m, n, k, block = 256, 512, 264, 128
    x, w, z, dy = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2), rnd((m, 2 * n), BF16, 3), rnd((m, n), BF16, 4)
    signs = dict(signs_n=H.hadamard_signs(2 * n, 1, DEV), signs_m=H.hadamard_signs(m, 2, DEV))
    check_bwd(H.linear_glu_bwd(dy, z, x, w, block, activation=act, **signs), dy, z, x, w, block, I8, I8,
              act, BF16, **signs)
    full = H.linear_glu_bwd(dy, z, x, w, block, activation=act)
    for want in ((True, False, False), (False, True, False), (False, False, True), (True, True, False)):
        got = H.linear_glu_bwd(dy, z, x, w, block, activation=act, want_dx=want[0], want_dw=want[1],
                               want_db=want[2])
        for g, f, there in zip(got, full, want):
            assert (g is not None) == there
            if there:
                assert float((g.double() - f.double()).norm()) <= 4e-3 * float(f.double().norm())
    if act in ("none", "relu"):   # exact slopes: the same stochastic codes as linear_bwd's
        kw = dict(grad_rounding="stochastic", seed=9, counter=4)
        dz = glu_grad64(dy, z, act).float()
        got = H.linear_glu_bwd(dy.float(), z.float(), x.float(), w.float(), block, activation=act, **kw)
        want = H.linear_bwd(dz, x.float(), w.float(), block, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(act):
    # db of a single row is dz: against central differences of the 64-bit formula, in fp32
    n = 2048
    g = torch.linspace(-9, 9, n, device=DEV)
    u = rnd((n,), F32, 6, 2.0)
    z, dy = torch.cat([g, u])[None], rnd((1, n), F32, 7)
    x, w = rnd((1, 8), F32, 1), rnd((2 * n, 8), F32, 2)
    db = H.linear_glu_bwd(dy, z, x, w, 8, activation=act, want_dx=False, want_dw=False)[2].double()
    h, g, u, d = 1e-5, g.double(), u.double(), dy.double()[0]
    dg = d * u * (act64(g + h, act) - act64(g - h, act)) / (2 * h)
    du = d * (act64(g, act) * (u + h) - act64(g, act) * (u - h)) / (2 * h)
    away = g.abs() > 1e-3 if act == "relu" else torch.ones_like(g, dtype=torch.bool)
    scale = 1 + (d * u).abs() + (d * act64(g, act)).abs()
    assert ((db[:n] - dg).abs() <= 1e-5 * scale)[away].all()
    assert ((db[n:] - du).abs() <= 1e-5 * scale).all()


FAR = [30.0, 1e4, 1e10, 1.9e19, 1e30]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("act", ACTS[1:])
def test_gates_far_out(act, dt):
    """Gates so large that every activation is g or 0 and every slope 1 or 0, with an up projection of
    2: y = 2 g or 0, dg = 2 dy or 0, du = dy g or 0 (the nearest gate, gelu at -30, is 30 exp(-450))."""
    v = torch.tensor(FAR + [-f for f in FAR], dtype=torch.float64, device=DEV).to(dt)
    n, k, block = v.numel() + 6, 64, 64
    bias = torch.zeros(2 * n, dtype=dt, device=DEV)
    bias[:v.numel()] = v
    bias[n:] = 2
    w = rnd((2 * n, k), dt, 1)
    pos = v.double().clamp(min=0)
    for m in (1, 40, 128):
        x = torch.zeros((m, k), dtype=dt, device=DEV)
        y, z = H.linear_glu_fwd(x, w, block, bias=bias, activation=act, want_z=True)
        assert torch.equal(z, bias.expand(m, 2 * n))
        assert ((y[:, :v.numel()].double() - 2 * pos).abs() <= 1e-10).all()
        dy = torch.zeros((m, n), dtype=dt, device=DEV)
        dy[0] = 1
        dx, dw, db = H.linear_glu_bwd(dy, z, x, w, block, activation=act)
        assert ((db[:v.numel()].double() - 2 * (v > 0)).abs() <= 1e-9).all()
        assert ((db[n:n + v.numel()].double() - pos).abs() <= 1e-10).all()
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_streams_graph_and_empty():
    m, n, k, block = 48, 256, 512, 64
    x, w, bias = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, 0.05), rnd((2 * n,), BF16, 3)
    dy = rnd((m, n), BF16, 5)
    qw, sw = H.fwht_quant(w, H.ROWS, block)

    def step():
        y, z = H.linear_glu_fwd(x, w, block, bias=bias, activation="gelu_tanh", want_z=I8)
        kept = H.checkpoint_pack(x, E4M3)
        return (y, z.codes, H.linear_glu_q(x, qw, sw, block, bias=bias), H.linear_glu_q(x[:1], qw, sw, block),
                *H.linear_glu_bwd(dy, z, kept, w, block, activation="gelu_tanh"))

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
    assert H.linear_glu_fwd(e, w, block, bias=bias).shape == (0, n)
    y, z = H.linear_glu_fwd(e, w, block, want_z=I8)
    assert y.shape == (0, n) and z.codes.shape == (0, n)
    assert H.linear_glu_q(e, qw, sw, block).shape == (0, n)


@pytest.mark.parametrize("kw", [dict(), dict(want_db=False), dict(want_dw=False), dict(want_dx=False),
                                dict(want_dx=False, want_dw=False), dict(grad_rounding="stochastic")])
@pytest.mark.parametrize("kept", [None, I8])
@pytest.mark.parametrize("m,n,k,block", [(300, 520, 264, 64), (4500, 256, 136, 128), (64, 128, 64, 32)])
def test_backward_in_its_own_workspace(m, n, k, block, kept, kw):
    x, w = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, k ** -0.5)
    z, dy = rnd((m, 2 * n), BF16, 3, 1.5), rnd((m, n), BF16, 4, 1e-3)
    if kept:
        x, z = H.checkpoint_pack(x, kept), H.checkpoint_pack(z.view(2 * m, n), kept)
    need = H.linear_kept_bwd_workspace_bytes(True, m, n, k, block, activation="silu", z_dtype=kept,
                                             x_dtype=kept, **kw)
    room = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    want = H.linear_glu_bwd(dy, z, x, w, block, **kw)
    got = H.linear_glu_bwd(dy, z, x, w, block, workspace=room[:need], **kw)
    for u, v in zip(got, want):
        assert (u is None and v is None) or torch.equal(u, v)
    assert (room[need:] == 77).all()
    with pytest.raises(H.HaloError, match="WORKSPACE"):
        H.linear_glu_bwd(dy, z, x, w, block, workspace=room[:need - 1], **kw)
