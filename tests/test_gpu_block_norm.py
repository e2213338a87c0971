"""The join between two blocks (block_norm_fwd / block_norm_bwd) against its formula in 64 bits.

Tolerances.  Every output is rounded once to its type (relative 2^-8 for bf16, 2^-24 for fp32).
The fp32 arithmetic before it adds at most GAMMA = 512 * 2^-24 of the sum of the absolute values
of the terms a result is made of: a sum runs over at most 64 + 64 + 16 additions in a chain
(elements of a lane, lanes, waves) for a row, 256 + 64 + 256 / 4 over tokens, and the factors
around it add a few roundings.  The absolute terms are computed beside the 64-bit result."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
GAMMA = 512 * 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF16, F32 = torch.bfloat16, torch.float32


def rnd(shape, dt, seed, scale=1.0, pad=0):
    """Normal values of a type; pad > 0: rows `pad` elements apart from each other."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    full = (shape[0], shape[1] + pad) if pad else shape
    t = (torch.randn(full, generator=g, device=DEV) * scale).to(dt)
    return t[:, :shape[1]] if pad else t


def check(got, ref, absolute, dt, what):
    got = got.double()
    assert got.shape == ref.shape, what
    tol = ROUND[dt] * (1 + 2.0 ** -6) * ref.abs() + GAMMA * absolute
    bad = (got - ref).abs() > tol
    assert torch.isfinite(got).all(), what
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() / (tol + 1e-300)).max()))


def rows_of(gate, t):
    return gate.double().repeat_interleave(t // gate.shape[0], 0)


def fwd64(r, y, gate, post, pre, scale, eps):
    t, d = r.shape
    out, terms, a = r.double(), r.double().abs(), None
    if y is not None:
        n = y.double()
        if post is not None:
            a = 1 / torch.sqrt(n.pow(2).mean(1) + eps)
            n = n * a[:, None] * post.double()
        if gate is not None:
            n = n * rows_of(gate, t)
        out = out + scale * n
        terms = terms + abs(scale) * n.abs()
    h = b = None
    if pre is not None:
        b = 1 / torch.sqrt(out.pow(2).mean(1) + eps)
        h = out * b[:, None] * pre.double()
    return out, terms, h, a, b


def bwd64(dr, dh, r, y, gate, post, pre, a, b, scale):
    """Gradients and, beside each, the sum of the absolute values it is made of."""
    ref = dr if dr is not None else dh
    t, d = ref.shape
    G = dr.double() if dr is not None else torch.zeros(t, d, dtype=torch.float64, device=DEV)
    A, dpre = G.abs(), None
    if pre is not None:
        rhat, u = r.double() * b.double()[:, None], dh.double() * pre.double()
        bb = b.double()[:, None]
        G = G + bb * (u - rhat * (u * rhat).mean(1, True))
        A = A + bb.abs() * (u.abs() + rhat.abs() * (u * rhat).abs().mean(1, True))
        dpre = ((dh.double() * rhat).sum(0), (dh.double() * rhat).abs().sum(0))
    res = {"dr": (G, A), "dpre": dpre}
    if y is not None:
        one = torch.ones(1, d, dtype=torch.float64, device=DEV)
        g = (rows_of(gate, t) if gate is not None else one) * scale
        w = post.double()[None] if post is not None else one
        yhat = y.double() * (a.double()[:, None] if post is not None else 1)
        groups = gate.shape[0] if gate is not None else 1
        gr = scale * yhat * w
        res["dgate"] = ((gr * G).view(groups, -1, d).sum(1), (gr.abs() * A).view(groups, -1, d).sum(1))
        res["dpost"] = ((g * G * yhat).sum(0), ((g * yhat).abs() * A).sum(0))
        c = g * w
        if post is not None:
            aa = a.double()[:, None]
            res["dy"] = (aa * (c * G - yhat * (c * G * yhat).mean(1, True)),
                         aa * (c.abs() * A + yhat.abs() * (c.abs() * A * yhat.abs()).mean(1, True)))
        else:
            res["dy"] = (c * G, c.abs() * A)
    return res


# tokens, dim, gate rows (0: no gate), row padding
SHAPES = [(1, 1, 1, 0), (3, 5, 3, 1), (2, 8, 2, 0), (9, 7, 0, 0), (1, 4096, 1, 0),
          (7, 1000, 7, 3), (300, 129, 4, 0), (1030, 2048, 1, 8), (5, 8200, 5, 0), (4, 513, 2, 1),
          (2050, 520, 2050, 0), (2048, 64, 16, 0), (3000, 257, 1000, 0), (640, 1026, 5, 2),
          (70, 4097, 2, 0)]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("t,d,groups,pad", SHAPES + [(3, 16384, 1, 0), (2, 16383, 2, 1)])
def test_forward_and_backward(t, d, groups, pad, dt):
    print(f"tokens {t} dim {d} gate rows {groups} padding {pad} {dt}", flush=True)
    r, y = rnd((t, d), dt, 1, 3.0, pad), rnd((t, d), dt, 2, 0.7, pad)
    gate = rnd((groups, d), dt, 3) if groups else None
    post, pre = rnd((d,), dt, 4) + 1, rnd((d,), dt, 5) + 1
    scale, eps = 0.625, 1e-5
    r0, y0 = r.clone(), y.clone()
    out, h, a, b = H.block_norm_fwd(r, y, gate=gate, post_weight=post, pre_weight=pre,
                                    scale=scale, eps=eps)
    assert torch.equal(r, r0) and torch.equal(y, y0)
    rout, rterms, rh, ra, rb = fwd64(r, y, gate, post, pre, scale, eps)
    check(out, rout, rterms, dt, "r_out")
    check(h, rh, rterms * rb[:, None] * pre.double().abs(), dt, "h")
    check(a, ra, ra, F32, "rstd_post")
    # b depends on r_out, whose own error is relative to its terms
    check(b, rb, rb ** 3 * (rout.abs() * rterms).mean(1) + rb, F32, "rstd_pre")

    dr, dh = rnd((t, d), dt, 6, 0.01, pad), rnd((t, d), dt, 7, 0.01)
    g = H.block_norm_bwd(dr, dh, out, y, gate=gate, post_weight=post, pre_weight=pre,
                         rstd_post=a, rstd_pre=b, scale=scale)
    ref = bwd64(dr, dh, out, y, gate, post, pre, a, b, scale)
    for name, v in zip(("dr", "dy", "dgate", "dpost", "dpre"), g):
        if name == "dgate" and gate is None:
            assert v is None
            continue
        check(v, *ref[name], dt, name)
    again = H.block_norm_bwd(dr, dh, out, y, gate=gate, post_weight=post, pre_weight=pre,
                             rstd_post=a, rstd_pre=b, scale=scale)
    for v, w in zip(g, again):
        assert v is None or torch.equal(v, w)   # sums in a fixed order


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("join,gated,post,pre,incoming",
                         [(False, False, False, True, True), (False, False, False, True, False),
                          (True, False, False, False, True), (True, True, False, False, True),
                          (True, False, True, False, True), (True, False, False, True, False),
                          (True, True, True, True, False)])
def test_parts_left_out(join, gated, post, pre, incoming, dt):
    t, d = 37, 2309
    r, y = rnd((t, d), dt, 1), rnd((t, d), dt, 2) if join else None
    gate = rnd((1, d), dt, 3)[0] if gated else None      # a 1-D gate is one row
    wp, wq = rnd((d,), dt, 4) if post else None, rnd((d,), dt, 5) if pre else None
    out, h, a, b = H.block_norm_fwd(r, y, gate=gate, post_weight=wp, pre_weight=wq, scale=-0.5)
    g2 = None if gate is None else gate[None]
    rout, terms, rh, ra, rb = fwd64(r, y, g2, wp, wq, -0.5, 1e-6)
    if join:
        check(out, rout, terms, dt, "r_out")
    else:
        assert out is r
    assert (h is None) == (not pre) and (a is None) == (not post) and (b is None) == (not pre)
    if pre:
        check(h, rh, terms * rb[:, None] * wq.double().abs(), dt, "h")
    dr = rnd((t, d), dt, 6) if incoming else None
    dh = rnd((t, d), dt, 7) if pre else None
    g = H.block_norm_bwd(dr, dh, out, y, gate=gate, post_weight=wp, pre_weight=wq, rstd_post=a,
                         rstd_pre=b, scale=-0.5)
    ref = bwd64(dr, dh, out, y, g2, wp, wq, a, b, -0.5)
    for name, v, there in zip(("dr", "dy", "dgate", "dpost", "dpre"), g,
                              (True, join, gated, post, pre)):
        assert (v is not None) == there, name
        if there:
            check(v, *ref[name], dt, name)


def test_gradient_against_differences():
    # L = <A, r_out> + <B, h> in fp32; the directional derivative of the 64-bit formula by
    # central differences (error O(step^2)) against the kernel's gradients along the direction
    t, d, groups, scale, eps = 24, 131, 3, 0.5, 1e-5
    names = ("r", "y", "gate", "post", "pre")
    x = {"r": rnd((t, d), F32, 1), "y": rnd((t, d), F32, 2), "gate": rnd((groups, d), F32, 3),
         "post": rnd((d,), F32, 4), "pre": rnd((d,), F32, 5)}
    A, B = rnd((t, d), F32, 6), rnd((t, d), F32, 7)
    out, h, a, b = H.block_norm_fwd(x["r"], x["y"], gate=x["gate"], post_weight=x["post"],
                                    pre_weight=x["pre"], scale=scale, eps=eps)
    dr, dy, dg, dp, dq = H.block_norm_bwd(A, B, out, x["y"], gate=x["gate"], post_weight=x["post"],
                                          pre_weight=x["pre"], rstd_post=a, rstd_pre=b, scale=scale)
    grads = {"r": dr, "y": dy, "gate": dg, "post": dp, "pre": dq}

    def loss(v):
        o, _, hh, _, _ = fwd64(v["r"], v["y"], v["gate"], v["post"], v["pre"], scale, eps)
        return float((A.double() * o).sum() + (B.double() * hh).sum())

    for n in names:
        v = rnd(tuple(x[n].shape), F32, 11).double()
        step = 1e-4
        up, down = ({k: w.double() + (s * v if k == n else 0) for k, w in x.items()}
                    for s in (step, -step))
        num = (loss(up) - loss(down)) / (2 * step)
        ours = float((grads[n].double() * v).sum())
        size = float((grads[n].double() * v).abs().sum())
        assert abs(num - ours) <= 1e-4 * size, (n, num, ours, size)


@pytest.mark.parametrize("d", [512, 1003, 8192])
def test_in_place_and_other_stream(d):
    t = 65
    r, y = rnd((t, d), BF16, 1), rnd((t, d), BF16, 2)
    w = rnd((d,), BF16, 3)
    want = H.block_norm_fwd(r, y, post_weight=w, pre_weight=w)
    plain = H.block_norm_fwd(r, y)[0]                       # a bare sum: no reduction in between
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r2, y2 = r.clone(), y.clone()
    s.wait_stream(torch.cuda.current_stream())
    got = H.block_norm_fwd(r2, y2, post_weight=w, pre_weight=w, r_out=r2, h=y2, stream=s)
    s.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    r2 = r.clone()
    assert torch.equal(H.block_norm_fwd(r2, y, r_out=r2)[0], plain)
    dr, dh = rnd((t, d), BF16, 4), rnd((t, d), BF16, 5)
    kw = dict(post_weight=w, pre_weight=w, rstd_post=want[2], rstd_pre=want[3])
    g = H.block_norm_bwd(dr, dh, want[0], y, **kw)
    dr2, y2 = dr.clone(), y.clone()
    g2 = H.block_norm_bwd(dr2, dh, want[0], y2, dr=dr2, dy=y2, **kw)
    for u, v in zip(g2, g):
        assert u is None or torch.equal(u, v)


def test_zero_rows_and_no_tokens():
    d = 320
    r, y, w = rnd((4, d), BF16, 1), rnd((4, d), BF16, 2), rnd((d,), BF16, 3)
    r[1], y[1], y[2] = 0, 0, 0
    out, h, a, b = H.block_norm_fwd(r, y, post_weight=w, pre_weight=w, eps=1e-6)
    assert (out[1] == 0).all() and (h[1] == 0).all() and torch.equal(out[2], r[2])
    g = H.block_norm_bwd(rnd((4, d), BF16, 4), rnd((4, d), BF16, 5), out, y, post_weight=w,
                         pre_weight=w, rstd_post=a, rstd_pre=b)
    assert all(v is None or torch.isfinite(v).all() for v in g)
    e = torch.empty((0, d), dtype=BF16, device=DEV)
    out, h, a, b = H.block_norm_fwd(e, e, post_weight=w, pre_weight=w)
    assert out.shape == (0, d) and h.shape == (0, d) and a.numel() == 0


def test_graph_replay():
    t, d = 96, 1024
    r, y, w = rnd((t, d), BF16, 1), rnd((t, d), BF16, 2), rnd((d,), BF16, 3)
    dr, dh = rnd((t, d), BF16, 4), rnd((t, d), BF16, 5)
    gate = rnd((3, d), BF16, 6)
    ws = torch.empty(H.block_norm_bwd_workspace_bytes(t, d, 3), dtype=torch.uint8, device=DEV)

    def step():
        out, h, a, b = H.block_norm_fwd(r, y, gate=gate, post_weight=w, pre_weight=w)
        return (out, h) + H.block_norm_bwd(dr, dh, out, y, gate=gate, post_weight=w,
                                           pre_weight=w, rstd_post=a, rstd_pre=b, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(3):
        r.copy_(rnd((t, d), BF16, 20 + k))
        dh.copy_(rnd((t, d), BF16, 30 + k))
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, step()):
            assert torch.equal(u, v), k


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("t,d,groups", [(300, 8200, 1), (260, 8203, 130), (600, 9216, 600), (70, 16384, 7),
                                        (40, 12001, 0)])
def test_widest_rows(t, d, groups, dt):
    # rows that go by column strips, in place and out of place
    print(f"tokens {t} dim {d} gate rows {groups} {dt}", flush=True)
    r, y = rnd((t, d), dt, 1), rnd((t, d), dt, 2)
    gate = rnd((groups, d), dt, 3) if groups else None
    post, pre = rnd((d,), dt, 4) + 1, rnd((d,), dt, 5) + 1
    out, h, a, b = H.block_norm_fwd(r, y, gate=gate, post_weight=post, pre_weight=pre, scale=0.5)
    dr, dh = rnd((t, d), dt, 6, 0.01), rnd((t, d), dt, 7, 0.01)
    kw = dict(gate=gate, post_weight=post, pre_weight=pre, rstd_post=a, rstd_pre=b, scale=0.5)
    g = H.block_norm_bwd(dr, dh, out, y, **kw)
    ref = bwd64(dr, dh, out, y, gate, post, pre, a, b, 0.5)
    for name, v in zip(("dr", "dy", "dgate", "dpost", "dpre"), g):
        if name != "dgate" or gate is not None:
            check(v, *ref[name], dt, name)
    dr2, y2 = dr.clone(), y.clone()
    g2 = H.block_norm_bwd(dr2, dh, out, y2, dr=dr2, dy=y2, **kw)
    for u, v in zip(g2, g):
        assert u is None or torch.equal(u, v)
    only = H.block_norm_bwd(dr, dh, out, y, want_dgate=False, want_dpost=False, want_dpre=False, **kw)
    assert torch.equal(only[0], g[0]) and torch.equal(only[1], g[1]) and only[2:] == (None,) * 3


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("t,d,pad", [(2, 64, 0), (1, 1000, 0), (2, 513, 1), (3, 8193, 0), (1, 4096, 8)])
def test_an_infinite_gradient_stays_in_its_column(t, d, pad, dt):
    """An infinity in a row's incoming gradient gives that column's sums over tokens an infinity of
    its sign; the other columns' sums do not see it."""
    print(f"tokens {t} dim {d} padding {pad} {dt}", flush=True)
    col = d // 2
    r, y = rnd((t, d), dt, 1, 3.0, pad), rnd((t, d), dt, 2, 0.7, pad)
    r[0, col], y[0, col] = 2.0, 0.5
    gate, post, pre = rnd((1, d), dt, 3).abs() + 1, rnd((d,), dt, 4).abs() + 1, rnd((d,), dt, 5) + 1
    out, h, a, b = H.block_norm_fwd(r, y, gate=gate, post_weight=post, pre_weight=pre, scale=1.0,
                                    eps=1e-5)
    assert out[0, col] > 0
    for inf_in in ("dr", "dh"):
        dr, dh = rnd((t, d), dt, 6, 0.01, pad), rnd((t, d), dt, 7, 0.01)
        (dr if inf_in == "dr" else dh)[0, col] = float("inf")
        _, _, dgate, dpost, dpre = H.block_norm_bwd(
            dr, dh, out, y, gate=gate, post_weight=post, pre_weight=pre, rstd_post=a, rstd_pre=b,
            scale=1.0)
        sums = (dgate[0], dpost) if inf_in == "dr" else (dpre,)
        for v in sums:
            assert v[col] == float("inf"), inf_in
            v[col] = 0
            assert torch.isfinite(v).all(), inf_in


# Widths that give every number of waves per token there is, each with whole chunks and with rows
# that end inside one, at a prime number of tokens (the last team of a workgroup is then one too
# many), and the widest rows.  bf16: a wave holds 512 elements per chunk of its lanes, fp32 256.
WIDTHS = {BF16: [1000, 1003, 1600, 1603, 2600, 2603, 4000, 4003, 5000, 5003, 6000, 6003, 7000, 7003,
                 8000, 8192, 8191],
          F32: [500, 503, 800, 803, 1300, 1303, 2000, 2003, 2500, 2503, 3000, 3003, 3500, 3503, 4000, 4003,
                4500, 4503, 5000, 5003, 5600, 5603, 6000, 6144, 6143]}


@pytest.mark.parametrize("dt,d", [(dt, d) for dt in WIDTHS for d in WIDTHS[dt]])
def test_every_number_of_waves(d, dt):
    test_forward_and_backward(1031, d, 1, 0, dt)


@pytest.mark.parametrize("t,d,groups,dt", [(3, 32768, 1, BF16), (5, 32767, 0, BF16), (2, 20001, 2, BF16),
                                           (1100, 20000, 1, BF16), (1100, 9001, 1100, F32),
                                           (1031, 1603, 1031, BF16), (1031, 2600, 1031, F32),
                                           (2062, 800, 2, F32), (1300, 7000, 13, BF16)])
def test_widest_rows_and_groups_of_many_tokens(t, d, groups, dt):
    test_forward_and_backward(t, d, groups, 0, dt)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("post,pre", [(True, False), (False, True), (False, False), (True, True)])
@pytest.mark.parametrize("d", [1600, 1603, 830])
def test_in_place_with_a_team_too_many(d, post, pre, dt):
    # two teams of two waves in a workgroup and an odd number of tokens, r_out in r's place
    d = d // 2 if dt == F32 and d > 1000 else d
    t = 1031
    r, y = rnd((t, d), dt, 1, 3.0), rnd((t, d), dt, 2)
    wp, wq = rnd((d,), dt, 3) if post else None, rnd((d,), dt, 4) if pre else None
    want = H.block_norm_fwd(r, y, post_weight=wp, pre_weight=wq, scale=0.5)
    rout, terms, rh, ra, rb = fwd64(r, y, None, wp, wq, 0.5, 1e-6)
    check(want[0], rout, terms, dt, "r_out")
    got = H.block_norm_fwd(r, y, post_weight=wp, pre_weight=wq, scale=0.5, r_out=r, h=y if pre else None)
    for u, v in zip(got, want):
        assert (u is None and v is None) or torch.equal(u, v)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("t,d,groups", [(1, 64, 1), (2, 64, 2), (1, 1000, 1), (2, 513, 2), (3, 8193, 1),
                                        (3, 8193, 3), (1, 4096, 1), (5, 2049, 5), (9, 300, 3)])
def test_infinite_inputs_stay_in_their_sums(t, d, groups, dt):
    """An infinity in r_out, y or a weight reaches the sums whose terms hold it, with its sign, and no
    others: also where a workgroup has more teams than rows."""
    print(f"tokens {t} dim {d} gate rows {groups} {dt}", flush=True)
    col, inf = d // 2, float("inf")
    ones = torch.ones(t, dtype=torch.float32, device=DEV)
    base = dict(gate=rnd((groups, d), dt, 3).abs() + 1, post_weight=rnd((d,), dt, 4).abs() + 1,
                pre_weight=rnd((d,), dt, 5) + 1, rstd_post=ones * 0.5, rstd_pre=ones * 0.5)
    rows = dict(dr_out=rnd((t, d), dt, 6).abs() + 0.5, dh=rnd((t, d), dt, 7, 1e-4).abs() + 1e-4,
                r_out=rnd((t, d), dt, 1, 0.1), y=rnd((t, d), dt, 2).abs() + 0.5)
    for where in ("r_out", "post_weight", "gate", "rstd_pre"):
        kw = {k: v.clone() for k, v in {**base, **rows}.items()}
        (kw[where][0] if where in ("r_out", "gate") else kw[where])[col if where != "rstd_pre" else 0] = inf
        got = dict(zip(("dr", "dy", "dgate", "dpost", "dpre"), H.block_norm_bwd(scale=1.0, **kw)))
        ref = bwd64(kw["dr_out"], kw["dh"], kw["r_out"], kw["y"], kw["gate"], kw["post_weight"],
                    kw["pre_weight"], kw["rstd_post"], kw["rstd_pre"], 1.0)
        for name in ("dgate", "dpost", "dpre"):
            want = ref[name][0]
            kind = lambda v: torch.where(v.isnan(), 3, torch.where(v == inf, 2, torch.where(v == -inf, 1, 0)))
            assert torch.equal(kind(got[name].double()), kind(want)), (where, name)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("t,d", [(3, 64), (2, 1000), (3, 1003), (2, 2051), (5, 4003), (2, 6003), (2, 9001)])
def test_an_infinity_reaches_its_rows_gradient_as_the_formula_has_it(t, d, dt):
    """dr infinite in one place: the other places of dy get the infinity of the mean, not NaN, also where
    the place is an element that two chunks of a row hold."""
    print(f"tokens {t} dim {d} {dt}", flush=True)
    inf, vec = float("inf"), 8 if dt == BF16 else 4
    ones = torch.ones(t, dtype=torch.float32, device=DEV)
    base = dict(gate=rnd((1, d), dt, 3).abs() + 1, post_weight=rnd((d,), dt, 4).abs() + 1,
                pre_weight=rnd((d,), dt, 5) + 1, rstd_post=ones * 0.5, rstd_pre=ones * 0.5,
                dr_out=rnd((t, d), dt, 6).abs() + 0.5, dh=rnd((t, d), dt, 7, 1e-4),
                r_out=rnd((t, d), dt, 1, 0.1), y=rnd((t, d), dt, 2).abs() + 0.5)
    kind = lambda v: torch.where(v.isnan(), 3, torch.where(v == inf, 2, torch.where(v == -inf, 1, 0)))
    for col in (0, d // 2, max(0, d - vec), d - 1):
        kw = {k: v.clone() for k, v in base.items()}
        kw["dr_out"][0, col] = inf
        got = dict(zip(("dr", "dy", "dgate", "dpost", "dpre"), H.block_norm_bwd(scale=1.0, **kw)))
        ref = bwd64(kw["dr_out"], kw["dh"], kw["r_out"], kw["y"], kw["gate"], kw["post_weight"],
                    kw["pre_weight"], kw["rstd_post"], kw["rstd_pre"], 1.0)
        for name in ("dr", "dy", "dgate", "dpost", "dpre"):
            assert torch.equal(kind(got[name].double()), kind(ref[name][0])), (col, name)
