"""Activations kept in 8 bits (checkpoint_pack, checkpoint_unpack), the forwards that write them and
the backward passes that read them.

A checkpoint is defined by exact operations (the least power of two that holds a group's largest
value, a division by it, one rounding to an integer or an E4M3 number), so codes, powers and values
are held to the definition in 64 bits without a tolerance.  What a forward keeps is the checkpoint of
its fp32 z, bit for bit, and the gradients from a checkpoint are those from the tensor it stands for:
the same fp32 dz, except that a multiply-add may be contracted in one kernel and not in another, which
moves a code in about 2^-20 of the places by one step: 1e-3 of the result in norm, as between the
forms of the plain backward."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I8, E4M3, E5M2 = (torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn,
                             torch.float8_e5m2)
U = 2.0 ** -24
QMAX = {I8: 127.0, E4M3: 448.0}
TOP = {I8: 248, E4M3: 246}


def rnd(shape, dt, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def plain(x, q):
    """Codes (as numbers), powers and values of a checkpoint of x, from the definition in 64 bits."""
    rows, cols = x.shape
    v = torch.zeros((rows, -(-cols // 32) * 32), dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    v = v.view(rows, -1, 32)
    top = v.abs().amax(2)
    lost = ~torch.isfinite(v).all(2)
    f, e = torch.frexp(torch.where(lost, 1.0, top) / QMAX[q])      # f in [0.5, 1)
    s = torch.where(top > 0, torch.where(f > 0.5, e, e - 1) + 127, 0).clamp(16, TOP[q])
    t = (v / torch.exp2(s.double() - 127)[:, :, None]).clamp(-QMAX[q], QMAX[q])
    if q == E4M3:
        quantum = torch.exp2((torch.frexp(t)[1] - 1).clamp(min=-6).double() - 3)
        t = torch.round(t / quantum) * quantum
    else:
        t = torch.round(t)
    val = t * torch.exp2(s.double() - 127)[:, :, None]
    val = torch.where(lost[:, :, None], float("nan"), val)
    s = torch.where(lost, 255, s).to(torch.uint8)
    return (t.reshape(rows, -1)[:, :cols], s, val.reshape(rows, -1)[:, :cols],
            lost[:, :, None].expand_as(t).reshape(rows, -1)[:, :cols])


def check(x, kept, q):
    codes, powers, val, lost = plain(x, q)
    assert torch.equal(kept.powers, powers)
    assert (kept.codes.double() == codes)[~lost].all()
    for dt in (BF16, F32):
        got = H.checkpoint_unpack(kept, dt).double()
        assert torch.equal(torch.isnan(got), lost)
        assert (got == val)[~lost].all()


SIZES = [(1, 1), (1, 31), (3, 32), (5, 33), (1, 4096), (2310, 2049), (700, 8), (64, 200), (33, 1000),
         (1, 100003), (4099, 40), (257, 11008), (16, 4104)]


@pytest.mark.parametrize("q", [I8, E4M3])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_pack_and_unpack(rows, cols, dt, q):
    print(f"rows {rows} cols {cols} {dt} {q}", flush=True)
    x = rnd((rows, cols), dt, 1, 3.0)
    x[:, 0] *= 30
    x[rows // 2] *= 1e-3
    check(x, H.checkpoint_pack(x, q), q)


@pytest.mark.parametrize("q", [I8, E4M3])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_values_where_it_can_go_wrong(dt, q):
    big = torch.finfo(dt).max
    rows = []
    for e in list(range(-148, 128, 7)) + [-149, -126, -127, -112, -111, -105, -104, 121, 122, 126, 127]:
        for m in (1.0, 127 / 64, 1.9921875, 1.75, 1.7578125, 1.5):   # borders of the codes' ranges
            rows.append([m * 2.0 ** e, -(2.0 ** e) * 0.3, 2.0 ** (e - 3) * 1.1] + [0.0] * 29)
    rows += [[0.0] * 32, [-0.0] * 32, [big] * 32, [-big, big / 3] * 16,
             [k + 0.5 for k in range(31)] + [127.0], [k + 0.5 for k in range(31)] + [126.0],
             [float("inf")] + [1.0] * 31, [float("-inf")] * 32, [float("nan")] + [2.0] * 31,
             [1.0] * 31 + [float("nan")], [float("nan"), float("inf")] + [0.0] * 30]
    x = torch.tensor(rows, dtype=torch.float64, device=DEV).to(F32).to(dt)
    check(x, H.checkpoint_pack(x, q), q)
    wide = x.reshape(1, -1)               # the same groups in one row
    check(wide, H.checkpoint_pack(wide, q), q)


@pytest.mark.parametrize("q", [I8, E4M3])
def test_strides_and_alignment(q):
    rows, cols = 37, 203
    want = None
    for dt in (BF16, F32):
        for pad, off in ((0, 0), (5, 1), (13, 3)):
            store = torch.full((rows, cols + pad), 9.0, dtype=dt, device=DEV).view(-1)
            x = store[off:off + rows * (cols + pad) - pad].as_strided((rows, cols), (cols + pad, 1)) \
                if off + rows * (cols + pad) - pad <= store.numel() else store.view(rows, -1)[:, :cols]
            x.copy_(rnd((rows, cols), BF16, 3, 2.0))
            codes = torch.full((rows, cols + pad), 5, dtype=torch.uint8, device=DEV).view(q)[:, :cols]
            powers = torch.full((rows, 7 + pad), 6, dtype=torch.uint8, device=DEV)
            kept = H.checkpoint_pack(x, q, out=H.Checkpoint(codes, powers[:, :7]))
            assert kept.codes is codes and (powers[:, 7:] == 6).all()
            check(x, kept, q)
            want = want or H.checkpoint_pack(x.contiguous(), q)
            assert torch.equal(kept.codes.contiguous().view(torch.uint8), want.codes.view(torch.uint8))
            back = torch.full((rows, cols + pad), 4.0, dtype=dt, device=DEV)
            H.checkpoint_unpack(kept, dt, x=back[:, :cols])
            assert torch.equal(back[:, :cols], H.checkpoint_unpack(want, dt)) and (back[:, cols:] == 4).all()


def test_streams_graph_and_empty():
    x = rnd((300, 520), BF16, 1)

    def step():
        k = H.checkpoint_pack(x)
        return k.codes, k.powers, H.checkpoint_unpack(k)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k = H.checkpoint_pack(x, stream=s)
    y = H.checkpoint_unpack(k, stream=s)
    s.synchronize()
    assert torch.equal(k.codes, want[0]) and torch.equal(y, want[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        x.copy_(rnd((300, 520), BF16, 10 + i, 2.0 ** i))
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, step()):
            assert torch.equal(u, v)
    for shape in ((0, 40), (40, 0), (0, 0)):
        k = H.checkpoint_pack(torch.empty(shape, dtype=BF16, device=DEV))
        assert k.codes.shape == shape and H.checkpoint_unpack(k).shape == shape


# few rows, waves that split the contraction, 64, 128 and 256 tiles; columns that end inside a group
@pytest.mark.parametrize("q", [I8, E4M3])
@pytest.mark.parametrize("m,n,k", [(1, 8, 32), (5, 40, 96), (16, 512, 1000), (203, 520, 1376),
                                   (400, 4096, 512), (1800, 2000, 160), (3800, 3848, 128)])
def test_forward_keeps_its_pre_activation(m, n, k, q):
    print(f"m {m} n {n} k {k} {q}", flush=True)
    for dt in (BF16, F32):
        x, w, bias = rnd((m, k), dt, 1), rnd((n, k), dt, 2, 2.0 * k ** -0.5), rnd((n,), dt, 3)
        y, z = H.linear_act_fwd(x, w, 32, bias=bias, activation="silu", want_z=q)
        y32, z32 = H.linear_act_fwd(x, w, 32, bias=bias.float(), activation="silu", want_z=True,
                                    y_dtype=F32)
        if m > 16:      # up to 16 rows another kernel writes a plain z (its product rounded before the bias)
            want = H.checkpoint_pack(z32, q)
            assert torch.equal(z.codes.view(torch.uint8), want.codes.view(torch.uint8))
            assert torch.equal(z.powers, want.powers)
            assert torch.equal(y, H.linear_act_fwd(x, w, 32, bias=bias, activation="silu"))
        else:
            val = H.checkpoint_unpack(z, F32)
            step = torch.exp2(z.powers.double() - 127).repeat_interleave(32, 1)[:, :n]
            half = 0.5 * step if q == I8 else (2.0 ** -4 * z32.double().abs() + 2.0 ** -10 * step)
            off = 10 * U * (z32.double().abs() + 2 * bias.double().abs())   # 5 roundings on each side
            assert ((val.double() - z32.double()).abs() <= half + 1.1 * off).all()
        out = H.Checkpoint(torch.empty_like(z.codes), torch.empty_like(z.powers))
        y2, z2 = H.linear_act_fwd(x, w, 32, bias=bias, activation="silu", z=out)
        assert z2 is out and torch.equal(z2.powers, z.powers)
        assert torch.equal(z2.codes.view(torch.uint8), z.codes.view(torch.uint8))


BWD = [(1, 8, 8, 8), (40, 64, 96, 32), (300, 520, 264, 64), (1000, 640, 512, 256),
       (4500, 256, 136, 128), (130, 4608, 256, 512), (256, 512, 256, 64), (4096, 64, 72, 1024),
       (8192, 200, 64, 256), (2000, 8192, 128, 128), (448, 640, 72, 64), (1000, 1000, 1000, 128)]


@pytest.mark.parametrize("act", ["none", "silu", "gelu_erf"])
@pytest.mark.parametrize("q,gq", [(I8, I8), (E4M3, E5M2), (E4M3, E4M3)])
@pytest.mark.parametrize("m,n,k,block", BWD)
def test_backward_from_checkpoints(m, n, k, block, q, gq, act):
    print(f"m {m} n {n} k {k} block {block} {q} {gq} {act}", flush=True)
    for dt, kx, kz in ((BF16, I8, E4M3), (BF16, E4M3, None), (BF16, None, I8), (F32, I8, I8)):
        x, w = rnd((m, k), dt, 1), rnd((n, k), dt, 2, k ** -0.5)
        x[:, k // 2] *= 30
        z, dy = rnd((m, n), dt, 3, 1.5), rnd((m, n), dt, 4, 1e-3)
        ck = H.checkpoint_pack(x, kx) if kx else x
        cz = H.checkpoint_pack(z, kz) if kz else z
        xv = H.checkpoint_unpack(ck, dt) if kx else x
        zv = H.checkpoint_unpack(cz, dt) if kz else z
        if act == "none":
            cz = zv = None
        want = H.linear_act_bwd(dy, zv, xv, w, block, q, gq, activation=act)
        got = H.linear_act_bwd(dy, cz, ck, w, block, q, gq, activation=act)
        for g, r, name in zip(got, want, ("dx", "dw", "db")):
            rel = float((g.double() - r.double()).norm() / r.double().norm())
            assert rel <= 1e-3, (name, rel)
        again = H.linear_act_bwd(dy, cz, ck, w, block, q, gq, activation=act)
        assert all(torch.equal(u, v) for u, v in zip(again, got))


def test_backward_options_and_parts():
    m, n, k, block = 256, 512, 264, 128
    x, w, z, dy = rnd((m, k), BF16, 1), rnd((n, k), BF16, 2), rnd((m, n), BF16, 3), rnd((m, n), BF16, 4)
    ck, cz = H.checkpoint_pack(x), H.checkpoint_pack(z, E4M3)
    xv, zv = H.checkpoint_unpack(ck), H.checkpoint_unpack(cz)
    signs = dict(signs_n=H.hadamard_signs(n, 1, DEV), signs_m=H.hadamard_signs(m, 2, DEV))
    for kw in (signs, dict(grad_rounding="stochastic", seed=9, counter=4), dict(want_dx=False),
               dict(want_dw=False), dict(want_db=False), dict(want_dx=False, want_dw=False),
               dict(want_dx=False, want_db=False)):
        for act in ("none", "relu"):        # relu's slope is exact
            want = H.linear_act_bwd(dy, zv, xv, w, block, activation=act, **kw)
            got = H.linear_act_bwd(dy, cz, ck, w, block, activation=act, **kw)
            for i, (g, r) in enumerate(zip(got, want)):
                assert (g is None) == (r is None)
                if g is not None and i < 2:
                    assert torch.equal(g, r)
                elif g is not None:      # another order of the fp32 sums
                    s = (dy.double() * ((zv.double() > 0) if act == "relu" else 1)).abs().sum(0)
                    assert ((g.double() - r.double()).abs() <= 2.0 ** -7 * r.double().abs() + 600 * U * s).all()


@pytest.mark.parametrize("kw", [dict(activation="silu"), dict(activation="silu", want_db=False),
                                dict(activation="gelu_erf", want_dw=False), dict(),
                                dict(activation="relu", want_dx=False, want_dw=False),
                                dict(activation="gelu_tanh", grad_rounding="stochastic")])
@pytest.mark.parametrize("m,n,k,block", [(300, 520, 264, 64), (4500, 256, 136, 128), (64, 128, 64, 32)])
def test_backward_in_its_own_workspace(m, n, k, block, kw):
    x, w = rnd((m, k), BF16, 1), rnd((n, k), BF16, 2, k ** -0.5)
    z, dy = H.checkpoint_pack(rnd((m, n), BF16, 3, 1.5), E4M3), rnd((m, n), BF16, 4, 1e-3)
    x = H.checkpoint_pack(x)
    need = H.linear_kept_bwd_workspace_bytes(False, m, n, k, block, z_dtype=E4M3, x_dtype=I8, **kw)
    room = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    want = H.linear_act_bwd(dy, z, x, w, block, **kw)
    got = H.linear_act_bwd(dy, z, x, w, block, workspace=room[:need], **kw)
    for u, v in zip(got, want):
        assert (u is None and v is None) or torch.equal(u, v)
    assert (room[need:] == 77).all()
    with pytest.raises(H.HaloError, match="WORKSPACE"):
        H.linear_act_bwd(dy, z, x, w, block, workspace=room[:need - 1], **kw)
