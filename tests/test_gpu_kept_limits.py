"""The gated layer and kept activations at their limits: the widest rows, columns split over many
workgroups, offsets that pass 32 bits, what lies around the outputs, infinities, calls side by side.
Tolerances are those of test_gpu_linear_glu and test_gpu_checkpoint."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H
import test_gpu_linear_glu as G

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I8, E4M3, E5M2 = (torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn,
                             torch.float8_e5m2)
rnd = G.rnd


# rows, columns of a half, contraction, block: every number of chunks a lane holds of a gated row, whole
# and shifted second parts, blocks up to a wave, and rows too wide for the pass
@pytest.mark.parametrize("m,n,k,block", [(3, 8200, 64, 128), (70, 16640, 64, 256), (65, 512, 64, 1024),
                                         (64, 16200, 64, 1024), (64, 32600, 64, 128), (130, 5504, 64, 256),
                                         (66, 7936, 64, 512), (64, 30000, 64, 512), (200, 40, 64, 64),
                                         (128, 8, 8, 64)])
@pytest.mark.parametrize("q,gq", [(I8, I8), (E4M3, E5M2)])
def test_gated_rows(m, n, k, block, q, gq):
    print(f"m {m} n {n} k {k} block {block} {q} {gq}", flush=True)
    x, w = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, k ** -0.5)
    z, dy = rnd((m, 2 * n), BF16, 3, 1.5), rnd((m, n), BF16, 4, 1e-3)
    signs = dict(signs_n=H.hadamard_signs(H.contraction_len(2 * n, block), 1, DEV),
                 signs_m=H.hadamard_signs(H.contraction_len(m, block), 2, DEV))
    for kw in ({}, signs):
        G.check_bwd(H.linear_glu_bwd(dy, z, x, w, block, q, gq, **kw), dy, z, x, w, block, q, gq, "silu",
                    BF16, **kw)
    ck, cz = H.checkpoint_pack(x, E4M3), H.checkpoint_pack(z.view(2 * m, n))
    got = H.linear_glu_bwd(dy, cz, ck, w, block, q, gq, **signs)
    G.check_bwd(got, dy, H.checkpoint_unpack(cz).view(m, 2 * n), H.checkpoint_unpack(ck), w, block, q, gq,
                "silu", BF16, **signs)


# lengths of columns between the tasks' sizes, whose last part is mostly idle, against the rows pass of
# the transpose: the codes and scales of one axis are those of the other
@pytest.mark.parametrize("rows", [64, 72, 120, 1000, 2112, 4104, 5000, 5128, 11008, 13000])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("q", [I8, E5M2])
def test_columns_of_any_length(rows, dt, q):
    for block in (16, 64, 256):   # (rows of codes start at 16 bytes)
        x = rnd((rows, 72), dt, 1)
        x[:, 3] *= 50
        signs = H.hadamard_signs(H.padded_len(rows, block), 4, DEV)
        for kw in ({}, {"signs": signs}):
            one, s1 = H.fwht_quant(x, H.COLS, block, q, **kw)
            two, s2 = H.fwht_quant(x.t().contiguous(), H.ROWS, block, q, **kw)
            assert torch.equal(one.view(torch.uint8), two.view(torch.uint8)) and torch.equal(s1, s2)
        if dt == BF16:
            kw = dict(rounding="stochastic", seed=3, counter=9)
            one, _ = H.fwht_quant(x, H.COLS, block, q, **kw)
            two, _ = H.fwht_quant(x.t().contiguous(), H.ROWS, block, q, **kw)
            assert torch.equal(one.view(torch.uint8), two.view(torch.uint8))


@pytest.mark.parametrize("q,gq", [(I8, I8), (E4M3, E5M2)])
def test_backward_when_tasks_stop_waiting(q, gq):
    """Columns split over 48 workgroups that exchange their maxima: with one poll of the bounded wait,
    tasks stop waiting and the launch behind stores their parts; the gradients are the same bits, and the
    bias gradient's sums are counted once."""
    m, n, k, block = 49152, 192, 64, 256
    x, w = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, k ** -0.5)
    z, dy = rnd((m, 2 * n), BF16, 3, 1.5), rnd((m, n), BF16, 4, 1e-3)
    ck, cz, cl = H.checkpoint_pack(x), H.checkpoint_pack(z.view(2 * m, n), E4M3), H.checkpoint_pack(z)
    dyl = rnd((m, 2 * n), BF16, 5, 1e-3)
    signs = dict(signs_m=H.hadamard_signs(m, 2, DEV))
    for kw in ({}, signs):
        for call in (lambda **o: H.linear_glu_bwd(dy, z, x, w, block, q, gq, **o),
                     lambda **o: H.linear_glu_bwd(dy, cz, ck, w, block, q, gq, **o),
                     lambda **o: H.linear_act_bwd(dyl, cl, ck, w, block, q, gq, activation="silu", **o),
                     lambda **o: H.linear_act_bwd(dyl, None, ck, w, block, q, gq, **o)):
            want = call(**kw)
            for _ in range(3):
                for u, v in zip(call(exchange_polls=1, **kw), want):
                    assert torch.equal(u, v)
    dz = G.glu_grad64(dy, z, "silu")
    db = H.linear_glu_bwd(dy, z, x, w, block, q, gq, **signs)[2]
    tol = 2.0 ** -8 * 1.01 * dz.sum(0).abs() + 2100 * 2.0 ** -24 * dz.abs().sum(0)
    assert ((db.double() - dz.sum(0)).abs() <= tol).all()


@pytest.mark.parametrize("q", [I8, E4M3])
def test_checkpoints_past_32_bits(q):
    rows, cols, last = 70000, 36000, 40
    print(f"{rows} x {cols} {q}", flush=True)
    assert rows * cols > 2 ** 31
    x = torch.zeros((rows, cols), dtype=BF16, device=DEV)
    x[-last:] = rnd((last, cols), BF16, 1, 3.0)
    kept, want = H.checkpoint_pack(x, q), H.checkpoint_pack(x[-last:], q)
    assert torch.equal(kept.codes[-last:].view(torch.uint8), want.codes.view(torch.uint8))
    assert torch.equal(kept.powers[-last:], want.powers)
    del x
    back = H.checkpoint_unpack(kept)
    assert torch.equal(back[-last:], H.checkpoint_unpack(want)) and not back[:-last].any()
    short = H.checkpoint_pack(back[:, :33], q)        # rows that start 36000 elements apart
    want = H.checkpoint_pack(back[-last:, :33].contiguous(), q)
    assert torch.equal(short.codes[-last:].view(torch.uint8), want.codes.view(torch.uint8))


def test_the_gated_layer_past_32_bits():
    m, n, k, block, last = 70000, 16384, 64, 64, 512
    print(f"m {m} n {n} k {k}", flush=True)
    assert 2 * m * n > 2 ** 31
    x, w = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, k ** -0.5)
    xl = x[-last:].contiguous()
    y, z = H.linear_glu_fwd(x, w, block, want_z=True)
    yl, zl = H.linear_glu_fwd(xl, w, block, want_z=True)
    assert torch.equal(y[-last:], yl) and torch.equal(z[-last:], zl)
    del z
    y, kz = H.linear_glu_fwd(x, w, block, want_z=I8)
    _, kl = H.linear_glu_fwd(xl, w, block, want_z=I8)
    assert torch.equal(y[-last:], yl) and torch.equal(kz.codes[-2 * last:], kl.codes)
    assert torch.equal(kz.powers[-2 * last:], kl.powers)
    # rows of dX are those of a call on these rows alone: each has its own scale
    dy = y.mul_(1e-3)
    dx = H.linear_glu_bwd(dy, kz, H.checkpoint_pack(x), w, block, want_db=False)[0]
    want = H.linear_glu_bwd(dy[-last:].contiguous(), kl, xl, w, block, want_db=False)[0]
    assert torch.equal(dx[-last:], want)


@pytest.mark.parametrize("m,n,k", [(1, 40, 96), (9, 72, 512), (40, 72, 96), (203, 2056, 512),
                                   (700, 1000, 256), (3800, 1928, 128)])
def test_nothing_around_the_outputs_is_written(m, n, k):
    def room(rows, cols, dt):
        full = torch.full((rows + 4, cols), 0.5 if dt.is_floating_point and dt != E4M3 else 7,
                          dtype=torch.uint8 if dt == E4M3 else dt, device=DEV)
        full = full.view(dt) if dt == E4M3 else full
        return full, full[2:-2]

    def clean(full):
        edge = torch.cat([full[:2], full[-2:]]).float() if full.dtype != E4M3 else \
            torch.cat([full.view(torch.uint8)[:2], full.view(torch.uint8)[-2:]]).float()
        return bool((edge == edge.flatten()[0]).all())

    x, w, dy = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, 0.1), rnd((m, n), BF16, 3)
    cols8 = 16   # rows of 16 bytes keep what is in the middle aligned
    if n % 8 == 0 and (2 * n * 2) % cols8 == 0:
        for kept in (None, I8, E4M3):
            fy, y = room(m, n, BF16)
            if kept is None:
                fz, z = room(m, 2 * n, BF16)
                full = [fy, fz]
            else:
                fc, c = room(2 * m, n, kept)
                fp, p = room(2 * m, -(-n // 32), torch.uint8)
                z, full = H.Checkpoint(c, p), [fy, fc, fp]
            if y.data_ptr() % 16 or (kept and c.data_ptr() % 16):
                continue
            H.linear_glu_fwd(x, w, 32, y=y, z=z)
            assert all(clean(f) for f in full), kept
            want = H.linear_glu_fwd(x, w, 32, want_z=True if kept is None else kept)
            assert torch.equal(y, want[0])
            fx, dx = room(m, k, BF16)
            fw, dw = room(2 * n, k, BF16)
            H.linear_glu_bwd(dy, z, x, w, 32, dx=dx, dw=dw)
            assert clean(fx) and clean(fw)
    fc, c = room(m, k, I8)
    fp, p = room(m, -(-k // 32), torch.uint8)
    H.checkpoint_pack(x, out=H.Checkpoint(c, p))
    fu, u = room(m, k, BF16)
    H.checkpoint_unpack(H.Checkpoint(c, p), x=u)
    assert clean(fc) and clean(fp) and clean(fu)


@pytest.mark.parametrize("m", [3, 40, 700])
def test_infinite_pre_activations(m):
    """A gate of infinity makes its own column infinite; kept in 8 bits its group of 32 is NaN and no
    other one."""
    n, k = 200, 64
    x, w, bias = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, 0.1), torch.zeros(2 * n, dtype=BF16, device=DEV)
    plain = H.linear_glu_fwd(x, w, 64, bias=bias, want_z=I8)
    bias[70] = float("inf")
    y, z = H.linear_glu_fwd(x, w, 64, bias=bias, want_z=I8)
    keep = torch.arange(n, device=DEV) != 70
    assert torch.equal(y[:, keep], plain[0][:, keep]) and not torch.isfinite(y[:, 70]).any()
    v, ref = H.checkpoint_unpack(z).view(m, 2 * n), H.checkpoint_unpack(plain[1]).view(m, 2 * n)
    lost = torch.zeros(2 * n, dtype=torch.bool, device=DEV)
    lost[64:96] = True
    assert torch.isnan(v[:, lost]).all() and torch.equal(v[:, ~lost], ref[:, ~lost])
    _, zp = H.linear_glu_fwd(x, w, 64, bias=bias, want_z=True)
    assert torch.isinf(zp[:, 70]).all() and torch.isfinite(zp[:, :70]).all()


def test_calls_side_by_side():
    m, n, k, block = 1000, 520, 264, 64
    x, w = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, 0.1)
    dys = [rnd((m, n), BF16, 10 + i) for i in range(2)]
    z = H.linear_glu_fwd(x, w, block, want_z=I8)[1]
    want = [H.linear_glu_bwd(d, z, x, w, block) for d in dys]
    streams = [torch.cuda.Stream() for _ in dys]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [H.linear_glu_bwd(d, z, x, w, block, stream=s) for d, s in zip(dys, streams)]
        torch.cuda.synchronize()
        for g, ref in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(g, ref))


def test_two_captured_graphs():
    # each graph has its own workspaces: replayed in turn, with eager calls between, both keep their results
    m, n, k, block = 256, 264, 128, 64
    x, w = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, 0.1)
    dys = [rnd((m, n), BF16, 10 + i) for i in range(2)]
    z = H.linear_glu_fwd(x, w, block, want_z=I8)[1]
    graphs, outs = [], []
    for d in dys:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(H.linear_glu_bwd(d, z, H.checkpoint_pack(x), w, block))
        graphs.append(g)
    for i in range(3):
        for d in dys:
            d.copy_(rnd((m, n), BF16, 30 + i))
        for g, d, out in zip(graphs, dys, outs):
            g.replay()
            torch.cuda.synchronize()
            want = H.linear_glu_bwd(d, z, H.checkpoint_pack(x), w, block)
            assert all(torch.equal(u, v) for u, v in zip(out, want))


# a product of few tiles and a long contraction beside one of many tiles and a short one, and products
# alike: both gradients of one call are those of a call for each, bit for bit
@pytest.mark.parametrize("m,n,k", [(128, 22016, 256), (1000, 14336, 512), (40, 11008, 1024), (4096, 64, 11008),
                                   (2048, 4096, 1024)])
@pytest.mark.parametrize("q,gq", [(I8, I8), (E4M3, E5M2)])
def test_both_gradients_are_each_ones(m, n, k, q, gq):
    x, w, dy = rnd((m, k), BF16, 1), rnd((n, k), BF16, 2, 0.1), rnd((m, n), BF16, 3)
    dx, dw = H.linear_bwd(dy, x, w, 64, q, gq)
    assert torch.equal(dx, H.linear_bwd(dy, x, w, 64, q, gq, want_dw=False)[0])
    assert torch.equal(dw, H.linear_bwd(dy, x, w, 64, q, gq, want_dx=False)[1])


# every tile the products run on: the same sums, so the rows of a batch are those of its parts
@pytest.mark.parametrize("n,k", [(2048, 160), (5504, 96), (504, 640)])
@pytest.mark.parametrize("q", [I8, E4M3])
def test_rows_do_not_depend_on_the_batch(n, k, q):
    w, x = rnd((2 * n, k), BF16, 2, k ** -0.5), rnd((4500, k), BF16, 1)
    qw, sw = H.fwht_quant(w, H.ROWS, 32, q)
    y, z = H.linear_glu_fwd(x, w, 32, q, want_z=True)
    for m in (1, 3, 17, 100, 203, 300, 700, 1500, 2310, 4100):
        part = H.linear_glu_fwd(x[:m].contiguous(), w, 32, q, want_z=True)
        served = H.linear_glu_q(x[:m].contiguous(), qw, sw, 32)
        if q == I8:   # integer sums
            assert torch.equal(part[0], y[:m]) and torch.equal(part[1], z[:m]) and torch.equal(served, y[:m])
        else:         # fp32 sums in another order where the contraction is split between waves
            G.check_fwd(x[:m].contiguous(), w, 32, q, "silu", None, *part, BF16)


@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_one_of_the_two_kept(act, dt):
    """x or z kept, the other plain: the gradient of the values, bit for bit as with both kept."""
    m, n, k = 260, 136, 72
    x, w, dy, z = rnd((m, k), dt, 1), rnd((n, k), dt, 2, 0.1), rnd((m, n), dt, 3), rnd((m, n), dt, 4)
    ck, cz = H.checkpoint_pack(x, E4M3), H.checkpoint_pack(z)
    xv, zv = H.checkpoint_unpack(ck, dt), H.checkpoint_unpack(cz, dt)
    # (the call with neither kept is another kernel, whose slopes may differ in the last bit of fp32:
    # test_backward_from_checkpoints compares the two)
    want = H.linear_act_bwd(dy, cz, ck, w, 64, activation=act)
    for xi, zi in ((ck, zv), (xv, cz)):
        for u, v in zip(H.linear_act_bwd(dy, zi, xi, w, 64, activation=act), want):
            assert torch.equal(u, v)
    z2 = rnd((m, 2 * n), dt, 5)
    c2 = H.checkpoint_pack(z2.view(2 * m, n))
    v2, w2 = H.checkpoint_unpack(c2, dt).view(m, 2 * n), rnd((2 * n, k), dt, 6, 0.1)
    want = H.linear_glu_bwd(dy, v2, xv, w2, 64, activation=act)
    for xi, zi in ((ck, v2), (xv, c2), (ck, c2)):
        for u, v in zip(H.linear_glu_bwd(dy, zi, xi, w2, 64, activation=act), want):
            assert torch.equal(u, v)


# few rows of narrow and wide layers: the kernel that reads the codes straight, and the tiles
@pytest.mark.parametrize("m", [1, 3, 5, 9, 16])
@pytest.mark.parametrize("n,k", [(4088, 640), (4096, 640), (4104, 9216)])
@pytest.mark.parametrize("q", [I8, E4M3])
def test_few_rows_of_wide_layers(m, n, k, q):
    x, w, bias = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2, k ** -0.5), rnd((2 * n,), BF16, 3, 0.1)
    y, z = H.linear_glu_fwd(x, w, 64, q, bias=bias, want_z=True)
    G.check_fwd(x, w, 64, q, "silu", bias, y, z, BF16)
    qw, sw = H.fwht_quant(w, H.ROWS, 64, q)
    served = H.linear_glu_q(x, qw, sw, 64, bias=bias)
    G.check_fwd(x, w, 64, q, "silu", bias, served, z, BF16)
    assert torch.equal(served, y)
