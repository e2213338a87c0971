"""A layer's y has the same bits whether z is kept as it is, in 8 bits or not at all, and the kept z is the
checkpoint of the plain fp32 one: in the few-rows kernel and on every tile."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV, BF16, F32, I8, E4M3 = "cuda", torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


def rnd(shape, dt, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


# rows, columns, contraction, block: columns that end inside a group and inside a workgroup's run
SHAPES = [(1, 8, 64, 32), (1, 1024, 4096, 256), (2, 40, 512, 64), (4, 264, 2048, 128), (7, 72, 1056, 32),
          (8, 2056, 1024, 64), (16, 512, 4096, 256), (16, 24, 8192, 64), (17, 264, 512, 64),
          (203, 520, 1376, 32), (700, 1000, 256, 64), (1800, 1000, 160, 32), (3840, 1920, 224, 32)]


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("q", [I8, E4M3])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("m,n,k,block", SHAPES)
def test_y_does_not_depend_on_how_z_is_kept(m, n, k, block, dt, q, glu):
    rows = 2 * n if glu else n
    x, w, bias = rnd((m, k), dt, m + k), rnd((rows, k), dt, 2, 2.0 * k ** -0.5), rnd((rows,), dt, 3)
    kw = dict(bias=bias, activation="silu")
    if not glu:
        kw["residual"] = rnd((m, n), dt, 4)
    f = H.linear_glu_fwd if glu else H.linear_act_fwd
    y = f(x, w, block, q, **kw)
    y1, z = f(x, w, block, q, want_z=True, **kw)
    assert torch.equal(y, y1)
    if H.contraction_len(k, block) == H.padded_len(k, block):  # served on weights quantised once
        qw, sw = H.fwht_quant(w, H.ROWS, block, q)
        assert torch.equal((H.linear_glu_q if glu else H.linear_act_q)(x, qw, sw, block, **kw), y)
    for kept in (I8, E4M3):
        c = torch.full(((2 * m if glu else m) + 1, n), 3, dtype=I8, device=DEV)  # a row behind the last
        p = torch.full((c.shape[0], -(-n // 32)), 7, dtype=torch.uint8, device=DEV)
        into = H.Checkpoint(c[:-1].view(kept), p[:-1])
        y8, z8 = f(x, w, block, q, z=into, **kw)
        assert torch.equal(y8, y)
        assert (c[-1] == 3).all() and (p[-1] == 7).all()
        if dt == F32:
            want = H.checkpoint_pack(z.view(-1, n), kept)
            assert torch.equal(z8.powers, want.powers)
            assert torch.equal(bits(z8.codes), bits(want.codes))


def test_infinities_stay_in_their_groups():
    m, n, k = 5, 96, 64
    x, w = rnd((m, k), BF16, 1), rnd((2 * n, k), BF16, 2)
    bias = torch.zeros(2 * n, dtype=BF16, device=DEV)
    bias[40] = float("inf")       # gate, second group
    bias[n + 95] = float("nan")   # up, third group
    _, z = H.linear_glu_fwd(x, w, 64, bias=bias, activation="none", want_z=I8)
    lost = (z.powers == 255).view(m, 2, 3)
    want = torch.tensor([[False, True, False], [False, False, True]], device=DEV)
    assert torch.equal(lost, want.expand(m, 2, 3))
