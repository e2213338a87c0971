"""linear_act_bwd where dz is formed in a pass of its own: with and without products, of a plain z and of the
same values kept in 8 bits, and a z that no activation reads."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV, BF16, F32, I8, E4M3 = "cuda", torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


def rnd(shape, dt, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("kept", [I8, E4M3])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu_tanh", "gelu_erf"])
@pytest.mark.parametrize("m,n,k", [(1, 8, 8), (33, 520, 96), (700, 1032, 64)])
def test_stored_dz_of_a_plain_and_of_a_kept_z(m, n, k, act, kept, dt):
    dy, x, w = rnd((m, n), dt, 1), rnd((m, k), dt, 3), rnd((n, k), dt, 4, 0.1)
    c = H.checkpoint_pack(rnd((m, n), dt, 2), kept)
    z = H.checkpoint_unpack(c, dt)
    block = 32  # below the blocks that form dz inside
    got = H.linear_act_bwd(dy, c, x, w, block, activation=act)
    want = H.linear_act_bwd(dy, z, x, w, block, activation=act)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    only = H.linear_act_bwd(dy, z, x, w, block, activation=act, want_dx=False, want_dw=False)
    assert only[0] is None and only[1] is None and torch.equal(only[2], want[2])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_a_plain_z_is_not_read_without_an_activation(dt):
    m, n, k = 96, 136, 64
    dy, w, x = rnd((m, n), dt, 1), rnd((n, k), dt, 4), rnd((m, k), dt, 3)
    z = torch.full((m, n), float("nan"), dtype=dt, device=DEV)
    for xi in (x, H.checkpoint_pack(x)):
        for got, want in zip(H.linear_act_bwd(dy, z, xi, w, 64), H.linear_act_bwd(dy, None, xi, w, 64)):
            assert torch.equal(got, want) and torch.isfinite(got).all()
    # the bias gradient alone: sums of m terms, each rounded to within half a step
    db = H.linear_act_bwd(dy, None, x, w, 64, want_dx=False, want_dw=False)[2]
    ref, mag = dy.double().sum(0), dy.double().abs().sum(0)
    eps = torch.finfo(dt).eps / 2
    assert ((db.double() - ref).abs() <= m * 2.0 ** -24 * mag + eps * ref.abs() * (1 + 1e-5)).all()
