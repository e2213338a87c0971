"""The gated layer's gradient where its factors are far apart: the tail of gelu in fp32, and pairs whose
product passes the largest fp32 value behind a slope of 0."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV, BF16, F32 = "cuda", torch.bfloat16, torch.float32
U = 2.0 ** -24


def rnd(shape, dt, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dt)


@pytest.mark.parametrize("g0", [-3.0, -5.0, -8.0])
def test_gelu_tail_in_fp32(g0):
    # db of the up half is the sum over rows of dy act(g), all of one sign.  act(g) = g erfc(t) / 2, t =
    # -g / sqrt 2: two roundings of t (its factor's, its product's) move erfc by its condition number, below
    # g^2 + 1 each; erfcf is good to 4 ulp, products and the rounding add 4, the sum a step a term.
    m, n, k = 48, 64, 64
    z = rnd((m, 2 * n), F32, 1)
    z[:, :n] = g0 - 0.25 * z[:, :n].abs().clamp(max=2.0)
    dy = 1.0 + rnd((m, n), F32, 2).abs()
    x, w = rnd((m, k), F32, 3), rnd((2 * n, k), F32, 4)
    db = H.linear_glu_bwd(dy, z, x, w, 64, activation="gelu_erf")[2]
    g = z[:, :n].double()
    want = (dy.double() * g * 0.5 * torch.erfc(-g * 0.5 ** 0.5)).sum(0)
    tol = (2 * ((g0 - 0.5) ** 2 + 1) + 8 + m) * U
    off = ((db[n:].double() - want) / want).abs().max()
    print(f"relative error {float(off):.2e} of {tol:.2e}", flush=True)
    assert off <= tol


@pytest.mark.parametrize("dt,want_dw", [(BF16, True), (BF16, False), (F32, True)])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu_tanh", "gelu_erf"])
@pytest.mark.parametrize("kept", [None, torch.int8])
def test_largest_values_behind_a_slope_of_zero(dt, want_dw, act, kept):
    m, n, k = 64, 128, 64
    top = float(torch.finfo(BF16).max)  # also an fp32 value; INT8 keeps it as 127 2^121
    z = rnd((m, 2 * n), dt, 1)
    z[:, 32:64] = -500.0               # act' = 0 and act = 0 there
    z[:, n + 32:n + 64] = -top
    dy = 2.0 + rnd((m, n), dt, 2).abs()
    x, w = rnd((m, k), dt, 3), rnd((2 * n, k), dt, 4)
    if kept is not None:
        z = H.checkpoint_pack(z.view(2 * m, n), kept)
    dx, dw, db = H.linear_glu_bwd(dy, z, x, w, 64, activation=act, want_dw=want_dw)
    assert torch.isfinite(dx).all() and torch.isfinite(db).all()
    assert (db[32:64] == 0).all() and (db[n + 32:n + 64] == 0).all()
    assert dw is None or torch.isfinite(dw).all()
