"""Layer gradients with stochastic codes of an fp32 dY or dz whose rows are longer than 16384."""
import numpy as np
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H
import oracle as O
import synth
from parity_util import (COUNTER64, CTR, DEV, KEY, SEED64, bound_ok, fp8_extra, rel_fro, signs_dev, to_dev,
                         to_np64)

pytestmark = pytest.mark.gpu
F32, BF16, I8, E4M3, E5M2 = (torch.float32, torch.bfloat16, torch.int8, torch.float8_e4m3fn,
                             torch.float8_e5m2)
SR = dict(grad_rounding="stochastic", seed=SEED64, counter=COUNTER64)


def rnd(shape, seed, dt=F32, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


@pytest.mark.parametrize("n,block,q,gq", [(20480, 256, "i8", "i8"), (16448, 64, "e4m3", "e5m2"),
                                          (22016, 512, "e4m3", "e4m3"), (65536, 4096, "i8", "i8")])
def test_fp32_rows_match_the_oracle(n, block, q, gq):
    code = {"i8": O.I8, "e4m3": O.E4M3, "e5m2": O.E5M2}
    tt = {"i8": I8, "e4m3": E4M3, "e5m2": E5M2}
    m, k = 5, 64
    x, w, dy = synth.layer(m, n, k, seed=n, io=synth.F32)
    sn = synth.sign_words(O.padded_len(n, block), seed=block)
    dx, _ = H.linear_bwd(to_dev(dy), to_dev(x), to_dev(w), block, tt[q], tt[gq], want_dw=False,
                         signs_n=signs_dev(sn), **SR)
    torch.cuda.synchronize()
    o = dict(signs_n=sn, grad_rounding=O.STOCHASTIC, key=KEY, ctr_hi=CTR)
    got = to_np64(dx)
    assert rel_fro(got, O.linear_bwd(dy, x, w, block, code[q], code[gq], precision=64, want_dw=False, **o)[0]) <= 1e-2
    r32 = O.linear_bwd(dy, x, w, block, code[q], code[gq], precision=32, want_dw=False, **o)[0]
    ex = 0.0
    if q != "i8":
        ex = fp8_extra(dy, O.ROWS, code[gq], w, O.COLS, code[q], block,
                       dict(signs=sn, rounding=O.STOCHASTIC, key=KEY, ctr_hi=CTR), dict(signs=sn))
    ok, bad = bound_ok(got, r32, 4 * 2.0 ** -24, ex)
    assert ok, bad


@pytest.mark.parametrize("n,q,gq", [(11008, I8, I8), (8200, E4M3, E5M2), (32768, I8, I8)])
def test_gated_layers_past_8192_wide(n, q, gq):
    # without an activation dz = [dy u, dy g] is exact to a rounding: the codes are those of linear_bwd on it
    m, k, block = 40, 64, 64
    dy, z = rnd((m, n), 1), rnd((m, 2 * n), 2)
    x, w = rnd((m, k), 3), rnd((2 * n, k), 4, scale=0.1)
    dz = torch.cat([dy * z[:, n:], dy * z[:, :n]], 1)
    dx, dw, db = H.linear_glu_bwd(dy, z, x, w, block, q, gq, activation="none", **SR)
    want = H.linear_bwd(dz, x, w, block, q, gq, **SR)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    ref = dz.double().sum(0)
    assert ((db.double() - ref).abs() <= (m + 1) * 2.0 ** -24 * dz.double().abs().sum(0)).all()
    again = H.linear_glu_bwd(dy, z, x, w, block, q, gq, activation="none", **SR)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_bf16_gated_layer_with_an_activation():
    m, n, k, block = 64, 11008, 128, 256
    dy, z = rnd((m, n), 1, BF16), rnd((m, 2 * n), 2, BF16)
    x, w = rnd((m, k), 3, BF16), rnd((2 * n, k), 4, BF16, 0.1)
    near = H.linear_glu_bwd(dy, z, x, w, block)
    got = H.linear_glu_bwd(dy, z, x, w, block, **SR)
    # a code off by less than a step of 1 / 127 of its vector's largest value instead of half of one
    for a, b in zip(got[:2], near[:2]):
        assert float((a.float() - b.float()).norm() / b.float().norm()) < 0.05
        assert not torch.equal(a, b)
    assert torch.equal(got[2], near[2]) or float((got[2].float() - near[2].float()).abs().max()
                                                 / near[2].float().abs().max()) <= 2.0 ** -7


def test_layer_with_an_activation():
    m, n, k, block = 24, 20480, 64, 128
    dy, z = rnd((m, n), 1), rnd((m, n), 2)
    x, w = rnd((m, k), 3), rnd((n, k), 4, scale=0.1)
    got = H.linear_act_bwd(dy, z, x, w, block, activation="relu", **SR)
    want = H.linear_bwd(torch.where(z > 0, dy, 0.0), x, w, block, **SR)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
