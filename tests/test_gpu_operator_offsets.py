"""Rows whose offsets pass 32 bits (elements and bytes): the last rows of a long call have the bits of
a call on those rows alone.  Where another split of a sum is allowed: two roundings to bf16
(2^-7 together), and 1e-3 for sums over tokens that cancel (at most 1024 terms below 16, of 2^-24
each)."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV, BF16 = "cuda", torch.bfloat16


def tail_only(shape, rows, seed, scale=1.0):
    """Zeros but for the last rows, which are normal: (all, the last rows)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = torch.zeros(shape, dtype=BF16, device=DEV)
    t[-rows:] = (torch.randn((rows, shape[1]), generator=g, device=DEV) * scale).to(BF16)
    return t, t[-rows:].contiguous()


def test_block_norms():
    t, d, rows = 530000, 4096, 64
    print(f"{t} x {d} bf16", flush=True)
    assert t * d > 2 ** 31
    r, rl = tail_only((t, d), rows, 1)
    y, yl = tail_only((t, d), rows, 2)
    w = torch.linspace(0.5, 1.5, d, device=DEV).to(BF16)
    kw = dict(post_weight=w, pre_weight=w, scale=0.5)
    out, h, a, b = H.block_norm_fwd(r, y, **kw)
    want = H.block_norm_fwd(rl, yl, **kw)
    # rows of the same width take another number of waves in a short call: the sums' order differs
    for got, ref in zip((out[-rows:], h[-rows:]), want):
        assert ((got.float() - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs() + 1e-6).all()
    del h
    dr, dl = tail_only((t, d), rows, 3)
    ol, al, bl = out[-rows:].contiguous(), a[-rows:].contiguous(), b[-rows:].contiguous()
    g = H.block_norm_bwd(dr, dr, out, y, rstd_post=a, rstd_pre=b, **kw)
    want = H.block_norm_bwd(dl, dl, ol, yl, rstd_post=al, rstd_pre=bl, **kw)
    assert torch.equal(g[0][-rows:], want[0]) and torch.equal(g[1][-rows:], want[1])
    for got, ref in ((g[3], want[3]), (g[4], want[4])):
        # sums over tokens, of zeros but for the last rows; another split of the rows
        assert ((got.float() - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs() + 1e-3).all()


def test_distillation():
    t, v, rows = 70000, 32000, 32
    print(f"{t} x {v} bf16", flush=True)
    assert t * v > 2 ** 31
    z, zl = tail_only((t, v), rows, 1, 3.0)
    idx = torch.arange(8, device=DEV, dtype=torch.int32).repeat(t, 1) * 3999
    tl = torch.linspace(-2, 2, 8, device=DEV).repeat(t, 1)
    w = torch.ones(t, device=DEV)
    want = H.distill_fwd_bwd(zl, idx[-rows:], tl[-rows:], w[-rows:])
    loss, lse = H.distill_fwd(z, idx, tl)
    assert torch.equal(loss[-rows:], want[0]) and torch.equal(lse[-rows:], want[1])
    assert torch.equal(H.distill_bwd(w, z, lse, idx, tl)[-rows:], want[2])
    got = H.distill_fwd_bwd(z, idx, tl, w, dlogits=z)
    assert torch.equal(got[0][-rows:], want[0]) and torch.equal(got[2][-rows:], want[2])


@pytest.mark.parametrize("block", [32, 256])   # dz stored, and formed inside the rotations
def test_layer(block):
    m, n, k, rows = 270336, 8192, 256, 1024
    print(f"{m} x {n} x {k} bf16 block {block}", flush=True)
    assert m * n > 2 ** 31 and m % 256 == 0
    x, xl = tail_only((m, k), rows, 1)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    w = (0.05 * torch.randn((n, k), generator=g, device=DEV)).to(BF16)
    bias = torch.linspace(-1, 1, n, device=DEV).to(BF16)
    y, z = H.linear_act_fwd(x, w, block, bias=bias, activation="silu", want_z=True)
    yl, zl = H.linear_act_fwd(xl, w, block, bias=bias, activation="silu", want_z=True)
    assert torch.equal(y[-rows:], yl) and torch.equal(z[-rows:], zl)
    del y
    dy, dl = tail_only((m, n), rows, 3, 0.01)
    got = H.linear_act_bwd(dy, z, x, w, block, activation="silu")
    want = H.linear_act_bwd(dl, zl, xl, w, block, activation="silu")
    # the rows before add zero codes and zero terms under the same scales
    assert torch.equal(got[0][-rows:], want[0]) and torch.equal(got[1], want[1])
    err = (got[2].float() - want[2].float()).abs()
    assert (err <= 2.0 ** -7 * want[2].float().abs() + 1e-3).all()


# HIP counts a launch's threads in 32 bits: a wave per token passes them at 2^26 tokens, 256 threads
# per token at 2^24
@pytest.mark.parametrize("t,d", [(2 ** 26 + 5, 8), (2 ** 26 + 4, 5)])
def test_more_tokens_than_a_launch_has_threads_for(t, d):
    print(f"{t} x {d} bf16", flush=True)
    r, rl = tail_only((t, d), 8, 1)
    r[:-8] = 1
    w = torch.full((d,), 2.0, dtype=BF16, device=DEV)
    out, h, a, b = H.block_norm_fwd(r, r, post_weight=w, pre_weight=w, eps=0.0)
    assert (h[:-8] == 2).all() and (out[:-8] == 3).all()
    want = H.block_norm_fwd(rl, rl, post_weight=w, pre_weight=w, eps=0.0)
    for got, ref in zip((out, h, a, b), want):
        assert torch.equal(got[-8:], ref)
    del out, h
    g = H.block_norm_bwd(r, None, r)
    assert torch.equal(g[0], r)
    del g
    idx = torch.zeros((t, 1), dtype=torch.int32, device=DEV)
    tl, one = torch.zeros((t, 1), device=DEV), torch.ones(t, device=DEV)
    want = H.distill_fwd_bwd(rl, idx[-8:], tl[-8:], one[-8:])
    loss, lse, grad = H.distill_fwd_bwd(r, idx, tl, one)
    first = H.distill_fwd_bwd(r[:1].contiguous(), idx[:1], tl[:1], one[:1])
    for got, ref, start in zip((loss, lse, grad), want, first):
        assert torch.equal(got[-8:], ref) and (got[:-8] == start).all()
    loss, lse = H.distill_fwd(r, idx, tl)
    assert torch.equal(loss[-8:], want[0]) and (loss[:-8] == first[0]).all()
    alone = H.distill_bwd(one, r, lse, idx, tl, dlogits=r)
    assert torch.equal(alone[-8:], want[2]) and (alone[:-8] == first[2]).all()


def test_more_rows_than_a_launch_has_threads_for():
    t, v = 2 ** 24 + 3, 2056
    print(f"{t} x {v} bf16", flush=True)
    z, zl = tail_only((t, v), 4, 1)
    idx = torch.zeros((t, 1), dtype=torch.int32, device=DEV)
    tl, one = torch.zeros((t, 1), device=DEV), torch.ones(t, device=DEV)
    want = H.distill_fwd_bwd(zl, idx[-4:], tl[-4:], one[-4:])
    first = H.distill_fwd_bwd(z[:1].contiguous(), idx[:1], tl[:1], one[:1])
    loss, lse, grad = H.distill_fwd_bwd(z, idx, tl, one, dlogits=z)
    assert torch.equal(grad[-4:], want[2]) and torch.equal(loss[-4:], want[0])
    assert (loss[:-4] == first[0]).all() and (lse[:-4] == first[1]).all()
    for k in range(0, t - 4, 2 ** 21):
        assert (grad[k:min(k + 2 ** 21, t - 4)] == first[2]).all()
