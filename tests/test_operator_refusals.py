"""Refusals of the block norms, the layer with its epilogue and the distillation loss: every
invalid call returns its status before any HIP call (CPU only; the fake device pointers are never
dereferenced), the size queries give 0, and halo_epilogue has the header's layout."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, BLOCK, DTYPE, ALIGN, WORKSPACE, HIP, OPTION = range(9)
F32, BF16, I8, E4M3, E5M2, I32 = range(6)


def ptr(i, off=0):
    return ctypes.c_void_p(0x100000 * (i + 1) + off)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(H.LIB_PATH):
        import hadamard_rotated_precision_halo_amd.build as b
        b.build()
    return H.lib()


def call(fn, defaults, **kw):
    assert not set(kw) - set(defaults), kw
    return fn(*{**defaults, **kw}.values())


NORM_FWD = dict(r=ptr(0), ldr=64, y=ptr(1), ldy=64, gate=ptr(2), ldg=64, groups=2, post=ptr(3),
                pre=ptr(4), io=BF16, tokens=8, dim=64, scale=1.0, eps=1e-6, r_out=ptr(5), ldro=64,
                h=ptr(6), ldh=64, rstd_post=ptr(7), rstd_pre=ptr(8), stream=None)
NORM_BWD = dict(dr_out=ptr(0), lddro=64, dh=ptr(1), lddh=64, r_out=ptr(2), ldro=64, y=ptr(3),
                ldy=64, gate=ptr(4), ldg=64, groups=2, post=ptr(5), pre=ptr(6), rstd_post=ptr(7),
                rstd_pre=ptr(8), io=F32, tokens=8, dim=64, scale=1.0, dr=ptr(9), lddr=64,
                dy=ptr(10), lddy=64, dgate=ptr(11), dpost=ptr(12), dpre=ptr(13), ws=ptr(14),
                ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(io=I8)), (DTYPE, dict(io=17)), (DTYPE, dict(io=-1)),
    (SHAPE, dict(tokens=-1)), (SHAPE, dict(tokens=7)), (SHAPE, dict(groups=0)),
    (SHAPE, dict(groups=16)), (SHAPE, dict(dim=0)), (SHAPE, dict(dim=32769)),
    (SHAPE, dict(io=F32, dim=16385)), (SHAPE, dict(tokens=1 << 31)), (SHAPE, dict(ldr=63)),
    (SHAPE, dict(ldy=63)), (SHAPE, dict(ldg=63)), (SHAPE, dict(ldro=63)), (SHAPE, dict(ldh=63)),
    (OPTION, dict(eps=-1e-6)), (OPTION, dict(eps=float("nan"))),
    (NULL, dict(r=None)), (NULL, dict(r_out=None)), (NULL, dict(h=None)), (NULL, dict(y=None)),
    (NULL, dict(pre=None)), (NULL, dict(post=None)),
    (NULL, dict(y=None, gate=None, post=None, r_out=None, rstd_post=None, pre=None, h=None,
                rstd_pre=None)),
    (ALIGN, dict(r=ptr(0, 1))), (ALIGN, dict(io=F32, h=ptr(6, 2))), (ALIGN, dict(rstd_pre=ptr(8, 2))),
])
def test_block_norm_fwd(L, status, kw):
    assert call(L.halo_block_norm_fwd, NORM_FWD, **kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(io=E4M3)), (SHAPE, dict(tokens=0, groups=1)), (SHAPE, dict(tokens=9)),
    (SHAPE, dict(dim=16385)), (SHAPE, dict(lddro=63)), (SHAPE, dict(lddh=63)),
    (SHAPE, dict(ldro=63)), (SHAPE, dict(ldy=63)), (SHAPE, dict(lddr=63)), (SHAPE, dict(lddy=63)),
    (SHAPE, dict(ldg=63)), (NULL, dict(dr=None)), (NULL, dict(dy=None)), (NULL, dict(y=None)),
    (NULL, dict(dh=None)), (NULL, dict(r_out=None)), (NULL, dict(rstd_pre=None)),
    (NULL, dict(rstd_post=None)), (NULL, dict(gate=None)), (NULL, dict(post=None)),
    (NULL, dict(pre=None)), (NULL, dict(dr_out=None, dh=None, pre=None, dpre=None)),
    (ALIGN, dict(dr=ptr(9, 2))), (ALIGN, dict(ws=ptr(14, 8))), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(ws_bytes=16)),
])
def test_block_norm_bwd(L, status, kw):
    assert call(L.halo_block_norm_bwd, NORM_BWD, **kw) == status


def test_block_norm_workspace(L):
    q = L.halo_block_norm_bwd_workspace_bytes
    assert q(8, 64, 2, F32) > 0
    for bad in ((8, 64, 3, F32), (0, 64, 1, F32), (8, 0, 1, F32), (8, 64, 0, F32), (8, 64, 2, I8),
                (8, 16385, 2, F32), (8, 64, 2, 99), (-8, 64, 2, F32)):
        assert q(*bad) == 0, bad


DISTILL = dict(logits=ptr(0), lt=BF16, ldl=1000, idx=ptr(1), ldi=16, tl=ptr(2), tt=F32, ldt=16)
D_TAIL = dict(tokens=4, vocab=1000, top=16, temperature=2.0)
FWD = {**DISTILL, **D_TAIL, "loss": ptr(3), "lse": ptr(4), "stream": None}
BWD = {"dloss": ptr(5), "logits": ptr(0), "lt": BF16, "ldl": 1000, "lse": ptr(4), "idx": ptr(1),
       "ldi": 16, "tl": ptr(2), "tt": F32, "ldt": 16, **D_TAIL, "dlogits": ptr(6), "ldd": 1000,
       "stream": None}
BOTH = {**DISTILL, "dloss": ptr(5), **D_TAIL, "loss": ptr(3), "lse": ptr(4), "dlogits": ptr(6),
        "ldd": 1000, "stream": None}
COMMON = [(DTYPE, dict(lt=I8)), (DTYPE, dict(tt=I32)), (DTYPE, dict(lt=55)),
          (SHAPE, dict(tokens=-1)), (SHAPE, dict(vocab=0)), (SHAPE, dict(vocab=1 << 31)),
          (SHAPE, dict(top=0)), (SHAPE, dict(top=1025, ldi=2000, ldt=2000)), (SHAPE, dict(ldl=999)),
          (SHAPE, dict(ldi=15)), (SHAPE, dict(ldt=15)), (OPTION, dict(temperature=0.0)),
          (OPTION, dict(temperature=-1.0)), (OPTION, dict(temperature=float("nan"))),
          (OPTION, dict(temperature=float("inf"))), (OPTION, dict(temperature=1e-39)),
          (NULL, dict(logits=None)), (NULL, dict(idx=None)), (NULL, dict(tl=None)),
          (ALIGN, dict(logits=ptr(0, 1))), (ALIGN, dict(idx=ptr(1, 2))), (ALIGN, dict(tl=ptr(2, 2)))]


@pytest.mark.parametrize("status,kw", COMMON)
def test_distill_shared(L, status, kw):
    assert call(L.halo_distill_fwd, FWD, **kw) == status
    assert call(L.halo_distill_bwd, BWD, **kw) == status
    assert call(L.halo_distill_fwd_bwd, BOTH, **kw) == status


def test_distill_own(L):
    assert call(L.halo_distill_fwd, FWD, loss=None) == NULL
    assert call(L.halo_distill_fwd, FWD, loss=ptr(3, 2)) == ALIGN
    for fn, d in ((L.halo_distill_bwd, BWD), (L.halo_distill_fwd_bwd, BOTH)):
        assert call(fn, d, dloss=None) == NULL
        assert call(fn, d, dlogits=None) == NULL
        assert call(fn, d, ldd=999) == SHAPE
        assert call(fn, d, dlogits=ptr(0), ldd=1008) == SHAPE   # in place needs one stride
        assert call(fn, d, dlogits=ptr(6, 1)) == ALIGN
    assert call(L.halo_distill_bwd, BWD, lse=None) == NULL
    assert call(L.halo_distill_fwd_bwd, BOTH, loss=None) == NULL


def ep(**kw):
    return ctypes.byref(H.Epilogue(kw.get("bias"), kw.get("residual"), kw.get("z"),
                                   kw.get("activation", 0)))


ACT_FWD = dict(x=ptr(0), w=ptr(1), io=BF16, m=64, n=128, k=256, block=64, q=I8, y=ptr(2), yt=BF16,
               ep=None, opts=None, ws=ptr(3), ws_bytes=1 << 30, stream=None)
ACT_Q = dict(x=ptr(0), io=BF16, qw=ptr(1), q=I8, sw=ptr(4), m=64, n=128, k=256, block=64, y=ptr(2),
             yt=BF16, ep=None, signs=None, ws=ptr(3), ws_bytes=1 << 30, stream=None)
ACT_BWD = dict(dy=ptr(0), z=ptr(1), act=2, x=ptr(2), w=ptr(3), io=BF16, m=64, n=128, k=256,
               block=64, q=I8, gq=I8, dx=ptr(4), dw=ptr(5), db=ptr(6), opts=None, ws=ptr(7),
               ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(io=I8)), (DTYPE, dict(q=E5M2)), (DTYPE, dict(yt=I32)), (DTYPE, dict(yt=-3)),
    (SHAPE, dict(m=-1)), (SHAPE, dict(k=0)), (SHAPE, dict(k=12)), (BLOCK, dict(block=48)),
    (ALIGN, dict(n=100)), (ALIGN, dict(x=ptr(0, 8))), (ALIGN, dict(y=ptr(2, 8))),
    (OPTION, dict(ep=ep(activation=5))), (OPTION, dict(ep=ep(activation=-1))),
    (ALIGN, dict(ep=ep(bias=ptr(8, 2)))), (ALIGN, dict(ep=ep(residual=ptr(8, 4)))),
    (ALIGN, dict(ep=ep(z=ptr(8, 8)))), (NULL, dict(x=None)), (NULL, dict(y=None)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=100)), (ALIGN, dict(ws=ptr(3, 8))),
])
def test_linear_act_forward(L, status, kw):
    assert call(L.halo_linear_act_fwd, ACT_FWD, **kw) == status
    assert call(L.halo_linear_act_q, ACT_Q, **kw) == status


def test_linear_act_q_own(L):
    assert call(L.halo_linear_act_q, ACT_Q, sw=None) == NULL
    assert call(L.halo_linear_act_q, ACT_Q, qw=None) == NULL
    assert call(L.halo_linear_act_q, ACT_Q, sw=ptr(4, 4)) == ALIGN
    assert call(L.halo_linear_act_q, ACT_Q, signs=ptr(5, 4)) == ALIGN
    assert call(L.halo_linear_act_q, ACT_Q, k=40, block=8) == SHAPE   # 40 codes: not a multiple of 32
    assert L.halo_linear_act_q_workspace_bytes(64, 256, 64) >= 64 * 256 + 64 * 4
    for bad in ((-1, 256, 64), (64, -1, 64), (64, 256, 48)):
        assert L.halo_linear_act_q_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(io=E4M3)), (DTYPE, dict(gq=E5M2)), (DTYPE, dict(q=F32)), (OPTION, dict(act=5)),
    (OPTION, dict(act=-1)), (NULL, dict(dy=None)), (NULL, dict(x=None)), (NULL, dict(w=None)),
    (NULL, dict(z=None)), (SHAPE, dict(m=0)), (SHAPE, dict(n=12)), (SHAPE, dict(k=4)),
    (BLOCK, dict(block=0)), (ALIGN, dict(z=ptr(1, 8))), (ALIGN, dict(db=ptr(6, 2))),
    (ALIGN, dict(dx=ptr(4, 2))), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=1000)),
    (ALIGN, dict(ws=ptr(7, 4))),
])
def test_linear_act_backward(L, status, kw):
    assert call(L.halo_linear_act_bwd, ACT_BWD, **kw) == status


def test_linear_act_backward_workspace(L):
    q = L.halo_linear_act_bwd_workspace_bytes
    assert q(64, 128, 256, 64, I8) > L.halo_linear_workspace_bytes_ex(64, 128, 256, 64, I8, 1)
    for bad in ((-1, 128, 256, 64, I8), (64, 128, 256, 3, I8), (64, 128, 256, 64, F32)):
        assert q(*bad) == 0


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs the host C compiler")
def test_epilogue_layout(tmp_path):
    fields = [f for f, _ in H.Epilogue._fields_]
    text = open(os.path.join(ROOT, "include", "halo.h"), encoding="utf-8").read()
    body = re.search(r"typedef struct \{([^{}]*)\} halo_epilogue;", text).group(1)
    assert re.findall(r"(\w+)\s*;", re.sub(r"/\*.*?\*/", "", body, flags=re.S)) == fields
    enum = re.search(r"typedef enum \{([^{}]*)\} halo_activation;", text).group(1)
    values = {a.lower(): int(v) for a, v in re.findall(r"HALO_ACT_(\w+) = (\d+)", enum)}
    assert values == H.ACTIVATIONS
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include "halo.h"\nint main(void) {\n'
                   + "".join(f'printf("%zu\\n", offsetof(halo_epilogue, {f}));\n' for f in fields)
                   + 'printf("%zu\\n", sizeof(halo_epilogue));\nreturn 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout
    assert [int(v) for v in out.split()] == [getattr(H.Epilogue, f).offset for f in fields] \
        + [ctypes.sizeof(H.Epilogue)]


def test_the_binding_wants_gpu_tensors():
    r = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    f = torch.zeros(4, 2)
    for fn in (lambda: H.block_norm_fwd(r, r, pre_weight=w[0]), lambda: H.block_norm_bwd(r, r, r),
               lambda: H.linear_act_fwd(r, w, 64), lambda: H.linear_act_q(r, w, w[0], 64),
               lambda: H.linear_act_bwd(r, r, r, w, 64), lambda: H.distill_fwd(r, i, f)):
        with pytest.raises(ValueError):
            fn()
    with pytest.raises(TypeError):
        H.block_norm_fwd(r.half())


@pytest.mark.gpu
def test_the_binding_refuses():
    dev, bf = "cuda", torch.bfloat16
    r, w = torch.zeros(4, 64, dtype=bf, device=dev), torch.zeros(64, 64, dtype=bf, device=dev)
    v, g3 = torch.zeros(64, dtype=bf, device=dev), torch.zeros(3, 64, dtype=bf, device=dev)
    i, f = torch.zeros(4, 2, dtype=torch.int32, device=dev), torch.zeros(4, 2, device=dev)
    one = torch.zeros(4, device=dev)
    q, s = torch.zeros(64, 64, dtype=torch.int8, device=dev), torch.zeros(64, device=dev)
    bad = [lambda: H.block_norm_fwd(r, r[:3], pre_weight=v), lambda: H.block_norm_fwd(r, r.float()),
           lambda: H.block_norm_fwd(r, r.t().contiguous().t()), lambda: H.block_norm_fwd(r, gate=v),
           lambda: H.block_norm_fwd(r, r, post_weight=v[:63]), lambda: H.block_norm_fwd(r, h=r),
           lambda: H.block_norm_fwd(r, r, r_out=r[:, :32]), lambda: H.block_norm_bwd(r, r, r),
           lambda: H.block_norm_bwd(r, None, r, post_weight=v),
           lambda: H.block_norm_bwd(None, r, r, pre_weight=v, rstd_pre=one[:2]),
           lambda: H.distill_fwd(r, i.long(), f), lambda: H.distill_fwd(r, i[:2], f),
           lambda: H.distill_bwd(one.to(bf), r, one, i, f),
           lambda: H.distill_fwd_bwd(r, i, f, one, dlogits=r.float()),
           lambda: H.linear_act_fwd(r, w, 64, activation="tanh"),
           lambda: H.linear_act_fwd(r, w[:, :32], 64), lambda: H.linear_act_fwd(r, w, 64, bias=v[:8]),
           lambda: H.linear_act_fwd(r, w, 64, residual=r.float()),
           lambda: H.linear_act_q(r, q[:, :32], s, 64), lambda: H.linear_act_q(r, q, s[:5], 64),
           lambda: H.linear_act_bwd(r, None, r, w, 64, activation="silu"),
           lambda: H.linear_act_bwd(r, r, r, w[:32], 64),
           lambda: H.linear_act_q(r, q, s, 64, workspace=one)]
    for k, fn in enumerate(bad):
        with pytest.raises(ValueError):
            fn()
            print("accepted", k)
    with pytest.raises(TypeError):
        H.linear_act_q(r, q.to(torch.int32), s, 64)
    with pytest.raises(H.HaloError):
        H.block_norm_fwd(r, r, gate=g3)                      # three gate rows for four tokens
    with pytest.raises(H.HaloError):
        H.distill_fwd(r, i, f, temperature=0.0)
    with pytest.raises(H.HaloError):
        H.linear_act_q(r, q, s, 64, workspace=torch.zeros(16, dtype=torch.uint8, device=dev))


@pytest.mark.gpu
def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch):
    """A call given a stream allocates its outputs and workspaces on that stream: memory of another
    stream could be handed on while the call's kernels still use it."""
    import torch
    dev, bf = torch.device("cuda", torch.cuda.current_device()), torch.bfloat16
    r, w, v = (torch.ones(s, dtype=bf, device=dev) for s in ((40, 64), (32, 64), (64,)))
    f, dloss = torch.zeros((40, 4), device=dev), torch.ones(40, device=dev)
    i = torch.arange(4, dtype=torch.int32, device=dev).repeat(40, 1)
    one = torch.ones(40, device=dev)
    dy = torch.ones((40, 32), dtype=bf, device=dev)
    q, s = H.fwht_quant(w, H.ROWS, 64)
    calls = [lambda **k: H.block_norm_fwd(r, r, post_weight=v, pre_weight=v, **k),
             lambda **k: H.block_norm_bwd(r, r, r, r, v, v, v, one, one, **k),
             lambda **k: H.distill_fwd(r, i, f, **k),
             lambda **k: H.distill_bwd(dloss, r, one, i, f, **k),
             lambda **k: H.distill_fwd_bwd(r, i, f, dloss, **k),
             lambda **k: H.linear_act_fwd(r, w, 64, want_z=True, activation="silu", **k),
             lambda **k: H.linear_act_q(r, q, s, 64, **k),
             lambda **k: H.linear_act_bwd(dy, dy, r, w, 64, activation="silu", **k)]
    side, at = torch.cuda.Stream(), []
    for name in ("empty", "empty_like"):
        def spy(*a, real=getattr(torch, name), **k):
            at.append(torch.cuda.current_stream(dev).cuda_stream)
            return real(*a, **k)
        monkeypatch.setattr(torch, name, spy)
    for n, call in enumerate(calls):
        want = call()
        side.wait_stream(torch.cuda.current_stream())
        at.clear()
        got = call(stream=side)
        assert at and set(at) == {side.cuda_stream}, n
        side.synchronize()
        one_or_more = lambda o: o if isinstance(o, tuple) else (o,)
        for a, b in zip(one_or_more(got), one_or_more(want)):
            assert (a is None and b is None) or torch.equal(a, b), n
        with pytest.raises(ValueError):
            call(stream=side.cuda_stream)


def test_workspace_of_an_empty_layer(L):
    # no rows, no outputs, no contraction: sizes, not a division by zero
    q = L.halo_linear_act_bwd_workspace_bytes
    for m, n, k in ((0, 128, 64), (64, 0, 64), (64, 128, 0), (0, 0, 0)):
        assert q(m, n, k, 64, I8) == L.halo_linear_workspace_bytes_ex(m, n, k, 64, I8, 1) \
            + (0 if m == 0 or n == 0 else 64 * 128 * 4 + 4 * 128 * 4)
        assert L.halo_linear_act_q_workspace_bytes(m, k, 64) == 64 * ((m * k + 255) // 256 * 4) \
            + (m * 4 + 255) // 256 * 256
    assert L.halo_block_norm_bwd_workspace_bytes(0, 64, 1, BF16) == 0
    assert L.halo_block_norm_bwd_workspace_bytes(4, 0, 1, BF16) == 0
    assert L.halo_block_norm_bwd_workspace_bytes(4, 64, 0, BF16) == 0


def test_workspace_of_a_gradients_own_form(L):
    """What a call must bring: the layer's workspace, a stored dz only where the rotation passes do not
    form it, partial rows only for a bias gradient."""
    every, own = L.halo_linear_act_bwd_workspace_bytes, L.halo_linear_act_bwd_workspace_bytes_ex
    m, n, k, silu, none = 512, 1024, 256, 2, 0
    layer = L.halo_linear_workspace_bytes_ex(m, n, k, 128, I8, 1)
    dz, parts = m * n * 4, 32 * n * 4      # 32 runs of 16 rows
    for q in (I8, E4M3):
        assert every(m, n, k, 128, q) == layer + dz + parts
        assert own(m, n, k, 128, BF16, q, silu, 7, 0) == layer + parts            # inside the passes
        assert own(m, n, k, 128, BF16, q, silu, 3, 0) == layer
        assert own(m, n, k, 128, BF16, q, none, 7, 0) == layer + parts
        assert own(m, n, k, 128, BF16, q, none, 3, 0) == layer
        for form in ((128, BF16, q, silu, 5, 0), (128, BF16, q, silu, 6, 0), (128, F32, q, silu, 7, 0),
                     (128, BF16, q, silu, 7, 1), (32, BF16, q, silu, 7, 0)):
            assert own(m, n, k, *form) == L.halo_linear_workspace_bytes_ex(m, n, k, form[0], q, 1) \
                + dz + parts, form
    for bad in ((BF16, F32, silu, 7, 0), (I8, I8, silu, 7, 0), (BF16, I8, 9, 7, 0), (BF16, I8, silu, 8, 0),
                (BF16, I8, silu, -1, 0), (BF16, I8, silu, 7, 2)):
        assert own(m, n, k, 128, *bad) == 0
    assert own(m, n, k, 3, BF16, I8, silu, 7, 0) == 0 and own(m, -1, k, 128, BF16, I8, silu, 7, 0) == 0
    assert own(m, 0, k, 128, BF16, I8, silu, 7, 0) > 0
    # a smaller one is refused, before anything is launched
    small = layer + parts - 1
    assert call(L.halo_linear_act_bwd, ACT_BWD, m=m, n=n, k=k, block=128, act=silu,
                ws_bytes=small) == WORKSPACE


def test_status_strings_name_the_operators_options(L):
    text = L.halo_status_str(OPTION).decode()
    for word in ("rounding", "activation", "eps", "temperature"):
        assert word in text
    assert "element" in L.halo_status_str(ALIGN).decode()   # rows of the row operators start anywhere
