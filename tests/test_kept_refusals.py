"""Refusals of the gated layer and of activations kept in 8 bits: every invalid call returns its
status before any HIP call (CPU only; the fake device pointers are never dereferenced), the size
queries give 0, the binding refuses tensors that do not fit, and halo_kept has the header's layout."""
import ctypes
import os
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


def kept(i, powers, dtype, off=0):
    return ctypes.byref(H.Kept(0x100000 * (i + 1) + off if i is not None else None,
                               0x100000 * (powers + 1) + 3 if powers is not None else None, dtype))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(H.LIB_PATH):
        import hadamard_rotated_precision_halo_amd.build as b
        b.build()
    return H.lib()


def call(fn, defaults, **kw):
    assert not set(kw) - set(defaults), kw
    return fn(*{**defaults, **kw}.values())


PACK = dict(x=ptr(0), xt=BF16, rows=8, cols=100, ldx=100, qt=I8, codes=ptr(1), ldc=100, powers=ptr(2, 1),
            ldp=4, stream=None)
UNPACK = dict(codes=ptr(1), qt=I8, ldc=100, powers=ptr(2, 1), ldp=4, rows=8, cols=100, x=ptr(0), xt=BF16,
              ldx=100, stream=None)


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(xt=I8)), (DTYPE, dict(xt=9)), (DTYPE, dict(qt=E5M2)), (DTYPE, dict(qt=BF16)),
    (DTYPE, dict(qt=-3)), (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=-1)), (SHAPE, dict(rows=1 << 31)),
    (SHAPE, dict(cols=1 << 31)), (SHAPE, dict(ldx=99)), (SHAPE, dict(ldc=99)), (SHAPE, dict(ldp=3)),
    (NULL, dict(x=None)), (NULL, dict(codes=None)), (NULL, dict(powers=None)), (ALIGN, dict(x=ptr(0, 1))),
    (ALIGN, dict(xt=F32, x=ptr(0, 2))), (OK, dict(rows=0, x=None, codes=None, powers=None)),
    (OK, dict(cols=0, ldx=0, ldc=0, ldp=0, x=None, codes=None, powers=None)),
])
def test_pack_and_unpack(L, status, kw):
    assert call(L.halo_checkpoint_pack, PACK, **kw) == status
    assert call(L.halo_checkpoint_unpack, UNPACK, **kw) == status


GLU_FWD = dict(x=ptr(0), w=ptr(1), io=BF16, m=32, n=64, k=128, block=64, qt=I8, y=ptr(2), yt=BF16,
               bias=ptr(3), act=2, z=kept(4, 5, I8), opts=None, ws=ptr(6), ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(io=I8)), (DTYPE, dict(qt=E5M2)), (DTYPE, dict(yt=I8)), (DTYPE, dict(yt=77)),
    (DTYPE, dict(z=kept(4, 5, E5M2))), (DTYPE, dict(z=kept(4, None, F32))), (DTYPE, dict(z=kept(4, 5, BF16))),
    (DTYPE, dict(z=kept(4, 5, 99))), (NULL, dict(z=kept(None, 5, I8))), (NULL, dict(z=kept(4, None, I8))),
    (NULL, dict(z=kept(None, None, BF16))), (ALIGN, dict(z=kept(4, 5, I8, 8))),
    (SHAPE, dict(n=60)), (SHAPE, dict(n=-64)), (SHAPE, dict(n=1 << 30)), (SHAPE, dict(m=-1)),
    (SHAPE, dict(yt=F32, n=68, z=kept(4, 5, I8))), (SHAPE, dict(k=124)), (BLOCK, dict(block=48)),
    (OPTION, dict(act=5)), (OPTION, dict(act=-1)), (ALIGN, dict(bias=ptr(3, 8))), (ALIGN, dict(y=ptr(2, 4))),
    (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(y=None)), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(ws_bytes=1024)), (ALIGN, dict(ws=ptr(6, 8))),
])
def test_glu_fwd(L, status, kw):
    assert call(L.halo_linear_glu_fwd, GLU_FWD, **kw) == status


GLU_Q = dict(x=ptr(0), io=BF16, qw=ptr(1), qt=I8, sw=ptr(2), m=32, n=64, k=128, block=64, y=ptr(3),
             yt=BF16, bias=None, act=2, signs=None, ws=ptr(4), ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(io=E4M3)), (DTYPE, dict(qt=E5M2)), (DTYPE, dict(yt=I32)), (SHAPE, dict(n=4)),
    (SHAPE, dict(n=1 << 30)), (SHAPE, dict(block=8, k=40)), (BLOCK, dict(block=0)), (OPTION, dict(act=6)),
    (NULL, dict(sw=None)), (NULL, dict(qw=None)), (ALIGN, dict(sw=ptr(2, 4))), (ALIGN, dict(bias=ptr(5, 2))),
    (ALIGN, dict(signs=ptr(5, 4))), (WORKSPACE, dict(ws_bytes=16)), (ALIGN, dict(ws=ptr(4, 8))),
    (OK, dict(m=0, x=None, y=None, ws=None)),
])
def test_glu_q(L, status, kw):
    assert call(L.halo_linear_glu_q, GLU_Q, **kw) == status


GLU_BWD = dict(dy=ptr(0), z=kept(1, 2, I8), act=2, x=kept(3, 4, E4M3), w=ptr(5), io=BF16, m=32, n=64,
               k=128, block=64, qt=I8, gqt=I8, dx=ptr(6), dw=ptr(7), db=ptr(8), opts=None, ws=ptr(9),
               ws_bytes=1 << 30, stream=None)
BWD = [
    (DTYPE, dict(io=I8)), (DTYPE, dict(qt=E5M2)), (DTYPE, dict(gqt=E5M2)), (DTYPE, dict(gqt=-1)),
    (OPTION, dict(act=9)), (NULL, dict(dy=None)), (NULL, dict(x=None)), (NULL, dict(w=None)),
    (NULL, dict(x=kept(None, 4, I8))), (NULL, dict(x=kept(3, None, I8))), (NULL, dict(z=None)),
    (NULL, dict(z=kept(1, None, E4M3))), (DTYPE, dict(x=kept(3, 4, E5M2))), (DTYPE, dict(x=kept(3, None, F32))),
    (DTYPE, dict(z=kept(1, 2, BF16))), (DTYPE, dict(z=kept(1, 2, 50))), (ALIGN, dict(x=kept(3, 4, I8, 4))),
    (ALIGN, dict(z=kept(1, 2, I8, 8))), (SHAPE, dict(n=60)), (SHAPE, dict(k=60)), (SHAPE, dict(m=0)),
    (SHAPE, dict(n=0)), (SHAPE, dict(n=1 << 30)), (BLOCK, dict(block=3)), (ALIGN, dict(db=ptr(8, 4))),
    (ALIGN, dict(dx=ptr(6, 4))), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=4096)),
    (ALIGN, dict(ws=ptr(9, 8))),
]


@pytest.mark.parametrize("status,kw", BWD)
def test_bwd(L, status, kw):
    assert call(L.halo_linear_glu_bwd, GLU_BWD, **kw) == status
    assert call(L.halo_linear_act_bwd_kept, GLU_BWD, **kw) == status


ACT_FWD = dict(x=ptr(0), w=ptr(1), io=BF16, m=32, n=64, k=128, block=64, qt=I8, y=ptr(2), yt=BF16,
               ep=None, z=kept(4, 5, I8), opts=None, ws=ptr(6), ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("status,kw", [
    (OPTION, dict(ep=ctypes.byref(H.Epilogue(None, None, 0x500000, 0)))),
    (OPTION, dict(ep=ctypes.byref(H.Epilogue(None, None, None, 7)))),
    (DTYPE, dict(z=kept(4, None, F32))), (DTYPE, dict(z=kept(4, 5, E5M2))), (NULL, dict(z=kept(4, None, E4M3))),
    (ALIGN, dict(z=kept(4, 5, I8, 4))), (SHAPE, dict(yt=F32, n=68)), (WORKSPACE, dict(ws_bytes=8)),
    (WORKSPACE, dict(z=None, ws=None)), (DTYPE, dict(qt=I32)),
])
def test_act_fwd_kept(L, status, kw):
    assert call(L.halo_linear_act_fwd_kept, ACT_FWD, **kw) == status


def test_workspace_queries(L):
    for glu, q in ((1, L.halo_linear_glu_bwd_workspace_bytes), (0, L.halo_linear_act_bwd_kept_workspace_bytes)):
        good = (32, 64, 128, 64, BF16, I8, 2, I8, E4M3, 7, 0)
        assert q(*good) >= L.halo_linear_workspace_bytes_ex(32, 64 * (1 + glu), 128, 64, I8, 1)
        for i, bad in ((0, -1), (1, -8), (1, 1 << 30), (1, -(1 << 31)), (2, -8), (3, 24), (4, I8), (4, 40),
                       (5, E5M2), (6, 5), (7, -2), (8, 33), (9, 8), (10, 2)):
            assert q(*good[:i], bad, *good[i + 1:]) == 0, (i, bad)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs the host C compiler")
def test_kept_has_the_headers_layout(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "halo.h"\nint main(void) {\n'
                   '  printf("%zu %zu %zu %zu\\n", sizeof(halo_kept), offsetof(halo_kept, data),\n'
                   '         offsetof(halo_kept, powers), offsetof(halo_kept, type));\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe)], check=True)
    out = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert out == [ctypes.sizeof(H.Kept)] + [getattr(H.Kept, f).offset for f, _ in H.Kept._fields_]


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    ck = H.Checkpoint(torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8, 2, dtype=torch.uint8))
    for f in (lambda: H.checkpoint_pack(x), lambda: H.checkpoint_unpack(ck),
              lambda: H.linear_glu_fwd(x, x, 64), lambda: H.linear_glu_bwd(x, x, x, x, 64),
              lambda: H.linear_act_bwd(x, ck, ck, x, 64)):
        with pytest.raises(ValueError, match="GPU tensor"):
            f()
    with pytest.raises(ValueError, match="Checkpoint"):
        H.checkpoint_unpack((x,))
    with pytest.raises(TypeError, match="dtype"):
        H.checkpoint_unpack((x, x))


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit():
    d = "cuda"
    bf = torch.bfloat16
    m, n, k, b = 16, 64, 128, 64
    x, w, dy = (torch.zeros(s, dtype=bf, device=d) for s in ((m, k), (2 * n, k), (m, n)))
    z = torch.zeros((m, 2 * n), dtype=bf, device=d)
    cx, cz = H.checkpoint_pack(x), H.checkpoint_pack(z.view(2 * m, n))
    H.linear_glu_bwd(dy, cz, cx, w, b)
    bad = [
        lambda: H.linear_glu_fwd(x, w[:2 * n - 1], b),
        lambda: H.linear_glu_fwd(x, w, b, z=z.view(2 * m, n)),
        lambda: H.linear_glu_fwd(x, w, b, z=H.checkpoint_pack(z)),
        lambda: H.linear_glu_fwd(x, w, b, bias=torch.zeros(n, dtype=bf, device=d)),
        lambda: H.linear_glu_fwd(x, w, b, y=torch.zeros((m, 2 * n), dtype=bf, device=d)),
        lambda: H.linear_glu_bwd(dy, H.checkpoint_pack(z), cx, w, b),
        lambda: H.linear_glu_bwd(dy, cz, H.checkpoint_pack(x[:8]), w, b),
        lambda: H.linear_glu_bwd(dy, cz, H.Checkpoint(cx.codes, cx.powers[:, :3]), w, b),
        lambda: H.linear_glu_bwd(dy, cz, H.Checkpoint(cx.codes.t(), cx.powers), w, b),
        lambda: H.linear_glu_bwd(dy, z[:, :n], x, w, b),
        lambda: H.linear_glu_bwd(dy, None, x, w, b),
        lambda: H.linear_glu_bwd(dy, cz, cx, w[:n], b),
        lambda: H.linear_act_bwd(dy, cz, cx, w[:n].contiguous(), b, activation="silu"),
        lambda: H.linear_act_bwd(z, None, H.Checkpoint(cx.codes, cx.powers.cpu()), w, b),
        lambda: H.linear_act_fwd(x, w, b, z=H.checkpoint_pack(z[:8])),
        lambda: H.checkpoint_pack(x, out=H.Checkpoint(cx.codes[:, :64], cx.powers)),
        lambda: H.checkpoint_unpack(H.Checkpoint(cx.codes, cx.powers[:8])),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("call", i, "was not refused")
    for f in (lambda: H.linear_glu_fwd(x, w, b, want_z=torch.float8_e5m2), lambda: H.checkpoint_pack(x, torch.uint8),
              lambda: H.checkpoint_pack(x.half())):
        with pytest.raises(TypeError):
            f()
