"""The bounded wait of the gradients from kept activations: with a limit of one poll some task of the columns
pass in question does stop waiting, and the launch behind it stores the strip's parts: the gradients keep
their bits.

Columns of 49152 rows are split over 48 workgroups a strip, and the shapes let one strip straddle the first
256 workgroups (one per compute unit), so that its first tasks arrive a task's time before the rest can
start.  The wait is bounded and every task ends by itself."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV, BF16, I8, E4M3, E5M2 = "cuda", torch.bfloat16, torch.int8, torch.float8_e4m3fn, torch.float8_e5m2
M, BLOCK, ATTEMPTS = 49152, 256, 10


def rnd(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF16)


def late_words(n, k):
    """Byte offsets of the counts of late tasks of dY's and X's columns passes in the workspace (n: columns
    of dz); W's columns are whole."""
    r = lambda v: (v + 255) // 256 * 256  # noqa: E731
    nq = H.contraction_len(n, BLOCK)
    assert nq <= 4096 and M % BLOCK == 0
    codes = r(M * nq) + r(4 * M) + r(k * nq) + r(4 * k) + r(n * M) + r(4 * n) + r(k * M) + r(4 * k)
    strips = -(-n // 64)
    return codes, codes + r(256 + r(4 * strips) + 4 * n)


FORMS = ["gated", "gated from 8 bits", "layer from 8 bits", "x in 8 bits"]


# which pass straddles the first wave, columns of dz, columns of x: W's columns are 1 task (2 of k = 192),
# dY's 48 for every 64 columns: strip 5 of dY's is tasks 241 to 288, strip 2 of X's 242 to 289
@pytest.mark.parametrize("which,n,k", [("dy", 384, 64), ("x", 192, 192)])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("q,gq", [(I8, I8), (E4M3, E5M2)])
def test_late_tasks_are_repaired(form, q, gq, which, n, k):
    x, w, z = rnd((M, k), 1), rnd((n, k), 2, k ** -0.5), rnd((M, n), 3, 1.5)
    ck = H.checkpoint_pack(x)
    kw = dict(signs_m=H.hadamard_signs(M, 2, DEV))
    glu, act = form.startswith("gated"), "none" if form == "x in 8 bits" else "silu"
    if glu:
        dy, cz = rnd((M, n // 2), 4, 1e-3), H.checkpoint_pack(z.view(2 * M, n // 2), E4M3)
        a = (dy, z, x) if form == "gated" else (dy, cz, ck)
        f = H.linear_glu_bwd
    else:
        dy = rnd((M, n), 4, 1e-3)
        a = (dy, None if act == "none" else H.checkpoint_pack(z), ck)
        f = H.linear_act_bwd
    want = f(*a, w, BLOCK, q, gq, activation=act, **kw)
    kept_z, kept_x = isinstance(a[1], tuple), isinstance(a[2], tuple)
    need = H.linear_kept_bwd_workspace_bytes(
        glu, M, dy.shape[1], k, BLOCK, q, activation=act, z_dtype=a[1].codes.dtype if kept_z else None,
        x_dtype=a[2].codes.dtype if kept_x else None)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    at = late_words(n, k)[which == "x"]
    late = 0
    for attempt in range(ATTEMPTS):
        got = f(*a, w, BLOCK, q, gq, activation=act, exchange_polls=1, workspace=ws, **kw)
        for u, v in zip(got, want):
            assert torch.equal(u, v), f"call {attempt}"
        late = int(ws[at:at + 4].view(torch.int32).item())
        if late:
            break
    print(f"call {attempt}: {late} tasks stopped waiting", flush=True)
    assert 0 < late <= 48 * 8, f"no task stopped waiting in {ATTEMPTS} calls"
    got = f(*a, w, BLOCK, q, gq, activation=act, workspace=ws, **kw)
    assert int(ws[at:at + 4].view(torch.int32).item()) == 0
    for u, v in zip(got, want):
        assert torch.equal(u, v)
