"""The distillation loss over a teacher's top logits and its gradient against the formula in 64
bits.

Tolerances, in units of u = 2^-24.  lse: the logits scaled by 1 / temperature carry 3 u |z| each
(the factor, the product, the maximum they are compared with), a row's sum of exponentials has a
chain of at most 256 additions, each exponential 8 u.  p: the same with the teacher's logits.  The
loss adds (|log p| + |z| + |lse|) u per entry.  A gradient element is off by its exponent's error,
relative, plus its rounding to the output type."""
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF16, F32 = torch.bfloat16, torch.float32


def ref64(logits, idx, tl, tau, dloss=None, lse=None):
    """Loss, lse, gradient in 64 bits and the tolerances of each."""
    z, v = logits.double() / tau, logits.shape[1]
    there = (idx >= 0) & (idx < v)
    u = torch.where(there, tl.double() / tau, float("-inf"))
    zmax = torch.where(z.isinf(), 0.0, z).abs().amax(1)
    own = torch.logsumexp(z, 1)
    lse_tol = U * (4 * zmax + 300 + 8)
    if lse is not None:
        own, lse_tol = lse.double(), torch.zeros_like(lse_tol)
    dead = (own == float("-inf")) | (u == float("-inf")).all(1)
    p = torch.softmax(torch.where(dead[:, None], 0.0, u), 1) * there
    at = idx.clamp(0, v - 1).long()
    logp = torch.where(p > 0, p, 1.0).log()
    zk = z.gather(1, at)
    term = torch.where((p > 0) & ~dead[:, None], p * (logp - zk + own[:, None]), 0.0)
    loss = tau ** 2 * term.sum(1)
    umax = torch.where(u.isinf(), 0.0, u).abs().amax(1)
    p_tol = U * (64 + 8 * umax + idx.shape[1] / 4)
    size = torch.where(p > 0, p * (logp.abs() + zk.abs() + own.abs()[:, None] + 1), 0.0).sum(1)
    loss_tol = tau ** 2 * (lse_tol + (p_tol + 8 * U) * size)
    out = [loss, torch.where(dead, 0.0, loss_tol), own, lse_tol]
    if dloss is not None:
        by = torch.where(dead | (dloss == 0), 0.0, dloss.double() * tau)[:, None]
        zz = torch.where(by == 0, 0.0, z)
        q = torch.exp(zz - torch.where(by[:, 0] == 0, 0.0, own)[:, None])
        spread = torch.zeros_like(q).scatter_add_(1, at, torch.where(there, p, 0.0))
        grad = by * (q - spread)
        e = U * (4 * torch.where(zz.isinf(), 0.0, zz).abs() + 4 * own.abs()[:, None].nan_to_num(0, 0, 0) + 16) + lse_tol[:, None]
        tol = by.abs() * (q * e + spread * p_tol[:, None]) + ROUND[logits.dtype] * 1.01 * grad.abs() + 1e-37
        out += [grad, tol]
    return out


def make(t, v, k, dt, seed, tdt=F32, pad=0, missing=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    full = (2.5 * torch.randn((t, v + pad), generator=g, device=DEV)).to(dt)
    logits = full[:, :v] if pad else full
    idx = torch.randint(0, v, (t, k), generator=g, device=DEV, dtype=torch.int32)   # repeats occur
    if missing:
        drop = torch.rand((t, k), generator=g, device=DEV) < 0.2
        idx = torch.where(drop, torch.randint(-3, 0, (t, k), generator=g, device=DEV, dtype=torch.int32), idx)
    tl = (4 * torch.randn((t, k), generator=g, device=DEV)).to(tdt)
    dloss = torch.rand(t, generator=g, device=DEV) * (torch.rand(t, generator=g, device=DEV) < 0.8)
    return logits, idx, tl, dloss


def within(got, ref, tol, what):
    got = got.double()
    same = (got == ref) | ((got - ref).abs() <= tol)
    assert same.all(), (what, int((~same).sum()), got[~same][:4], ref[~same][:4])


def check_all(logits, idx, tl, dloss, tau):
    loss, lse = H.distill_fwd(logits, idx, tl, temperature=tau)
    rl, tl_, re, te, rg, tg = ref64(logits, idx, tl, tau, dloss)
    within(lse, re, te, "lse")
    within(loss, rl, tl_, "loss")
    both = H.distill_fwd_bwd(logits, idx, tl, dloss, temperature=tau)
    assert torch.equal(both[0], loss) and torch.equal(both[1], lse)
    within(both[2], rg, tg, "gradient of the joint call")
    grad = H.distill_bwd(dloss, logits, lse, idx, tl, temperature=tau)
    g2 = ref64(logits, idx, tl, tau, dloss, lse)
    within(grad, g2[4], g2[5], "gradient")
    assert torch.equal(grad, both[2])


# tokens, vocabulary, kept entries, row padding: every size of the held row and the longer ones
SHAPES = [(1, 1, 1, 0), (3, 7, 4, 0), (2, 8, 8, 3), (5, 1000, 33, 0), (4, 4100, 128, 5),
          (3, 8192, 5, 0), (3, 8200, 64, 0), (2, 32771, 300, 1), (3, 50257, 20, 0),
          (2, 65536, 16, 0), (1, 131072, 1024, 0), (2, 131075, 64, 0), (1, 262147, 7, 0)]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("t,v,k,pad", SHAPES)
def test_loss_and_gradient(t, v, k, pad, dt):
    print(f"tokens {t} vocabulary {v} kept {k} padding {pad} {dt}", flush=True)
    for seed, tau in ((1, 1.0), (2, 2.5)):
        check_all(*make(t, v, k, dt, seed, pad=pad), tau)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_teacher_in_bf16_and_strided(dt):
    logits, idx, tl, dloss = make(33, 2000, 24, dt, 5, tdt=BF16)
    wide_i = torch.full((33, 31), 7, dtype=torch.int32, device=DEV)
    wide_t = torch.zeros((33, 40), dtype=BF16, device=DEV)
    wide_i[:, :24], wide_t[:, :24] = idx, tl
    check_all(logits, wide_i[:, :24], wide_t[:, :24], dloss, 3.0)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("v", [1003, 140000])
def test_masked_places(v, dt):
    inf = float("inf")
    lowest = torch.finfo(dt).min
    logits, idx, tl, dloss = make(8, v, 16, dt, 9, missing=False)
    dloss = dloss + 0.25
    logits[0, v // 2:] = -inf              # half the vocabulary masked
    idx[0] = torch.arange(16, device=DEV, dtype=torch.int32)
    logits[1, 1:] = lowest                 # masked with the type's lowest value
    idx[1, :], idx[1, 0] = -1, 0           # one entry, at the only live logit: loss 0
    tl[2, 3:] = -inf                       # most of the teacher's entries without weight
    idx[3, :] = -1                         # no entry
    tl[4, :] = -inf                        # entries, none with weight
    idx[5, :] = v                          # outside the vocabulary: no entry
    logits[6, :] = -inf                    # nothing left of the student
    idx[7] = 5                             # one index sixteen times
    check_all(logits, idx, tl, dloss, 1.5)
    loss, lse, grad = H.distill_fwd_bwd(logits, idx, tl, dloss, temperature=1.5)
    for row in (3, 4, 5, 6):
        assert loss[row] == 0 and (grad[row] == 0).all()
    assert lse[6] == -inf
    assert (grad[0, v // 2:] == 0).all()
    # an entry with weight at a masked logit: infinite loss, finite gradient
    idx[0, 0] = v - 1
    loss, lse, grad = H.distill_fwd_bwd(logits, idx, tl, dloss, temperature=1.5)
    assert loss[0] == inf and torch.isfinite(grad[0]).all() and grad[0, v - 1] < 0


@pytest.mark.parametrize("dt", [BF16, F32])
def test_nan_stays_in_its_token(dt):
    nan, inf = float("nan"), float("inf")
    logits, idx, tl, dloss = make(6, 777, 9, dt, 3, missing=False)
    dloss = torch.ones_like(dloss)
    clean = H.distill_fwd_bwd(logits, idx, tl, dloss)
    logits[0, 5], logits[1, :], logits[2, 3], tl[3, 0], tl[4, :] = nan, nan, inf, nan, nan
    loss, lse, grad = H.distill_fwd_bwd(logits, idx, tl, dloss)
    assert loss[:5].isnan().all() and lse[:3].isnan().all() and not lse[3:].isnan().any()
    assert grad[0].isnan().all() and grad[1].isnan().all()
    for a, b in zip((loss, lse, grad), clean):
        assert torch.equal(a[5], b[5])
    # a token with dloss 0 has gradient 0 whatever its logits
    dloss[:5] = 0
    assert (H.distill_fwd_bwd(logits, idx, tl, dloss)[2][:5] == 0).all()
    assert (H.distill_bwd(dloss, logits, lse, idx, tl)[:5] == 0).all()


@pytest.mark.parametrize("dt,v", [(BF16, 5001), (F32, 40000), (BF16, 150001)])
def test_in_place_on_another_stream(dt, v):
    logits, idx, tl, dloss = make(9, v, 40, dt, 7)
    want = H.distill_fwd_bwd(logits, idx, tl, dloss, temperature=2.0)
    a, b = logits.clone(), logits.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = H.distill_fwd_bwd(a, idx, tl, dloss, temperature=2.0, dlogits=a, stream=s)
    g = H.distill_bwd(dloss, b, want[1], idx, tl, temperature=2.0, dlogits=b, stream=s)
    s.synchronize()
    assert got[2].data_ptr() == a.data_ptr()
    assert torch.equal(got[0], want[0]) and torch.equal(a, want[2]) and torch.equal(g, want[2])


def test_gradient_against_differences():
    # the sum of the weighted losses of the 64-bit formula by central differences
    logits, idx, tl, dloss = make(6, 301, 12, F32, 13)
    tau, step = 1.7, 1e-4
    grad = H.distill_fwd_bwd(logits, idx, tl, dloss, temperature=tau)[2].double()
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for _ in range(4):
        v = torch.randn(logits.shape, generator=g, device=DEV, dtype=torch.float64)
        up, down = (float((ref64(logits.double() + s * v, idx, tl, tau)[0] * dloss).sum())
                    for s in (step, -step))
        num, ours = (up - down) / (2 * step), float((grad * v).sum())
        assert abs(num - ours) <= 1e-5 * float((grad * v).abs().sum()), (num, ours)


def test_offsets_past_32_bits():
    # the last tokens of a batch whose logits span more than 2^32 bytes, each checked alone
    t, v = 20000, 120001
    logits = torch.zeros((t, v), dtype=BF16, device=DEV)
    small = make(3, v, 10, BF16, 1)
    logits[-3:] = small[0]
    idx = torch.full((t, 10), -1, dtype=torch.int32, device=DEV)
    tl = torch.zeros((t, 10), device=DEV)
    dloss = torch.zeros(t, device=DEV)
    idx[-3:], tl[-3:], dloss[-3:] = small[1], small[2], small[3]
    want = H.distill_fwd_bwd(*small)
    loss, lse, grad = H.distill_fwd_bwd(logits, idx, tl, dloss, dlogits=logits)
    assert torch.equal(loss[-3:], want[0]) and torch.equal(grad[-3:], want[2])
    assert (loss[:-3] == 0).all() and (grad[:-3].view(torch.int16).amax(1) == 0).all()


def test_no_tokens():
    e = torch.empty((0, 100), dtype=BF16, device=DEV)
    i = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    loss, lse, grad = H.distill_fwd_bwd(e, i, torch.empty((0, 4), device=DEV),
                                        torch.empty(0, device=DEV))
    assert loss.numel() == 0 and grad.shape == (0, 100)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("v", [5, 33, 1001, 2055, 16383, 16401, 33000])
def test_rows_that_start_anywhere(v, dt):
    # every start of a row within 64 bytes, in place and out of place: the gradient alone works on
    # parts that start on 64 bytes, and gives the joint call's bits
    step = 4 if dt == F32 else 2
    for shift in range(0, 64 // step, 3):
        logits, idx, tl, dloss = make(3, v, 6, dt, 11 + shift, missing=False)
        idx[0, 0], idx[0, 1], idx[1, 0] = 0, v - 1, min(v - 1, 40)
        room = torch.zeros(3 * (v + 5) + 64, dtype=dt, device=DEV)
        view = room[shift:shift + 3 * (v + 5)].view(3, v + 5)[:, :v]
        view.copy_(logits)
        guard = room.clone()
        loss, lse, want = H.distill_fwd_bwd(logits, idx, tl, dloss + 0.5, temperature=1.5)
        got = H.distill_bwd(dloss + 0.5, view, lse, idx, tl, temperature=1.5)
        assert torch.equal(got, want), shift
        H.distill_bwd(dloss + 0.5, view, lse, idx, tl, temperature=1.5, dlogits=view)
        assert torch.equal(view, want), shift
        view.copy_(logits)
        assert torch.equal(room, guard), shift   # nothing written outside the rows


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("v,k", [(1000, 64), (1000, 65), (5000, 257), (9001, 1023), (70000, 1024)])
def test_many_entries_that_repeat(v, k, dt):
    """Entries whose indices repeat up to k / 8 times (a sum of that many p adds k / 8 roundings, which
    the tolerance's k / 4 covers), far apart, next to each other, or in steps of a power of two."""
    print(f"vocabulary {v} kept {k} {dt}", flush=True)
    logits, idx, tl, dloss = make(6, v, k, dt, 21)
    dloss = dloss + 0.25
    n = torch.arange(k, device=DEV, dtype=torch.int32)
    idx[0] = n % v                                  # one each
    idx[1] = n % 8                                  # eight indices, each k / 8 times
    idx[2] = n.flip(0) // 2                         # neighbours, twice
    idx[3] = (n * 64) % v
    idx[4] = torch.where(n % 3 == 0, n // 8 * 8, -1)  # with places that are no entry between
    idx[5] = v - 1 - (n * 4096) % v
    repeats = torch.stack([torch.bincount(i[i >= 0].long(), minlength=v).max() for i in idx[:3]])
    assert (repeats <= -(-k // 8)).all()
    check_all(logits, idx, tl, dloss, 2.0)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("tau", [0.7, 1.0, 1.5, 3.0])
@pytest.mark.parametrize("value", ["lowest", -1e30, -1e10])
@pytest.mark.parametrize("v", [250, 2000, 9001, 70001, 140001])
def test_most_of_the_vocabulary_masked(v, value, tau, dt):
    """Masked places of a large negative value have weight exp(-1e10 / 3) = 0 whichever it is, so the
    formula's values are those of -inf there, with the live logits' tolerances."""
    print(f"vocabulary {v} value {value} temperature {tau} {dt}", flush=True)
    logits, idx, tl, dloss = make(5, v, 12, dt, 31, missing=False)
    dloss = dloss + 0.25
    at = torch.arange(v, device=DEV)
    live = torch.stack([at < 40, at >= v - 13, at % 97 == 3, (at < v // 8) | (at >= v - v // 8),
                        (at // 8) % 2 == 0])
    logits = torch.where(live, logits.float(), torch.finfo(dt).min if value == "lowest" else value).to(dt)
    for row in range(5):                     # the teacher's entries are live
        where = torch.nonzero(live[row])[:, 0]
        idx[row] = where[torch.arange(12, device=DEV) % len(where)].to(torch.int32)
    oracle = logits.masked_fill(~live, float("-inf"))
    loss, lse = H.distill_fwd(logits, idx, tl, temperature=tau)
    rl, tl_, re, te, rg, tg = ref64(oracle, idx, tl, tau, dloss)
    within(lse, re, te, "lse")
    within(loss, rl, tl_, "loss")
    both = H.distill_fwd_bwd(logits, idx, tl, dloss, temperature=tau)
    assert torch.equal(both[0], loss) and torch.equal(both[1], lse)
    within(both[2], rg, tg, "gradient of the joint call")
    assert (both[2][~live] == 0).all()
    assert torch.equal(H.distill_bwd(dloss, logits, lse, idx, tl, temperature=tau), both[2])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("tau", [1.0, 1.5, 3.0])
@pytest.mark.parametrize("v", [3, 250, 2000, 70001, 140001])
def test_rows_of_one_value(v, tau, dt):
    """A row whose logits are all the same has q = 1 / vocabulary, also where the value is the type's
    lowest or so large that lse is the value itself.

    Tolerances: the sum of exponentials carries at most 300 u (its chain of additions and 8 u each), so
    log q 310 u beside u |log V| per rounding; lse rounds |value| / temperature three times.  Up to
    4096 the gradient takes q from lse (8 u |lse|); beyond, from the sum itself."""
    print(f"vocabulary {v} temperature {tau} {dt}", flush=True)
    values = [torch.finfo(dt).min, -3e30, -1e10, -7.5e4, -1000.0, 0.0, 5.0, 6e4, 3e38]
    t = len(values)
    _, idx, tl, dloss = make(t, v, 9, dt, 41, missing=False)
    dloss = dloss + 0.25
    logits = torch.tensor(values, dtype=torch.float64, device=DEV)[:, None].expand(t, v).to(dt).contiguous()
    c = logits[:, 0].double() / tau
    logv = torch.log(torch.tensor(float(v), dtype=torch.float64)).item()
    p = torch.softmax(tl.double() / tau, 1)
    p_tol = (U * (64 + 8 * (tl.double() / tau).abs().amax(1) + 9 / 4))[:, None]
    loss, lse, grad = H.distill_fwd_bwd(logits, idx, tl, dloss, temperature=tau)
    within(lse, c + logv, U * (4 * c.abs() + 4 * logv + 310), "lse")
    tol = tau ** 2 * ((p * (p_tol + 16 * U) * (p.log().abs() + logv + 1)).sum(1) + 310 * U)
    within(loss, tau ** 2 * (p * (p.log() + logv)).sum(1), tol, "loss")
    l2, e2 = H.distill_fwd(logits, idx, tl, temperature=tau)
    assert torch.equal(l2, loss) and torch.equal(e2, lse)
    by = (dloss.double() * tau)[:, None]
    spread = torch.zeros((t, v), dtype=torch.float64, device=DEV).scatter_add_(1, idx.long(), p)
    want = by * (1 / v - spread)
    size = lse.double().abs()[:, None]
    e = U * (400 + 16 * logv + 8 * torch.where(size <= 4097, size, 0.0))
    tol = by * (e / v + spread * p_tol) + ROUND[dt] * 1.01 * want.abs()
    within(grad, want, tol, "gradient of the joint call")
    # from lse alone: as good as lse is where that says something, and never outside 0 <= q <= 1
    alone = H.distill_bwd(dloss, logits, lse, idx, tl, temperature=tau).double()
    top = by * (1 - spread)
    slack = by * spread * p_tol + ROUND[dt] * 1.01 * torch.maximum(top.abs(), (by * spread).abs())
    assert ((alone >= -by * spread - slack) & (alone <= top + slack)).all()
    near = size[:, 0] < 1e5
    e = U * (400 + 16 * logv + 8 * size)
    tol = by * (e / v * (1 + e) + spread * p_tol) + ROUND[dt] * 1.01 * (want.abs() + by * e / v)
    within(alone[near], want[near], tol[near], "gradient")


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("v", [3, 2000, 140001])
def test_logits_beyond_the_range_of_lse(v, dt):
    """At a temperature below 1 the type's extremes scale past fp32: lse is an infinity, loss and
    gradient of the joint call are still those of q = 1 / vocabulary (tolerances as for rows of one
    value, without lse), and the gradient from lse alone stays finite."""
    ext = torch.finfo(dt).max
    logits = torch.tensor([-ext, ext], dtype=torch.float64, device=DEV)[:, None].expand(2, v).to(dt).contiguous()
    _, idx, tl, dloss = make(2, v, 9, dt, 51, missing=False)
    dloss, tau, logv = dloss + 0.25, 0.7, torch.log(torch.tensor(float(v), dtype=torch.float64)).item()
    p = torch.softmax(tl.double() / tau, 1)
    p_tol = (U * (64 + 8 * (tl.double() / tau).abs().amax(1) + 9 / 4))[:, None]
    loss, lse, grad = H.distill_fwd_bwd(logits, idx, tl, dloss, temperature=tau)
    assert lse.tolist() == [float("-inf"), float("inf")]
    tol = tau ** 2 * ((p * (p_tol + 16 * U) * (p.log().abs() + logv + 1)).sum(1) + 310 * U)
    within(loss, tau ** 2 * (p * (p.log() + logv)).sum(1), tol, "loss")
    by = (dloss.double() * tau)[:, None]
    spread = torch.zeros((2, v), dtype=torch.float64, device=DEV).scatter_add_(1, idx.long(), p)
    want = by * (1 / v - spread)
    tol = by * (U * (400 + 16 * logv) / v + spread * p_tol) + ROUND[dt] * 1.01 * want.abs()
    within(grad, want, tol, "gradient of the joint call")
    l2, e2 = H.distill_fwd(logits, idx, tl, temperature=tau)
    assert torch.equal(l2, loss) and torch.equal(e2, lse)
    alone = H.distill_bwd(dloss, logits, lse, idx, tl, temperature=tau)
    assert torch.isfinite(alone).all() and (alone[0] == 0).all()   # of -inf alone: nothing left
