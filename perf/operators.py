"""Cases, plain forms and 64-bit values of the training and serving operators around the rotated
8-bit layer.

Three operators, as one block of a model and the loss on top of it use them:

  norm     block_norm_fwd / block_norm_bwd: a block's output y joins the residual stream r and the
           next block's input is normalised, r' = r + scale gate * rms(y) post_weight,
           h = rms(r') pre_weight, and its gradient.  gate is [G, D]: row g belongs to the g-th
           run of T / G consecutive tokens (G = 1: one gate per channel, G = T: one per token).
  linear   linear_act_fwd / linear_act_q / linear_act_bwd: the Hadamard-rotated 8-bit layer with
           y = act(X W^T + bias) + residual (the pre-activation z kept for the backward), the same
           on weights quantised once (serving), and its gradient.
  distill  distill_fwd / distill_bwd / distill_fwd_bwd: the divergence of a student's softmax over
           the vocabulary from a teacher's softmax over its top logits, per token, and its gradient
           for the logits.

`own` picks the side `run` takes: the plain form in elementary torch operations, or the library's
entry points.
"""
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
QMAX = {"i8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
GRAD_CODES = {"i8": "i8", "e4m3": "e5m2"}   # codes of dY beside codes of X and W


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of a small batch: latency of the join between two blocks
        {"name": "norm_fwd_decode", "op": "norm", "dir": "fwd", "t": 8, "d": 4096, "groups": 1,
         "type": "bf16"},
        # the same join over a training batch (or a long prompt)
        {"name": "norm_fwd_train", "op": "norm", "dir": "fwd", "t": 8192, "d": 4096, "groups": 1,
         "type": "bf16"},
        # its gradient over the same training batch, one gate per channel
        {"name": "norm_bwd_train", "op": "norm", "dir": "bwd", "t": 8192, "d": 4096, "groups": 1,
         "type": "bf16"},
        # full-precision stream of an odd width, gates per sequence (conditioned blocks)
        {"name": "norm_bwd_f32_odd", "op": "norm", "dir": "bwd", "t": 2310, "d": 2049, "groups": 6,
         "type": "f32"},
        # serving, one token: the layer on weights quantised once
        {"name": "linear_q_one_token", "op": "linear", "dir": "q", "m": 1, "n": 4096, "k": 4096,
         "block": 256, "codes": "i8", "act": "gelu_tanh", "bias": True, "res": False},
        # serving, a ragged batch of tokens, FP8 weights, back into the residual stream
        {"name": "linear_q_ragged_fp8", "op": "linear", "dir": "q", "m": 203, "n": 4096,
         "k": 11008, "block": 128, "codes": "e4m3", "act": "none", "bias": True, "res": True},
        # training forward of a wide projection, pre-activation kept
        {"name": "linear_fwd_train", "op": "linear", "dir": "fwd", "m": 8192, "n": 11008,
         "k": 4096, "block": 128, "codes": "i8", "act": "silu", "bias": True, "res": False},
        # training backward at the layer's headline size: dX, dW and the bias gradient
        {"name": "linear_bwd_train", "op": "linear", "dir": "bwd", "m": 4096, "n": 4096,
         "k": 4096, "block": 256, "codes": "i8", "act": "gelu_tanh", "bias": True, "res": False},
        # a few tokens: latency of loss and gradient together
        {"name": "distill_few_tokens", "op": "distill", "dir": "fwd_bwd", "t": 16, "v": 32000,
         "k": 32, "tau": 2.0, "type": "bf16"},
        # a training batch over a large vocabulary, loss and gradient together
        {"name": "distill_train", "op": "distill", "dir": "fwd_bwd", "t": 4096, "v": 131072,
         "k": 64, "tau": 1.0, "type": "bf16"},
        # full-precision logits of an odd vocabulary, the gradient alone under an upstream one
        {"name": "distill_bwd_f32_odd", "op": "distill", "dir": "bwd", "t": 777, "v": 50257,
         "k": 100, "tau": 1.5, "type": "f32"},
        # evaluation: the loss alone
        {"name": "distill_fwd_eval", "op": "distill", "dir": "fwd", "t": 2048, "v": 65536, "k": 8,
         "tau": 1.0, "type": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """A whole number spread evenly over its logarithm."""
    return min(hi, max(lo, int(lo * (hi / lo) ** rng.random() + rng.random())))


def draw(rng):
    op = rng.choice(["norm", "linear", "distill"])
    if op == "norm":
        d = _log_int(rng, 64, 8192)
        t = _log_int(rng, 1, min(16384, (8192 * 4096) // d))
        groups = rng.choice([1, 1, t] + [g for g in (2, 3, 4, 6, 8) if t % g == 0])
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "t": t, "d": d, "groups": groups,
                "type": rng.choice(["bf16", "bf16", "f32"])}
    if op == "linear":
        d = rng.choice(["q", "q", "fwd", "bwd"])
        n, k = 8 * _log_int(rng, 32, 1376), 32 * _log_int(rng, 8, 344)
        m = _log_int(rng, 1, 512) if d == "q" else _log_int(rng, 128, 4096)
        return {"op": op, "dir": d, "m": m, "n": n, "k": k, "block": rng.choice([64, 128, 256]),
                "codes": rng.choice(["i8", "i8", "e4m3"]),
                "act": rng.choice(["none", "relu", "silu", "gelu_tanh", "gelu_erf"]),
                "bias": rng.random() < 0.75, "res": d != "bwd" and rng.random() < 0.5}
    v = _log_int(rng, 1000, 131072)
    t = _log_int(rng, 1, min(8192, (4096 * 131072) // (4 * v)))
    return {"op": op, "dir": rng.choice(["fwd", "bwd", "fwd_bwd", "fwd_bwd"]), "t": t, "v": v,
            "k": _log_int(rng, 1, 128), "tau": rng.choice([1.0, 1.5, 2.0, 4.0]),
            "type": rng.choice(["bf16", "bf16", "f32"])}


def work(case):
    if case["op"] == "norm":
        e = 2 if case["type"] == "bf16" else 4
        td, t, d, g = case["t"] * case["d"], case["t"], case["d"], case["groups"]
        if case["dir"] == "fwd":    # r, y -> r', h; two weights, the gate, two statistics
            return {"bytes": 4 * td * e + (2 * d + g * d) * e + 8 * t, "flops": 12 * td}
        # dr', dh, r', y -> dr, dy; weights and gate and their gradients
        return {"bytes": 6 * td * e + 2 * (2 * d + g * d) * e + 8 * t, "flops": 30 * td}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        extra = 2 * n * case["bias"] + 2 * m * n * case["res"]
        if case["dir"] == "q":      # x, the weights' codes and scales -> y
            return {"bytes": 2 * m * k + n * _padded(k, case["block"]) + 4 * n + 2 * m * n + extra,
                    "flops": 2 * m * n * k}
        if case["dir"] == "fwd":    # x, w -> y, z
            return {"bytes": 2 * (m * k + n * k + 2 * m * n) + extra, "flops": 2 * m * n * k}
        # dy, z, x, w -> dx, dw, db
        return {"bytes": 2 * (2 * m * n + 2 * m * k + 2 * n * k) + extra, "flops": 4 * m * n * k}
    e = 2 if case["type"] == "bf16" else 4
    t, v, k = case["t"], case["v"], case["k"]
    once = t * v * e
    return {"bytes": (once if case["dir"] == "fwd" else 2 * once) + t * k * 8 + 12 * t,
            "flops": (4 if case["dir"] == "fwd" else 8) * t * v}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _padded(length, block):
    """The contraction length: zero padded to a multiple of the block and of 32."""
    step = max(block, 32)
    return -(-length // step) * step


def _hadamard(b, dtype):
    """The Sylvester matrix of order b: (-1) ** (number of common one bits of row and column)."""
    i = torch.arange(b, device=DEV)
    c = i[:, None] & i[None, :]
    for s in (8, 4, 2, 1):   # parity of the (at most 13) bits
        c = c ^ (c >> s)
    return (1 - 2 * (c & 1)).to(dtype)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, rows, cols):
    """Activations as a residual stream has them: a few channels are far larger than the rest."""
    x = _normal(g, rows, cols)
    x *= torch.where(torch.rand(cols, generator=g, device=DEV) < 0.004, 30.0, 1.0)
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        t, d, dt = case["t"], case["d"], TYPES[case["type"]]
        s["r"] = _activations(g, t, d).to(dt)
        s["y"] = (0.7 * _normal(g, t, d)).to(dt)
        s["gate"] = (0.5 + 0.3 * _normal(g, case["groups"], d)).to(dt)
        s["post"] = (1 + 0.1 * _normal(g, d)).to(dt)
        s["pre"] = (1 + 0.1 * _normal(g, d)).to(dt)
        s["scale"], s["eps"] = 0.5, 1e-6
        if case["dir"] == "bwd":
            s["rstd_post"] = torch.rsqrt(s["y"].float().square().mean(1) + s["eps"])
            s["rstd_pre"] = torch.rsqrt(s["r"].float().square().mean(1) + s["eps"])
            s["dr"] = (1e-2 * _normal(g, t, d)).to(dt)
            s["dh"] = (1e-2 * _normal(g, t, d)).to(dt)
        return s
    if case["op"] == "linear":
        m, n, k, block = case["m"], case["n"], case["k"], case["block"]
        bf = torch.bfloat16
        s["x"] = _activations(g, m, k).to(bf)
        w = (k ** -0.5 * _normal(g, n, k)).to(bf)
        if case["dir"] == "q":
            s["qw"], s["sw"] = _quantised_plain(w.float(), block, case["codes"])
            s["qw"] = s["qw"].to(CODES[case["codes"]])
        else:
            s["w"] = w
        s["bias"] = (0.1 * _normal(g, n)).to(bf) if case["bias"] else None
        s["res"] = _activations(g, m, n).to(bf) if case["res"] else None
        if case["dir"] == "bwd":
            s["z"] = (1.5 * _normal(g, m, n)).to(bf)
            s["dy"] = (1e-3 * _normal(g, m, n) / (0.3 + torch.rand(m, 1, generator=g, device=DEV))).to(bf)
        return s
    t, v, k, dt = case["t"], case["v"], case["k"], TYPES[case["type"]]
    s["logits"] = (2.5 * _normal(g, t, v)).to(dt)
    # the teacher's indices, all different in a token: one in each of k equal parts of the
    # vocabulary; a token in sixteen has fewer of them (the rest -1), some have none
    part = v // k
    idx = torch.arange(k, device=DEV)[None, :] * part \
        + torch.randint(0, part, (t, k), generator=g, device=DEV)
    keep = torch.where(torch.rand(t, 1, generator=g, device=DEV) < 1 / 16,
                       torch.randint(0, k, (t, 1), generator=g, device=DEV), k)
    s["idx"] = torch.where(torch.arange(k, device=DEV)[None, :] < keep, idx, -1).to(torch.int32)
    s["tlogits"] = 8 + 3 * _normal(g, t, k).sort(dim=1, descending=True).values
    # the student already knows part of what the teacher says
    rows = torch.arange(t, device=DEV)[:, None].expand(t, k)
    s["logits"][rows, idx] = (0.8 * s["tlogits"] + 1.0 * _normal(g, t, k)).to(dt)
    s["tau"] = case["tau"]
    if case["dir"] != "fwd":
        s["dloss"] = (torch.rand(t, generator=g, device=DEV) < 0.9).float() / max(1, t)
    if case["dir"] == "bwd":
        s["lse"] = torch.logsumexp(s["logits"].float() / s["tau"], 1)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _norm_fwd_plain(s):
    dt = s["r"].dtype
    r, y = s["r"].float(), s["y"].float()
    t, d = r.shape
    gate = s["gate"].float().repeat_interleave(t // s["gate"].shape[0], 0)
    rstd_post = torch.rsqrt((y * y).mean(1) + s["eps"])
    joined = r + s["scale"] * gate * (y * rstd_post[:, None] * s["post"].float())
    rstd_pre = torch.rsqrt((joined * joined).mean(1) + s["eps"])
    h = joined * rstd_pre[:, None] * s["pre"].float()
    return joined.to(dt), h.to(dt), rstd_post, rstd_pre


def _norm_bwd_plain(s):
    dt = s["r"].dtype
    r, y, dh = s["r"].float(), s["y"].float(), s["dh"].float()
    t, d = r.shape
    groups = s["gate"].shape[0]
    gate = s["gate"].float().repeat_interleave(t // groups, 0)
    rhat = r * s["rstd_pre"][:, None]
    drhat = dh * s["pre"].float()
    dr = s["dr"].float() + s["rstd_pre"][:, None] * (drhat - rhat * (drhat * rhat).mean(1, True))
    yhat = y * s["rstd_post"][:, None]
    dn = s["scale"] * gate * dr
    dgate = (s["scale"] * dr * (yhat * s["post"].float())).view(groups, t // groups, d).sum(1)
    dyhat = dn * s["post"].float()
    dy = s["rstd_post"][:, None] * (dyhat - yhat * (dyhat * yhat).mean(1, True))
    dpost, dpre = (dn * yhat).sum(0), (dh * rhat).sum(0)
    return dr.to(dt), dy.to(dt), dgate.to(dt), dpost.to(dt), dpre.to(dt)


def _quantised_plain(v, block, codes):
    """The rotated, quantised rows of v (32 bits): codes as the numbers they stand for, scales."""
    rows, length = v.shape
    lp = _padded(length, block)
    if lp != length:
        v = torch.cat([v, v.new_zeros(rows, lp - length)], 1)
    b = (v.reshape(-1, block) @ _hadamard(block, torch.float32)).view(rows, lp)
    top = b.abs().amax(1)
    mul = torch.where(top > 0, QMAX[codes] / top, 0.0)
    c = b * mul[:, None]
    c = torch.round(c) if codes == "i8" else c.to(CODES[codes]).float()
    return c, top / (QMAX[codes] * block ** 0.5)


def _act_plain(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))


def _act_slope_plain(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu_erf":
        return 0.5 * (1 + torch.erf(z * 0.7071067811865476)) \
            + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    u = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + u) + 0.5 * z * (1 - u * u) * 0.7978845608028654 * (1 + 0.134145 * z * z)


def _linear_plain(s):
    c = s["case"]
    block, codes = c["block"], c["codes"]
    qx, sx = _quantised_plain(s["x"].float(), block, codes)
    qw, sw = (s["qw"].float(), s["sw"]) if c["dir"] == "q" else _quantised_plain(s["w"].float(), block, codes)
    z = (qx @ qw.t()) * sx[:, None] * sw[None, :]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act_plain(z, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    y = y.to(torch.bfloat16)
    return (y, z.to(torch.bfloat16)) if c["dir"] == "fwd" else y


def _linear_bwd_plain(s):
    c = s["case"]
    block, codes, grad = c["block"], c["codes"], GRAD_CODES[c["codes"]]
    dz = s["dy"].float() * _act_slope_plain(s["z"].float(), c["act"])
    qa, sa = _quantised_plain(dz, block, grad)
    qb, sb = _quantised_plain(s["w"].float().t().contiguous(), block, codes)
    dx = (qa @ qb.t()) * sa[:, None] * sb[None, :]
    qa, sa = _quantised_plain(dz.t().contiguous(), block, grad)
    qb, sb = _quantised_plain(s["x"].float().t().contiguous(), block, codes)
    dw = (qa @ qb.t()) * sa[:, None] * sb[None, :]
    out = (dx.to(torch.bfloat16), dw.to(torch.bfloat16))
    return out + (dz.sum(0).to(torch.bfloat16),) if c["bias"] else out


def _distill_plain(s):
    c, tau = s["case"], s["tau"]
    z = s["logits"].float() * (1 / tau)
    if c["dir"] == "bwd":
        lse = s["lse"]
    else:
        top = z.amax(1)
        lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    there = s["idx"] >= 0
    some = there.any(1)
    at = torch.where(there, s["idx"], 0).long()
    tl = torch.where(there, s["tlogits"] / tau, float("-inf"))
    tl = tl - torch.where(some, tl.amax(1), 0.0)[:, None]
    p = torch.exp(tl)
    total = torch.where(some, p.sum(1), 1.0)
    p = p / total[:, None]
    logp = torch.where(there, tl - torch.log(total)[:, None], 0.0)
    logq = z.gather(1, at) - lse[:, None]
    loss = tau * tau * (p * (logp - logq)).sum(1)
    if c["dir"] == "fwd":
        return loss, lse
    by = tau * torch.where(some, s["dloss"], 0.0)
    grad = torch.exp(z - lse[:, None]) * by[:, None]
    grad.scatter_add_(1, at, -p * by[:, None])
    grad = grad.to(s["logits"].dtype)
    return grad if c["dir"] == "bwd" else (loss, lse, grad)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _norm_fwd_plain(s) if c["dir"] == "fwd" else _norm_bwd_plain(s)
    if c["op"] == "linear":
        return _linear_bwd_plain(s) if c["dir"] == "bwd" else _linear_plain(s)
    return _distill_plain(s)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _library(s):
    import hadamard_rotated_precision_halo_amd as H
    c = s["case"]
    if c["op"] == "norm":
        if c["dir"] == "fwd":
            return H.block_norm_fwd(s["r"], s["y"], gate=s["gate"], post_weight=s["post"],
                                    pre_weight=s["pre"], scale=s["scale"], eps=s["eps"])
        return H.block_norm_bwd(s["dr"], s["dh"], s["r"], s["y"], gate=s["gate"],
                                post_weight=s["post"], pre_weight=s["pre"],
                                rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"],
                                scale=s["scale"])
    if c["op"] == "linear":
        if c["dir"] == "q":
            return H.linear_act_q(s["x"], s["qw"], s["sw"], c["block"], bias=s["bias"],
                                  activation=c["act"], residual=s["res"])
        if c["dir"] == "fwd":
            return H.linear_act_fwd(s["x"], s["w"], c["block"], CODES[c["codes"]], bias=s["bias"],
                                    activation=c["act"], residual=s["res"], want_z=True)
        out = H.linear_act_bwd(s["dy"], s["z"], s["x"], s["w"], c["block"], CODES[c["codes"]],
                               CODES[GRAD_CODES[c["codes"]]], activation=c["act"],
                               want_db=c["bias"])
        return out if c["bias"] else out[:2]
    if c["dir"] == "fwd":
        return H.distill_fwd(s["logits"], s["idx"], s["tlogits"], temperature=s["tau"])
    if c["dir"] == "bwd":
        return H.distill_bwd(s["dloss"], s["logits"], s["lse"], s["idx"], s["tlogits"],
                             temperature=s["tau"])
    return H.distill_fwd_bwd(s["logits"], s["idx"], s["tlogits"], s["dloss"],
                             temperature=s["tau"])


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def _codes64(v, block, codes):
    """Row codes (as numbers) and scales of v by the definition: orthonormal block transform by
    butterflies, absmax scale, nearest code with ties to even."""
    rows, length = v.shape
    lp = _padded(length, block)
    u = v.new_zeros(rows, lp)
    u[:, :length] = v
    step = 1
    while step < block:
        w = u.view(rows, lp // (2 * step), 2, step)
        u = torch.stack([w[:, :, 0] + w[:, :, 1], w[:, :, 0] - w[:, :, 1]], 2).view(rows, lp)
        step *= 2
    u = u / block ** 0.5
    top = u.abs().amax(1, keepdim=True)
    a = torch.where(top > 0, u / torch.where(top > 0, top, 1.0) * QMAX[codes], 0.0)
    if codes == "i8":
        quantum = 1.0
    else:   # grid step of a's binade, the subnormal one at the bottom
        bits, lowest = (3, -6) if codes == "e4m3" else (2, -14)
        _, e = torch.frexp(a)
        quantum = torch.exp2((torch.clamp(e - 1, min=lowest) - bits).double())
    return torch.round(a / quantum) * quantum, (top / QMAX[codes]).squeeze(1)


def _act64(z, act):
    """act(z) and its slope."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if act == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu_erf":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    a, b = (2 / torch.pi) ** 0.5, 0.044715
    p = torch.special.expit(2 * a * (z + b * z ** 3))   # (1 + tanh u) / 2
    return z * p, p + z * 2 * p * (1 - p) * a * (1 + 3 * b * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    f = {n: v.double() if isinstance(v, torch.Tensor) and n not in ("idx",) else v
         for n, v in s.items()}
    if case["op"] == "norm":
        t, d, groups = case["t"], case["d"], case["groups"]
        gate = f["gate"].view(groups, 1, d).expand(groups, t // groups, d).reshape(t, d) * f["scale"]
        if case["dir"] == "fwd":
            a = 1 / torch.sqrt(f["y"].pow(2).sum(1) / d + f["eps"])
            out = f["r"] + gate * f["post"] * f["y"] * a[:, None]
            b = 1 / torch.sqrt(out.pow(2).sum(1) / d + f["eps"])
            return out, out * f["pre"] * b[:, None], a, b
        a, b = f["rstd_post"][:, None], f["rstd_pre"][:, None]
        u = f["dh"] * f["pre"]
        dr = f["dr"] + b * u - f["r"] * b ** 3 * (u * f["r"]).sum(1, keepdim=True) / d
        v = dr * gate * f["post"]
        dy = a * v - f["y"] * a ** 3 * (v * f["y"]).sum(1, keepdim=True) / d
        dgate = (f["scale"] * dr * f["y"] * a * f["post"]).view(groups, -1, d).sum(1)
        return dr, dy, dgate, (dr * gate * f["y"] * a).sum(0), (f["dh"] * f["r"] * b).sum(0)
    if case["op"] == "linear":
        block, codes, grad = case["block"], case["codes"], GRAD_CODES[case["codes"]]

        def product(a, b):
            (qa, sa), (qb, sb) = a, b
            return (qa @ qb.t()) * (sa[:, None] * sb[None, :])

        if case["dir"] == "bwd":
            dz = f["dy"] * _act64(f["z"], case["act"])[1]
            dx = product(_codes64(dz, block, grad), _codes64(f["w"].t().contiguous(), block, codes))
            dw = product(_codes64(dz.t().contiguous(), block, grad),
                         _codes64(f["x"].t().contiguous(), block, codes))
            return (dx, dw, dz.sum(0)) if case["bias"] else (dx, dw)
        right = (f["qw"], f["sw"]) if case["dir"] == "q" else _codes64(f["w"], block, codes)
        z = product(_codes64(f["x"], block, codes), right)
        if case["bias"]:
            z = z + f["bias"]
        y = _act64(z, case["act"])[0]
        if case["res"]:
            y = y + f["res"]
        return (y, z) if case["dir"] == "fwd" else y
    tau = f["tau"]
    z = f["logits"] / tau
    lse = f["lse"] if case["dir"] == "bwd" else torch.logsumexp(z, 1)
    there = s["idx"] >= 0
    none = ~there.any(1, keepdim=True)
    u = torch.where(there, f["tlogits"] / tau, float("-inf"))
    u = torch.where(none, 0.0, u)
    logp = torch.log_softmax(u, 1)
    p = torch.where(there, torch.exp(logp), 0.0)
    at = s["idx"].clamp(min=0).long()
    loss = tau ** 2 * torch.where(there, p * (logp - z.gather(1, at) + lse[:, None]), 0.0).sum(1)
    if case["dir"] == "fwd":
        return loss, lse
    by = torch.where(none, 0.0, f["dloss"][:, None] * tau)
    z = z.sub_(lse[:, None]).exp_()
    z.scatter_add_(1, at, -p)
    z = z.mul_(by)
    return z if case["dir"] == "bwd" else (loss, lse, z)
