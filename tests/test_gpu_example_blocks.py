"""The operators together: a stack of blocks tuned towards a teacher's top logits, and served."""
import pytest
import torch

from hadamard_rotated_precision_halo_amd import example_blocks as E

pytestmark = pytest.mark.gpu


def plain_loss(student, x, idx, kept, tau):
    """The stack in fp32 torch with autograd, on the same parameters (no 8-bit codes)."""
    p = {k: v.float().clone().requires_grad_(True) for k, v in student.p.items()}

    def norm(v, w):
        return v * torch.rsqrt(v.square().mean(1, True) + 1e-6) * w

    r = x.float()
    h = norm(r, p["pre0"])
    for i in range(student.layers):
        u = torch.nn.functional.gelu(h @ p[f"w1.{i}"].t() + p[f"b1.{i}"], approximate="tanh")
        y = u @ p[f"w2.{i}"].t() + p[f"b2.{i}"]
        r = r + student.scale * p[f"gate.{i}"] * norm(y, p[f"post.{i}"])
        h = norm(r, p[f"pre{i + 1}"])
    logq = torch.log_softmax(h @ p["head"].t() / tau, 1).gather(1, idx.long())
    logp = torch.log_softmax(kept / tau, 1)
    loss = tau ** 2 * (logp.exp() * (logp - logq)).sum(1).mean()
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in p.items()}


def test_a_step_against_autograd():
    # every operator's forward and gradient in one chain: the 8-bit codes leave some per cent
    s = E.Blocks(layers=2, dim=256, hidden=512, vocab=1000, block=64, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(300, 256, generator=g, device="cuda").bfloat16()
    idx = torch.randint(0, 1000, (300, 16), generator=g, device="cuda", dtype=torch.int32)
    kept = 3 * torch.randn(300, 16, generator=g, device="cuda")
    want, grads = plain_loss(s, x, idx, kept, 2.0)
    logits, saved = s.forward(x)
    loss, _, dlogits = E.H.distill_fwd_bwd(logits, idx, kept, torch.full((300,), 1 / 300, device="cuda"),
                                           temperature=2.0)
    assert abs(float(loss.mean()) - want) <= 0.02 * want
    for k, v in s.backward(dlogits, saved).items():
        ref = grads[k].double()
        rel = float((v.double() - ref).norm() / ref.norm())
        assert rel <= 0.15, (k, rel)


def test_training_and_serving():
    losses, student, x = E.train(steps=8, tokens=256, report=lambda s: None, layers=2, dim=256,
                                 hidden=1024, vocab=2000, block=64)
    assert all(b < a for a, b in zip(losses, losses[1:])) and losses[-1] < 0.8 * losses[0], losses
    q = student.quantised()
    for n in (1, 4, 40):   # the serving kernels against the training forward, bit for bit
        assert torch.equal(student.serve(x[:n], q), student.forward(x[:n])[0])
