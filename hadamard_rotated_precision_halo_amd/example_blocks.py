"""A stack of residual blocks in rotated 8-bit layers, tuned towards a teacher's top logits.

Shows the library's operators as a training step and a serving step use them together:

  forward    h = norm(r); per block  u = gelu(h W1^T + b1) (pre-activation kept), or gated,
             u = silu(h Wg^T + bg) (h Wu^T + bu) with W1 = [Wg, Wu],  y = u W2^T + b2,
             r = r + scale gate norm(y), h = norm(r); logits = h Wv^T; the layers' inputs and
             pre-activations kept for the backward in bf16 or, with `kept`, in 8 bits;
  loss       the divergence from the teacher's softmax over its top logits, with its gradient;
  backward   the same in reverse: every product and every gradient product in 8 bits;
  serving    the same forward for a few tokens, on weights quantised once.

Run it on a GPU:  python -m hadamard_rotated_precision_halo_amd.example_blocks [--gated] [--keep8]
"""
import argparse

import torch

import hadamard_rotated_precision_halo_amd as H


class Blocks:
    """bf16 parameters of a stack, their fp32 copies for the update, and the steps on them."""

    def __init__(self, layers=2, dim=512, hidden=2048, vocab=4096, block=128, seed=0,
                 device="cuda", gated=False, kept=None):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)

        def weight(rows, cols):
            return torch.randn(rows, cols, generator=g) * cols ** -0.5

        self.layers, self.block, self.scale = layers, block, 0.5
        self.gated, self.kept = gated, kept
        wide = 2 * hidden if gated else hidden
        p = {"pre0": torch.ones(dim), "head": weight(vocab, dim)}
        for i in range(layers):
            p[f"w1.{i}"], p[f"b1.{i}"] = weight(wide, dim), torch.zeros(wide)
            p[f"w2.{i}"], p[f"b2.{i}"] = weight(dim, hidden), torch.zeros(dim)
            p[f"gate.{i}"], p[f"post.{i}"] = torch.ones(1, dim), torch.ones(dim)
            p[f"pre{i + 1}"] = torch.ones(dim)
        self.full = {k: v.to(device) for k, v in p.items()}
        self.p = {k: v.to(torch.bfloat16) for k, v in self.full.items()}

    def keep(self, t):
        """A layer's input as the backward gets it."""
        return t if self.kept is None else H.checkpoint_pack(t, self.kept)

    def forward(self, x):
        """Logits of the tokens x [tokens, dim] (bf16) and what the backward needs."""
        p, saved = self.p, []
        r, h, _, rstd = H.block_norm_fwd(x, pre_weight=p["pre0"])
        first = (r, rstd)
        for i in range(self.layers):
            first_layer, act = ((H.linear_glu_fwd, "silu") if self.gated
                                else (H.linear_act_fwd, "gelu_tanh"))
            u, z = first_layer(h, p[f"w1.{i}"], self.block, bias=p[f"b1.{i}"], activation=act,
                               want_z=self.kept or True)
            y = H.linear_act_fwd(u, p[f"w2.{i}"], self.block, bias=p[f"b2.{i}"])
            r, h2, rstd_post, rstd_pre = H.block_norm_fwd(
                r, y, gate=p[f"gate.{i}"], post_weight=p[f"post.{i}"],
                pre_weight=p[f"pre{i + 1}"], scale=self.scale)
            saved.append((self.keep(h), z, self.keep(u), y, r, rstd_post, rstd_pre))
            h = h2
        return H.linear_act_fwd(h, p["head"], self.block), (first, saved, self.keep(h))

    def backward(self, dlogits, kept):
        """Gradients of every parameter, by name."""
        p, (first, saved, h), grads = self.p, kept, {}
        dh, grads["head"], _ = H.linear_act_bwd(dlogits, None, h, p["head"], self.block,
                                                want_db=False)
        dr = None
        for i in reversed(range(self.layers)):
            h, z, u, y, r, rstd_post, rstd_pre = saved[i]
            dr, dy, grads[f"gate.{i}"], grads[f"post.{i}"], grads[f"pre{i + 1}"] = H.block_norm_bwd(
                dr, dh, r, y, gate=p[f"gate.{i}"], post_weight=p[f"post.{i}"],
                pre_weight=p[f"pre{i + 1}"], rstd_post=rstd_post, rstd_pre=rstd_pre,
                scale=self.scale)
            du, grads[f"w2.{i}"], grads[f"b2.{i}"] = H.linear_act_bwd(dy, None, u, p[f"w2.{i}"],
                                                                      self.block)
            first_layer, act = ((H.linear_glu_bwd, "silu") if self.gated
                                else (H.linear_act_bwd, "gelu_tanh"))
            dh, grads[f"w1.{i}"], grads[f"b1.{i}"] = first_layer(
                du, z, h, p[f"w1.{i}"], self.block, activation=act)
        grads["pre0"] = H.block_norm_bwd(dr, dh, first[0], pre_weight=p["pre0"],
                                         rstd_pre=first[1])[4]
        return grads

    def update(self, grads, rate):
        """One step of normalised gradient descent on the fp32 copies."""
        for k, g in grads.items():
            g = g.float()
            size = self.full[k].norm() / (g.norm() + 1e-12)
            self.full[k] -= rate * size * g
            self.p[k].copy_(self.full[k])

    def quantised(self):
        """The weights' codes and scales, laid out once for serving."""
        return {k: H.fwht_quant(v, H.ROWS, self.block) for k, v in self.p.items()
                if k[0] == "w" or k == "head"}

    def serve(self, x, q):
        """forward's logits for a few tokens, on the weights quantised() gave."""
        p = self.p
        r, h, _, _ = H.block_norm_fwd(x, pre_weight=p["pre0"])
        for i in range(self.layers):
            first_layer, act = ((H.linear_glu_q, "silu") if self.gated
                                else (H.linear_act_q, "gelu_tanh"))
            u = first_layer(h, *q[f"w1.{i}"], self.block, bias=p[f"b1.{i}"], activation=act)
            y = H.linear_act_q(u, *q[f"w2.{i}"], self.block, bias=p[f"b2.{i}"])
            r, h, _, _ = H.block_norm_fwd(r, y, gate=p[f"gate.{i}"], post_weight=p[f"post.{i}"],
                                          pre_weight=p[f"pre{i + 1}"], scale=self.scale)
        return H.linear_act_q(h, *q["head"], self.block)


def train(steps=12, tokens=512, top=32, temperature=2.0, rate=0.02, seed=1, report=print, **shape):
    """Tunes a student, started apart from its teacher, on the teacher's top logits; returns the
    mean losses of the steps, the student and a batch."""
    teacher, student = Blocks(seed=seed, **shape), Blocks(seed=seed, **shape)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for k, v in student.full.items():
        v += 0.3 * v.std(unbiased=False).nan_to_num() * torch.randn(v.shape, generator=g, device=v.device)
        student.p[k].copy_(v)
    x = torch.randn(tokens, teacher.full["pre0"].numel(), generator=g, device="cuda").bfloat16()
    kept, idx = teacher.forward(x)[0].float().topk(top, dim=1)
    idx = idx.to(torch.int32)
    dloss = torch.full((tokens,), 1.0 / tokens, device="cuda")
    losses = []
    for step in range(steps):
        logits, saved = student.forward(x)
        loss, _, dlogits = H.distill_fwd_bwd(logits, idx, kept, dloss, temperature=temperature,
                                             dlogits=logits)   # the gradient replaces the logits
        student.update(student.backward(dlogits, saved), rate)
        losses.append(float(loss.mean()))
        report(f"step {step:3d}  loss {losses[-1]:.4f}")
    return losses, student, x


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--gated", action="store_true", help="gated feed-forward blocks")
    ap.add_argument("--keep8", action="store_true",
                    help="keep the layers' inputs and pre-activations in 8 bits")
    a = ap.parse_args()
    _, student, x = train(a.steps, a.tokens, gated=a.gated, kept=torch.int8 if a.keep8 else None)
    served, trained = student.serve(x[:4], student.quantised()), student.forward(x[:4])[0]
    print("serving 4 tokens on quantised weights: the same logits as the forward:",
          bool(torch.equal(served, trained)))


if __name__ == "__main__":
    main()
