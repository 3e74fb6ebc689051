"""A small encoder trained with the 1-bit Adam step: the model's side and the
optimizer's side of the library together.

Each of the W simulated workers runs the encoder on its own batch: attention
with the learned bucketed position bias and attention dropout, dropout added
to the residual stream (momentum_compression_gb300.model), plain matrix
products around them.  The workers' gradients, in bf16 fused buffers, go
through OneBitOptimizer: Adam warmup, then compressed steps.  The task is
synthetic: every position must name the token `shift` places before it, so
only attention over positions can solve it.

    python examples/train_encoder.py [--steps 200] [--warmup 100]
"""
import argparse
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import momentum_compression_gb300 as ob  # noqa: E402
from momentum_compression_gb300 import model as M  # noqa: E402

BF16 = torch.bfloat16


class Encoder:
    """Two pre-norm layers; parameters are views of one fused fp32 buffer (the
    optimizer's p), gradients are written to a fused bf16 buffer."""

    def __init__(self, vocab=64, dim=256, heads=4, ffn=512, layers=2, p=0.1, seed=1234):
        self.dim, self.heads, self.layers, self.p, self.seed = dim, heads, layers, p, seed
        self.relpos = M.RelPos(32, 128, two_sided=True)
        self.shapes = [("emb", (vocab, dim)), ("head", (dim, vocab)),
                       ("bias", (self.relpos.num_buckets, heads))]
        for i in range(layers):
            self.shapes += [(f"{i}.qkv", (dim, 3 * dim)), (f"{i}.out", (dim, dim)),
                            (f"{i}.up", (dim, ffn)), (f"{i}.down", (ffn, dim))]
        self.n = sum(math.prod(s) for _, s in self.shapes)

    def initialise(self, fused):
        g = torch.Generator(device="cuda")
        g.manual_seed(self.seed)
        for name, w in self._views(fused):
            std = 1.0 if name == "emb" else 0.02 if name == "bias" else w.shape[0] ** -0.5
            w.copy_(torch.randn(w.shape, generator=g, device="cuda") * std)

    def _views(self, fused):
        at = 0
        for name, shape in self.shapes:
            m = math.prod(shape)
            yield name, fused[at:at + m].view(shape)
            at += m

    def loss(self, w, tokens, lengths, target, step):
        """Mean cross entropy of the valid positions; `step` names this pass's random numbers."""
        B, L = tokens.shape
        x = w["emb"][tokens]
        draw = step * 3 * self.layers  # offsets of this pass: three calls a layer
        for i in range(self.layers):
            y = F.layer_norm(x, (self.dim,))
            q, k, v = (y @ w[f"{i}.qkv"]).view(B, L, 3, self.heads, -1).unbind(2)
            # the table is kept at 1/32 of the bias, so that one step size suits all parameters
            a = M.attention(q, k, v, table=w["bias"] * 32, relpos=self.relpos, kv_len=lengths,
                            p=self.p, seed=self.seed, offset=draw)
            x = M.dropout(a.reshape(B, L, -1) @ w[f"{i}.out"], self.p, self.seed, draw + 1, x)
            y = F.gelu(F.layer_norm(x, (self.dim,)) @ w[f"{i}.up"]) @ w[f"{i}.down"]
            x = M.dropout(y, self.p, self.seed, draw + 2, x)
            draw += 3
        logits = (F.layer_norm(x, (self.dim,)) @ w["head"]).float()
        valid = torch.arange(L, device="cuda")[None, :] < lengths[:, None]
        return F.cross_entropy(logits[valid], target[valid])

    def gradients(self, fused, out, batch, step):
        """Writes the gradients of one batch into the bf16 buffer `out`; returns the loss."""
        w = {name: v.to(BF16).requires_grad_() for name, v in self._views(fused)}
        loss = self.loss(w, *batch, step)
        grads = torch.autograd.grad(loss, list(w.values()))
        for (_, view), g in zip(self._views(out), grads):
            view.copy_(g)
        return loss.detach()


def batch(g, B=16, L=48, vocab=64, shift=3):
    tokens = torch.randint(vocab, (B, L), generator=g, device="cuda")
    lengths = torch.randint(L // 2, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    return tokens, lengths, tokens.roll(shift, 1)


def train(steps=200, warmup=100, W=2, lr=1e-3, log=print):
    net = Encoder()
    opt = ob.OneBitOptimizer(net.n, W, 1 << 16, grad_dtype="bf16", lr=lr, eps=1e-8)
    net.initialise(opt.p)
    grads = opt.grad_buffers()
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    losses = []
    for t in range(warmup + steps):
        if t == warmup:
            opt.begin_compression()
        loss = sum(net.gradients(opt.p, grads[w], batch(g), t * W + w) for w in range(W)) / W
        opt.warmup_step(grads) if t < warmup else opt.compressed_step(grads)
        losses.append(loss)
        if t % 20 == 0:
            phase = "warmup    " if t < warmup else "compressed"
            log(f"step {t:4d} {phase} loss {loss.item():.4f}")
    torch.cuda.synchronize()
    opt.close()
    return [x.item() for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--warmup", type=int, default=100)
    a = ap.parse_args()
    losses = train(a.steps, a.warmup)
    print(f"loss {losses[0]:.4f} -> {sum(losses[-10:]) / len(losses[-10:]):.4f}")
