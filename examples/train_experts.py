"""A small language-model step made of the library's products: experts' feed-forward block, a dense
feed-forward block with its residual, and the head's cross entropy, forward and backward, then one
token through the trained weights.

    python examples/train_experts.py [--steps 60]

Every matrix product runs in the library; torch holds the memory, routes the tokens and updates the
weights.  The data is synthetic: each next token is a fixed function of the current one, so the loss
falls from log(vocabulary) towards 0.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_dense_amd as mp  # noqa: E402

T, TYPE = "bf16", torch.bfloat16


def new(*shape, dtype=TYPE):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Model:
    """Sizes are multiples of 8, so that rows are whole 16-byte blocks."""

    def __init__(self, vocab=1000, width=128, inner=256, experts=8, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.h = mp.Handle()
        self.vocab, self.width, self.inner, self.experts = vocab, width, inner, experts

        def weight(*shape):
            return (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).cuda()

        # FP32 masters; the products take BF16 copies
        self.master = {"embed": weight(vocab, width) * width ** 0.5 * 0.5, "up": weight(experts, inner, width),
                       "down": weight(experts, width, inner), "w1": weight(inner, width), "w2": weight(width, inner),
                       "head": weight(vocab, width), "b1": torch.zeros(inner, device="cuda"),
                       "b2": torch.zeros(width, device="cuda")}
        self.w = {k: v.to(TYPE) for k, v in self.master.items()}
        self.momentum = {}

    def route(self, tokens):
        """Tokens sorted by expert and where each expert's rows start; stays on the device."""
        expert = tokens % self.experts
        order = torch.argsort(expert, stable=True)
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.bincount(expert, minlength=self.experts).cumsum(0)
        return order, offsets

    # ------------------------------------------------------------------ the products
    def dense(self, a, w, act="none", bias=None, keep=None, residual=None, transposed=True):
        """act(a w^T + bias) + residual; transposed=False: a w."""
        m, k = a.shape
        n = w.shape[0] if transposed else w.shape[1]
        d = new(m, n)
        epi = mp.Epilogue(act=act, bias=bias, bias_type="f32", aux=keep, ld_aux=n)
        mp.mpgemm_run_epilogue(self.h.h, False, transposed, m, n, k, 1.0, a, T, a.stride(0), w, T, w.stride(0), epi,
                               0.0 if residual is None else 1.0, residual, T, n, d, T, n)
        return d

    def dense_grad(self, a, w, act, kept):
        """((a w) act'(kept), its column sums)."""
        m, k = a.shape
        n = w.shape[1]
        d, db = new(m, n), new(n, dtype=torch.float32)
        size = mp.mpgemm_epilogue_grad_workspace_size(1, m, n)
        mp.mpgemm_run_epilogue_grad(self.h.h, False, False, m, n, k, 1.0, a, T, k, w, T, n, act, kept, n, d, T, n, db,
                                    new(size, dtype=torch.uint8), size)
        return d, db

    def weight_grad(self, dy, x):
        """dy^T x in FP32."""
        m, n = dy.shape[1], x.shape[1]
        d = new(m, n, dtype=torch.float32)
        mp.mpgemm_run(self.h.h, True, False, m, n, dy.shape[0], 1.0, dy, T, m, x, T, n, 0.0, None, "f32", n, d, "f32")
        return d

    def grouped(self, a, w, offsets, act="none", keep=None, transposed=True):
        rows, k = a.shape
        n = w.shape[1] if transposed else w.shape[2]
        d = new(rows, n)
        epi = mp.Epilogue(act=act, aux=keep, ld_aux=n)
        mp.mpgemm_run_grouped(self.h.h, transposed, self.experts, rows, n, k, 1.0, a, T, k, offsets, w, T, w.stride(1),
                              w.stride(0), epi, d, T, n)
        return d

    def grouped_grad(self, a, w, offsets, act, kept):
        rows, k = a.shape
        n = w.shape[2]
        d = new(rows, n)
        mp.mpgemm_run_grouped_grad(self.h.h, False, self.experts, rows, n, k, 1.0, a, T, k, offsets, w, T, n, w.stride(0),
                                   act, kept, n, d, T, n, None, None, 0)
        return d

    def grouped_weight_grad(self, dy, x, offsets):
        rows, m = dy.shape
        n = x.shape[1]
        d = new(self.experts, m, n, dtype=torch.float32)
        mp.mpgemm_run_grouped_wgrad(self.h.h, self.experts, rows, m, n, 1.0, dy, T, m, x, T, n, offsets, 0.0, d, "f32", n,
                                    m * n)
        return d

    # ------------------------------------------------------------------ the model
    def forward(self, tokens, keep=True):
        w, s = self.w, {}
        rows = tokens.numel()
        s["x"] = w["embed"][tokens]
        s["order"], s["offsets"] = self.route(tokens)
        s["xs"] = s["x"][s["order"]]
        s["zu"] = new(rows, self.inner) if keep else None
        s["hu"] = self.grouped(s["xs"], w["up"], s["offsets"], "silu", s["zu"])
        out = self.grouped(s["hu"], w["down"], s["offsets"])
        s["y"] = s["x"].index_add(0, s["order"], out)
        s["z1"] = new(rows, self.inner) if keep else None
        s["h1"] = self.dense(s["y"], w["w1"], "gelu", self.master["b1"], s["z1"])
        s["y2"] = self.dense(s["h1"], w["w2"], "none", self.master["b2"], residual=s["y"])
        return s

    def loss_and_gradients(self, tokens, target):
        w, s = self.w, self.forward(tokens)
        m, n, k = tokens.numel(), self.vocab, self.width
        size = mp.mpgemm_linear_ce_workspace_size(m, n, k, T, True)
        ws = new(size, dtype=torch.uint8)
        loss, lse = new(m, dtype=torch.float32), new(m, dtype=torch.float32)
        counts = (target >= 0).sum().clamp(min=1)
        mp.mpgemm_run_linear_ce(self.h.h, m, n, k, 1.0, s["y2"], T, k, w["head"], k, target, loss, lse, ws, size)
        weight = (1.0 / counts).float().expand(m).contiguous()
        dy2, dhead = new(m, k), new(n, k)
        mp.mpgemm_run_linear_ce_grad(self.h.h, m, n, k, 1.0, s["y2"], T, k, w["head"], k, target, lse, weight, dy2, k, dhead,
                                     k, ws, size)
        g = {"head": dhead.float(), "b2": dy2.float().sum(0), "w2": self.weight_grad(dy2, s["h1"])}
        dz1, g["b1"] = self.dense_grad(dy2, w["w2"], "gelu", s["z1"])
        g["w1"] = self.weight_grad(dz1, s["y"])
        dy = self.dense(dz1, w["w1"], residual=dy2, transposed=False)
        dout = dy[s["order"]]
        g["down"] = self.grouped_weight_grad(dout, s["hu"], s["offsets"])
        dzu = self.grouped_grad(dout, w["down"], s["offsets"], "silu", s["zu"])
        g["up"] = self.grouped_weight_grad(dzu, s["xs"], s["offsets"])
        dx = dy.float().index_add(0, s["order"], self.grouped(dzu, w["up"], s["offsets"], transposed=False).float())
        g["embed"] = torch.zeros_like(self.master["embed"]).index_add(0, tokens, dx)
        return loss.sum() / counts, g

    def update(self, grads, rate):
        for name, g in grads.items():
            v = self.momentum.setdefault(name, torch.zeros_like(g))
            v.mul_(0.9).add_(g)
            self.master[name] -= rate * v
            self.w[name].copy_(self.master[name])

    def next_token(self, token):
        """The most likely token after one token: single rows through every product."""
        s = self.forward(token, keep=False)
        return self.dense(s["y2"], self.w["head"]).float().argmax(1)


def train(steps=60, batch=512, vocab=1000, seed=0):
    """(losses, share of tokens whose successor the trained model names)."""
    g = torch.Generator().manual_seed(seed + 1)
    model = Model(vocab=vocab, seed=seed)
    successor = torch.randperm(vocab, generator=g).cuda()
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, vocab, (batch,), generator=g).cuda()
        target = successor[tokens]
        target[::16] = -100                        # some rows that do not count
        loss, grads = model.loss_and_gradients(tokens, target)
        model.update(grads, 0.5)
        losses.append(loss)
    losses = [float(v) for v in losses]
    probe = torch.arange(64, device="cuda")
    right = sum(int(model.next_token(probe[i:i + 1])[0] == successor[i]) for i in range(64)) / 64
    return losses, right


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--steps", type=int, default=60)
    losses, right = train(a.parse_args().steps)
    for i in range(0, len(losses), 10):
        print(f"step {i:4d}  loss {losses[i]:.3f}")
    print(f"last loss {losses[-1]:.3f} (log vocabulary {math.log(1000):.3f}); {100 * right:.0f} % of single tokens right")
