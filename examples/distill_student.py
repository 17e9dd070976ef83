"""A student that learns from a teacher's answers, made of the library's products: the teacher's log
probabilities and alternatives, a gated feed-forward block and gated experts, and the distillation loss
of the head, forward and backward; then the student's own log probabilities of single tokens.

    python examples/distill_student.py [--steps 60]

Every matrix product and everything around it runs in the library; torch holds the memory, routes the
tokens and updates the weights.  The teacher is a random linear map of the current token, so that the
loss falls towards 0 as the student comes to agree with it.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_dense_amd as mp  # noqa: E402

T, TYPE = "bf16", torch.bfloat16


def new(*shape, dtype=TYPE):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def logprobs(h, logits, target=None, top=0, alpha=1.0):
    """(log probability of the targets, log-sum-exp, entropy, columns and log probabilities of the alternatives)."""
    m, n = logits.shape
    t = "f32" if logits.dtype == torch.float32 else T
    own = new(m, dtype=torch.float32) if target is not None else None
    lse, entropy = new(m, dtype=torch.float32), new(m, dtype=torch.float32)
    at, value = new(m, top, dtype=torch.int64), new(m, top, dtype=torch.float32)
    size = mp.mpgemm_logprobs_workspace_size(m, n, t, top)
    mp.mpgemm_run_logprobs(h, m, n, alpha, logits, t, logits.stride(0), target, own, lse, entropy, top, at if top else None,
                           value if top else None, top, new(size, dtype=torch.uint8), size)
    return own, lse, entropy, at, value


class Teacher:
    """Answers a token with the `top` most likely successors and their log probabilities."""

    def __init__(self, vocab, width, top, seed):
        g = torch.Generator().manual_seed(seed)
        self.h, self.vocab, self.width, self.top = mp.Handle(), vocab, width, top
        self.embed = torch.randn(vocab, width, generator=g).cuda().to(TYPE)
        self.head = (torch.randn(vocab, width, generator=g) * 3 * width ** -0.5).cuda().to(TYPE)

    def answer(self, tokens):
        x, m, n, k = self.embed[tokens], tokens.numel(), self.vocab, self.width
        logits = new(m, n, dtype=torch.float32)
        mp.mpgemm_run(self.h.h, False, True, m, n, k, 1.0, x, T, k, self.head, T, k, 0.0, None, "f32", n, logits, "f32")
        _, _, _, at, value = logprobs(self.h.h, logits, top=self.top)
        return at, value


class Student:
    """Sizes are multiples of 8, so that rows are whole 16-byte blocks."""

    def __init__(self, vocab=1000, width=64, inner=128, experts=4, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.h = mp.Handle()
        self.vocab, self.width, self.inner, self.experts = vocab, width, inner, experts

        def weight(*shape):
            return (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).cuda()

        # FP32 masters; the products take BF16 copies.  A gated block's two projections are one matrix: the gate's
        # rows, then the up projection's.
        self.master = {"embed": weight(vocab, width) * width ** 0.5, "gated": weight(2 * inner, width), "down": weight(width, inner),
                       "egated": weight(experts, 2 * inner, width), "edown": weight(experts, width, inner),
                       "head": weight(vocab, width), "bias": torch.zeros(2, inner, device="cuda")}
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
    def product(self, a, w, residual=None, transposed=True):
        """a w^T (transposed=False: a w) + residual."""
        m, k = a.shape
        n = w.shape[0] if transposed else w.shape[1]
        d = new(m, n)
        mp.mpgemm_run_epilogue(self.h.h, False, transposed, m, n, k, 1.0, a, T, k, w, T, w.stride(0), mp.Epilogue(),
                               0.0 if residual is None else 1.0, residual, T, n, d, T, n)
        return d

    def weight_grad(self, dy, x):
        m, n = dy.shape[1], x.shape[1]
        d = new(m, n, dtype=torch.float32)
        mp.mpgemm_run(self.h.h, True, False, m, n, dy.shape[0], 1.0, dy, T, m, x, T, n, 0.0, None, "f32", n, d, "f32")
        return d

    def gated(self, x, keep):
        """silu(x G^T + b) (x U^T + b'), with both factors kept."""
        m, k, n = x.shape[0], self.width, self.inner
        d = new(m, n)
        mp.mpgemm_run_gated(self.h.h, True, m, n, k, 1.0, x, T, k, self.w["gated"], T, k, n * k,
                            mp.Gated(act="silu", bias_gate=self.master["bias"][0], bias_up=self.master["bias"][1], kept=keep,
                                     ld_kept=2 * n, stride_kept=n), d, T, n)
        return d

    def gated_grad(self, dy, kept):
        """The gradients of both factors, side by side in the place of what was kept, and their column sums."""
        m, k, n = dy.shape[0], self.width, self.inner
        sums, size = new(2, n, dtype=torch.float32), mp.mpgemm_gated_grad_workspace_size(1, m, n)
        mp.mpgemm_run_gated_grad(self.h.h, False, m, n, k, 1.0, dy, T, k, self.w["down"], T, n,
                                 mp.GatedGrad(act="silu", kept=kept, ld_kept=2 * n, stride_kept=n, dbias=sums), kept, T, 2 * n, n,
                                 new(size, dtype=torch.uint8), size)
        return kept, sums

    def experts_gated(self, x, offsets, keep):
        m, k, n = x.shape[0], self.width, self.inner
        d = new(m, n)
        mp.mpgemm_run_grouped_gated(self.h.h, True, self.experts, m, n, k, 1.0, x, T, k, offsets, self.w["egated"], T, k, 2 * n * k,
                                    n * k, mp.Gated(act="silu", kept=keep, ld_kept=2 * n, stride_kept=n), d, T, n)
        return d

    def experts_gated_grad(self, dy, offsets, kept):
        """The gradients of both factors side by side, and the block's middle formed again."""
        m, k, n = dy.shape[0], self.width, self.inner
        d, made = new(m, 2 * n), new(m, n)
        mp.mpgemm_run_grouped_gated_grad(self.h.h, False, self.experts, m, n, k, 1.0, dy, T, k, offsets, self.w["edown"], T, n, k * n,
                                         mp.GatedGrad(act="silu", kept=kept, ld_kept=2 * n, stride_kept=n, H=made, ldh=n), d, T, 2 * n,
                                         n, None, 0)
        return d, made

    def experts_product(self, a, w, offsets, transposed=True):
        rows, k = a.shape
        n = w.shape[1] if transposed else w.shape[2]
        d = new(rows, n)
        mp.mpgemm_run_grouped(self.h.h, transposed, self.experts, rows, n, k, 1.0, a, T, k, offsets, w, T, w.stride(1), w.stride(0),
                              mp.Epilogue(), d, T, n)
        return d

    def experts_weight_grad(self, dy, x, offsets):
        rows, m = dy.shape
        n = x.shape[1]
        d = new(self.experts, m, n, dtype=torch.float32)
        mp.mpgemm_run_grouped_wgrad(self.h.h, self.experts, rows, m, n, 1.0, dy, T, m, x, T, n, offsets, 0.0, d, "f32", n, m * n)
        return d

    # ------------------------------------------------------------------ the model
    def forward(self, tokens, keep=True):
        w, s, rows = self.w, {}, tokens.numel()
        s["x"] = w["embed"][tokens]
        s["kept"] = new(rows, 2 * self.inner) if keep else None
        s["h"] = self.gated(s["x"], s["kept"])
        s["y"] = self.product(s["h"], w["down"], s["x"])
        s["order"], s["offsets"] = self.route(tokens)
        s["ys"] = s["y"][s["order"]]
        s["ekept"] = new(rows, 2 * self.inner) if keep else None
        out = self.experts_product(self.experts_gated(s["ys"], s["offsets"], s["ekept"]), w["edown"], s["offsets"])
        s["y2"] = s["y"].index_add(0, s["order"], out)
        return s

    def loss_and_gradients(self, tokens, index, logit):
        """Against the teacher's top log probabilities, whose log-sum-exp over all columns is 0."""
        w, s = self.w, self.forward(tokens)
        m, n, k, top = tokens.numel(), self.vocab, self.width, index.shape[1]
        size = mp.mpgemm_linear_distill_workspace_size(m, n, k, top, T, True)
        ws = new(size, dtype=torch.uint8)
        loss, lse, picked = (new(m, c, dtype=torch.float32) for c in (1, 1, top))
        teacher = mp.Teacher(top, index, logit, top, lse=torch.zeros(m, device="cuda"))
        mp.mpgemm_run_linear_distill(self.h.h, m, n, k, 1.0, s["y2"], T, k, w["head"], k, teacher, loss, lse, picked, ws, size)
        counts = (index >= 0).any(1).sum().clamp(min=1)
        weight = (1.0 / counts).float().expand(m).contiguous()
        dy2, dhead = new(m, k), new(n, k)
        mp.mpgemm_run_linear_distill_grad(self.h.h, m, n, k, 1.0, s["y2"], T, k, w["head"], k, teacher, lse, picked, weight, dy2, k,
                                          dhead, k, ws, size)
        g = {"head": dhead.float()}
        dout = dy2[s["order"]]
        dpair, made = self.experts_gated_grad(dout, s["offsets"], s["ekept"])
        g["edown"] = self.experts_weight_grad(dout, made, s["offsets"])
        g["egated"] = self.experts_weight_grad(dpair, s["ys"], s["offsets"])
        dy = dy2.index_add(0, s["order"], self.experts_product(dpair, w["egated"], s["offsets"], transposed=False))
        g["down"] = self.weight_grad(dy, s["h"])
        dpair, g["bias"] = self.gated_grad(dy, s["kept"])
        g["gated"] = self.weight_grad(dpair, s["x"])
        dx = self.product(dpair, w["gated"], dy, transposed=False)
        g["embed"] = torch.zeros_like(self.master["embed"]).index_add(0, tokens, dx.float())
        return loss.sum() / counts, g

    def update(self, grads, rate):
        for name, g in grads.items():
            v = self.momentum.setdefault(name, torch.zeros_like(g))
            v.mul_(0.9).add_(g)
            self.master[name] -= rate * v
            self.w[name].copy_(self.master[name])

    def answer(self, tokens, target=None, top=4):
        """(log probability of the targets, entropy, the alternatives' columns and log probabilities)."""
        s = self.forward(tokens, keep=False)
        own, _, entropy, at, value = logprobs(self.h.h, self.product(s["y2"], self.w["head"]), target, top)
        return own, entropy, at, value


def train(steps=60, batch=512, vocab=1000, top=32, seed=0):
    """(student, teacher, losses)."""
    g = torch.Generator().manual_seed(seed + 1)
    teacher, student, losses = Teacher(vocab, 48, top, seed + 2), Student(vocab, seed=seed), []
    for _ in range(steps):
        tokens = torch.randint(0, vocab, (batch,), generator=g).cuda()
        index, value = teacher.answer(tokens)
        index[::16] = -1                           # some rows that do not count
        loss, grads = student.loss_and_gradients(tokens, index, value)
        student.update(grads, 0.5)
        losses.append(loss)
    return student, teacher, [float(v) for v in losses]


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--steps", type=int, default=60)
    student, teacher, losses = train(a.parse_args().steps)
    for i in range(0, len(losses), 10):
        print(f"step {i:4d}  loss {losses[i]:.3f}")
    tokens = torch.arange(8, device="cuda")
    best = teacher.answer(tokens)[0][:, 0].contiguous()
    own, entropy, at, value = student.answer(tokens, best)
    for i in range(8):
        print(f"token {i}: teacher's choice {int(best[i])} has log probability {float(own[i]):.2f}; alternatives "
              f"{at[i].tolist()}, entropy {float(entropy[i]):.2f}")
