"""Gated feed-forward products, a head's distillation loss and log probabilities, as cases that can be timed.

Six kinds of calls:

  gated          D = act(alpha A op(Bg) + bg) * (alpha A op(Bu) + bu), with both factors before the
                 activation kept for the backward pass; single tokens up to whole batches.
  grouped_gated  the same for each expert's rows, given by offsets on the device.
  gated_grad     with E = alpha A op(B), the gradient that reaches the block's middle: dG = E U act'(G),
                 dU = E act(G), their column sums, and H = act(G) U formed again; `groups` > 0: of experts' rows.
  distill        the loss of a linear head's logits X W^T against a teacher's top logits, without keeping the logits.
  distill_train  the same with the gradients of X and W.
  logprobs       of stored logits: the log probability of a given token, the entropy and the top alternatives.

Where ``own`` is false the operators are computed in their plain form (elementary torch operations
in 32 bits); where it is true by the library's entry points."""
import math

import torch

own = False

F = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a feed-forward block's first half: serving, where latency counts
        dict(name="gated_one_token", kind="gated", m=1, n=8192, k=4096, type="bf16", out="bf16", tb=True, act="silu",
             bias=False, keep=False),
        # a few dozen tokens of odd count, odd widths
        dict(name="gated_odd_small", kind="gated", m=39, n=2501, k=1001, type="f16", out="f32", tb=False,
             act="gelu_tanh", bias=True, keep=False),
        # a training batch that keeps both factors
        dict(name="gated_batch", kind="gated", m=8192, n=4096, k=2048, type="bf16", out="bf16", tb=True, act="silu",
             bias=False, keep=True),
        # experts while serving: a few rows for each, all weights read
        dict(name="grouped_gated_tokens", kind="grouped_gated", m=64, groups=32, n=1408, k=2048, type="bf16", out="bf16",
             tb=True, act="silu", bias=False, keep=False, skew=0.5),
        # experts over a prompt or a training batch
        dict(name="grouped_gated_batch", kind="grouped_gated", m=16384, groups=64, n=1408, k=2048, type="bf16",
             out="bf16", tb=True, act="silu", bias=False, keep=True, skew=0.5),
        # the backward pass of the batch
        dict(name="gated_grad_batch", kind="gated_grad", m=4096, groups=0, n=8192, k=4096, type="bf16", out="bf16",
             tb=False, act="silu", remake=True, skew=0.0),
        # the same of a few experts, ragged and uneven
        dict(name="gated_grad_experts", kind="gated_grad", m=1999, groups=7, n=1490, k=1003, type="f16", out="f16",
             tb=True, act="gelu_tanh", remake=False, skew=2.0),
        # how far a student is from a teacher on a few tokens: the head's weights are read once
        dict(name="distill_few_tokens", kind="distill", m=8, n=32000, k=4096, type="bf16", top=20, mass="kept",
             ignored=0.0),
        # a small training step over an odd vocabulary, part of the teacher's mass beyond its top logits
        dict(name="distill_train_odd", kind="distill_train", m=517, n=50021, k=1000, type="f16", top=33, mass="given",
             ignored=0.1),
        # a training step of the head
        dict(name="distill_train_batch", kind="distill_train", m=4096, n=128000, k=4096, type="bf16", top=64,
             mass="kept", ignored=0.1),
        # single tokens while serving, with alternatives
        dict(name="logprobs_tokens", kind="logprobs", m=16, n=128000, type="f32", alpha=1.25, top=20, masked=0.01),
        # a prompt's log probabilities
        dict(name="logprobs_prompt", kind="logprobs", m=4095, n=128000, type="bf16", alpha=1.0, top=8, masked=0.0),
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; two in five are odd ones, the others multiples of 8 where they can be."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 16 and rng.random() < 0.6:
        v = v // 8 * 8
    return max(lo, min(hi, v))


def draw(rng):
    kind = rng.choice(["gated", "gated", "grouped_gated", "gated_grad", "gated_grad", "distill", "distill_train", "logprobs",
                       "logprobs"])
    t = rng.choice(["bf16", "f16"])
    out = rng.choice([t, t, "f32"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "silu"])
    if kind == "gated":
        return dict(kind=kind, m=_log(rng, 1, 8192), n=_log(rng, 128, 8192), k=_log(rng, 64, 4096), type=t, out=out,
                    tb=rng.random() < 0.6, act=act, bias=rng.random() < 0.4, keep=rng.random() < 0.5)
    if kind == "grouped_gated":
        return dict(kind=kind, m=_log(rng, 8, 16384), groups=_log(rng, 2, 64), n=_log(rng, 128, 2048),
                    k=_log(rng, 128, 2048), type=t, out=out, tb=rng.random() < 0.6, act=act, bias=rng.random() < 0.4,
                    keep=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 2.0]))
    if kind == "gated_grad":
        groups = rng.choice([0, 0, _log(rng, 2, 64)])
        return dict(kind=kind, m=_log(rng, 64, 8192), groups=groups, n=_log(rng, 128, 2048 if groups else 8192),
                    k=_log(rng, 64, 2048 if groups else 4096), type=t, out=out, tb=rng.random() < 0.5, act=act,
                    remake=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 2.0]) if groups else 0.0)
    if kind == "logprobs":
        return dict(kind=kind, m=_log(rng, 1, 4096), n=_log(rng, 1000, 128000), type=rng.choice(["bf16", "f16", "f32"]),
                    alpha=rng.choice([1.0, 1.25, 0.5]), top=rng.choice([0, 1, 5, 20, 64]), masked=rng.choice([0.0, 0.01, 0.5]))
    return dict(kind=kind, m=_log(rng, 16 if kind == "distill_train" else 1, 4096), n=_log(rng, 2000, 128000),
                k=_log(rng, 256, 4096), type=t, top=_log(rng, 1, 128), mass=rng.choice(["kept", "given"]),
                ignored=rng.choice([0.0, 0.1, 0.5]))


# ----------------------------------------------------------------------------- inputs
def _up8(v):
    return -(-v // 8) * 8


def _matrix(rows, cols, dtype, gen, scale=1.0):
    """rows x cols random normal values in rows of whole 16-byte blocks, as the library's alignment asks."""
    return (torch.randn(rows, _up8(cols), device="cuda", generator=gen) * scale).to(dtype)[:, :cols]


def _experts(case, seed):
    """Rows of each expert: a draw from uneven shares, as a router's choices are."""
    gen = torch.Generator().manual_seed(seed + 7919)
    share = torch.softmax(case["skew"] * torch.randn(case["groups"], generator=gen), 0)
    where = torch.multinomial(share, case["m"], replacement=True, generator=gen)
    counts = torch.bincount(where, minlength=case["groups"])
    ends = counts.cumsum(0)
    return torch.cat([torch.zeros(1, dtype=torch.int64), ends]), int(counts.max())


def _halves(x, n):
    """The gate's and the up projection's columns of a matrix that holds both, each from a whole 16-byte block."""
    return x[..., :n], x[..., _up8(n):_up8(n) + n]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    t = F[case["type"]]
    kind, m, n = case["kind"], case["m"], case["n"]
    if kind in ("gated", "grouped_gated", "gated_grad"):
        k = case["k"]
        groups = case.get("groups", 0)
        if groups:
            offsets, s["most"] = _experts(case, seed)
            s["offsets"] = offsets.to(torch.int32).cuda()
        e = max(groups, 1)
        s["A"] = _matrix(m, k, t, gen)
        both = 1 if kind == "gated_grad" else 2
        if case["tb"]:                       # gate rows, then up rows
            s["B"] = _matrix(e * both * n, k, t, gen, k ** -0.5).unflatten(0, (e, both * n))
        else:                                # gate columns, then up columns
            s["B"] = _matrix(e * k, both * _up8(n) if both == 2 else n, t, gen, k ** -0.5).unflatten(0, (e, k))
        if kind == "gated_grad":
            s["kept"] = _matrix(m, 2 * _up8(n), t, gen)
        else:
            s["biases"] = torch.randn(2, e, n, device="cuda", generator=gen).mul(0.5).to(t) if case["bias"] else None
    elif kind == "logprobs":
        z = _matrix(m, n, torch.float32, gen, 3.0)
        taken = torch.rand(n, device="cuda", generator=gen) >= case["masked"]
        z[:, ~taken] = -math.inf             # tokens that may not be taken
        s["Z"] = torch.zeros(m, _up8(n), device="cuda", dtype=t)[:, :n].copy_(z)
        allowed = taken.nonzero()[:, 0]
        s["target"] = allowed[torch.randint(0, allowed.numel(), (m,), device="cuda", generator=gen)]
    else:
        k, top = case["k"], case["top"]
        s["X"] = _matrix(m, k, t, gen)
        s["W"] = _matrix(n, k, t, gen, 2.0 * k ** -0.5)
        # a teacher's top tokens: different ones, their logits falling; some rows have fewer, some none
        start = torch.randint(0, n, (m, 1), device="cuda", generator=gen)
        step = torch.randint(1, max(2, n // top), (m, 1), device="cuda", generator=gen)
        j = torch.arange(top, device="cuda")
        index = (start + j * step) % n
        fewer = torch.rand(m, 1, device="cuda", generator=gen) < 0.1
        index = torch.where(fewer & (j >= (top + 1) // 2), -1, index)
        out = torch.rand(m, 1, device="cuda", generator=gen) < case["ignored"]
        s["index"] = torch.where(out, torch.full_like(index, -1), index)
        s["logit"] = (torch.randn(m, top, device="cuda", generator=gen) * 2 + 6).sort(1, descending=True).values
        beyond = torch.rand(m, device="cuda", generator=gen) * 0.5
        s["teacher_lse"] = torch.logsumexp(s["logit"] * 0.5, 1) + beyond if case["mass"] == "given" else None
        # the gradient that comes in: that of a mean over the rows that count, with the usual
        # loss scale where fp16 needs one
        g = (65536.0 if case["type"] == "f16" else 1.0) / max(1, m * (1 - case["ignored"]))
        s["g"] = torch.full((m,), g, device="cuda")
    return s


TEACHER = 0.5   # what the teacher's logits are multiplied by: temperature 2


# ----------------------------------------------------------------------------- plain forms
def _act(name, z):
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def _rows_of(s):
    """Expert and place within it of every row."""
    row = torch.arange(s["m"], device="cuda")
    e = torch.bucketize(row, s["offsets"][1:].long(), right=True)
    return e, row - s["offsets"].long()[e]


def _product(s, b):
    """A op(B_e) of every row, in 32 bits; b: experts x ..., with the rows' experts."""
    b = b.float()
    b = b.transpose(1, 2).contiguous() if s["tb"] else b
    if not s.get("groups"):
        return s["A"].float() @ b[0]
    e, place = _rows_of(s)
    a = torch.zeros(s["groups"], s["most"], s["k"], device="cuda")
    a[e, place] = s["A"].float()
    return torch.bmm(a, b.contiguous())[e, place]


def _weights(s):
    """The gate's and the up projection's weights, experts x (n x k or k x n)."""
    n = s["n"]
    if s["tb"]:
        return s["B"][:, :n], s["B"][:, n:]
    return _halves(s["B"], n)


def _plain(s):
    kind, n = s["kind"], s["n"]
    t = F[s["type"]]
    if kind in ("gated", "grouped_gated"):
        bg, bu = _weights(s)
        g, u = _product(s, bg), _product(s, bu)
        if s["bias"]:
            e = _rows_of(s)[0] if s.get("groups") else torch.zeros(s["m"], dtype=torch.int64, device="cuda")
            g, u = g + s["biases"][0].float()[e], u + s["biases"][1].float()[e]
        r = {"D": (_act(s["act"], g) * u).to(F[s["out"]])}
        if s["keep"]:
            r["G"], r["U"] = g.to(t), u.to(t)
        return r
    if kind == "gated_grad":
        d = _product(s, s["B"])
        g, u = (x.float() for x in _halves(s["kept"], n))
        a = _act(s["act"], g)
        dg, du = d * u * _act_slope(s["act"], g), d * a
        e = _rows_of(s)[0] if s["groups"] else torch.zeros(s["m"], dtype=torch.int64, device="cuda")
        sums = torch.zeros(max(s["groups"], 1), 2, n, device="cuda")
        sums[:, 0].index_add_(0, e, dg)
        sums[:, 1].index_add_(0, e, du)
        r = {"dG": dg.to(F[s["out"]]), "dU": du.to(F[s["out"]]), "dbias": sums}
        if s["remake"]:
            r["H"] = (a * u).to(t)
        return r
    if kind == "logprobs":
        z = s["Z"].float() * s["alpha"]
        top = z.amax(1, keepdim=True)
        e = torch.exp(z - top)
        total = e.sum(1)
        lse = top[:, 0] + torch.log(total)
        below = torch.where(e > 0, (z - top) * e, torch.zeros_like(e)).sum(1)
        r = {"logprob": z.gather(1, s["target"][:, None])[:, 0] - lse, "lse": lse, "entropy": torch.log(total) - below / total}
        if s["top"]:
            # by value, then by the lower index: one key of both (the sign of a float's bits turned into an order)
            bits = (s["Z"].float() + 0.0).view(torch.int32)   # (+ 0.0: the two zeros are one value)
            order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
            key = order * (1 << 24) + (s["n"] - 1 - torch.arange(s["n"], device="cuda"))
            best = torch.topk(key, s["top"], dim=1, sorted=True).values
            at = s["n"] - 1 - best % (1 << 24)
            r["top_index"] = at
            r["top_logprob"] = z.gather(1, at) - lse[:, None]
        return r
    x, w = s["X"].float(), s["W"].float()
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(1, keepdim=True)
    lse = top + torch.log(total)
    counts = s["index"] >= 0
    at = torch.where(counts, s["index"], torch.zeros_like(s["index"]))
    picked = torch.where(counts, logits.gather(1, at), torch.zeros_like(s["logit"]))
    y = torch.where(counts, s["logit"] * TEACHER, torch.full_like(s["logit"], -math.inf))
    if s["mass"] == "given":
        level = s["teacher_lse"][:, None]
    else:
        most = y.amax(1, keepdim=True).clamp(min=-1e30)
        level = most + torch.log(torch.exp(y - most).sum(1, keepdim=True))
    level = torch.where(counts.any(1, keepdim=True), level, torch.zeros_like(level))
    q = torch.exp(y - level)
    loss = torch.where(counts, q * (y.clamp(min=-1e30) - level - picked + lse), torch.zeros_like(q)).sum(1)
    r = {"loss": loss, "lse": lse[:, 0], "picked": picked}
    if kind == "distill_train":
        p = p / total * q.sum(1, keepdim=True)
        p.scatter_add_(1, at, -q)
        p = p * s["g"][:, None]
        r["dX"] = (p @ w).to(t)
        r["dW"] = (p.t() @ x).to(t)
    return r


# ----------------------------------------------------------------------------- the library's calls
_kept = {}


def _library():
    """The library and one handle, which a program makes once."""
    if not _kept:
        import mixed_precision_dense_amd as mp
        _kept["mp"], _kept["h"] = mp, mp.Handle()
    return _kept["mp"], _kept["h"].h


def _new(rows, cols, dtype):
    return torch.empty(rows, _up8(cols), device="cuda", dtype=dtype)[:, :cols]


def _workspace(size):
    return torch.empty(size, dtype=torch.uint8, device="cuda")


def _own(s):
    mp, h = _library()
    kind, t, m, n = s["kind"], s["type"], s["m"], s["n"]
    n8 = _up8(n)
    if kind in ("gated", "grouped_gated"):
        k, b = s["k"], s["B"]
        d = _new(m, n, F[s["out"]])
        both = _new(m, 2 * n8, F[t]) if s["keep"] else None
        bias = s["biases"]
        gated = mp.Gated(act=s["act"], bias_gate=None if bias is None else bias[0], bias_up=None if bias is None else bias[1],
                         bias_type=t, bias_stride=n, kept=both, ld_kept=2 * n8, stride_kept=n8)
        up = n * b.stride(1) if s["tb"] else n8
        if kind == "gated":
            mp.mpgemm_run_gated(h, s["tb"], m, n, k, 1.0, s["A"], t, s["A"].stride(0), b, t, b.stride(1), up, gated, d,
                                s["out"], d.stride(0))
        else:
            mp.mpgemm_run_grouped_gated(h, s["tb"], s["groups"], m, n, k, 1.0, s["A"], t, s["A"].stride(0), s["offsets"], b, t,
                                        b.stride(1), b.stride(0), up, gated, d, s["out"], d.stride(0))
        r = {"D": d}
        if s["keep"]:
            r["G"], r["U"] = _halves(both, n)
        return r
    if kind == "gated_grad":
        k, b, groups = s["k"], s["B"], s["groups"]
        d = _new(m, 2 * n8, F[s["out"]])
        sums = torch.empty(max(groups, 1), 2, n, device="cuda")
        made = _new(m, n, F[t]) if s["remake"] else None
        size = mp.mpgemm_gated_grad_workspace_size(max(groups, 1), m, n)
        grad = mp.GatedGrad(act=s["act"], kept=s["kept"], ld_kept=s["kept"].stride(0), stride_kept=n8, H=made, ldh=n8,
                            dbias=sums)
        if groups:
            mp.mpgemm_run_grouped_gated_grad(h, s["tb"], groups, m, n, k, 1.0, s["A"], t, s["A"].stride(0), s["offsets"], b, t,
                                             b.stride(1), b.stride(0), grad, d, s["out"], d.stride(0), n8, _workspace(size),
                                             size)
        else:
            mp.mpgemm_run_gated_grad(h, s["tb"], m, n, k, 1.0, s["A"], t, s["A"].stride(0), b, t, b.stride(1), grad, d, s["out"],
                                     d.stride(0), n8, _workspace(size), size)
        dg, du = _halves(d, n)
        r = {"dG": dg, "dU": du, "dbias": sums}
        if s["remake"]:
            r["H"] = made
        return r
    if kind == "logprobs":
        top = s["top"]
        logprob, lse, entropy = (torch.empty(m, device="cuda") for _ in range(3))
        at = torch.empty(m, top, dtype=torch.int64, device="cuda") if top else None
        value = torch.empty(m, top, device="cuda") if top else None
        size = mp.mpgemm_logprobs_workspace_size(m, n, t, top)
        mp.mpgemm_run_logprobs(h, m, n, s["alpha"], s["Z"], t, s["Z"].stride(0), s["target"], logprob, lse, entropy, top, at,
                               value, top, _workspace(size), size)
        r = {"logprob": logprob, "lse": lse, "entropy": entropy}
        if top:
            r["top_index"], r["top_logprob"] = at, value
        return r
    k, top, x, w = s["k"], s["top"], s["X"], s["W"]
    loss, lse = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    picked = torch.empty(m, top, device="cuda")
    train = kind == "distill_train"
    size = mp.mpgemm_linear_distill_workspace_size(m, n, k, top, t, train)
    ws = _workspace(size)
    teacher = mp.Teacher(top, s["index"], s["logit"], top, scale=TEACHER, lse=s["teacher_lse"])
    mp.mpgemm_run_linear_distill(h, m, n, k, 1.0, x, t, x.stride(0), w, w.stride(0), teacher, loss, lse, picked, ws, size)
    r = {"loss": loss, "lse": lse, "picked": picked}
    if train:
        dx, dw = _new(m, k, F[t]), _new(n, k, F[t])
        mp.mpgemm_run_linear_distill_grad(h, m, n, k, 1.0, x, t, x.stride(0), w, w.stride(0), teacher, lse, picked, s["g"], dx,
                                          dx.stride(0), dw, dw.stride(0), ws, size)
        r["dX"], r["dW"] = dx, dw
    return r


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- what cannot be done without
def work(case):
    kind, m, n = case["kind"], case["m"], case["n"]
    tb = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
    ob = {"bf16": 2, "f16": 2, "f32": 4}[case.get("out", case["type"])]
    if kind in ("gated", "grouped_gated", "gated_grad"):
        k, groups = case["k"], case.get("groups", 0)
        used = groups * (1 - math.exp(-m / groups)) if groups else 1   # experts that have rows, where the shares are even
        if kind == "gated_grad":
            b = tb * (m * k + used * k * n + 2 * m * n + m * n * case["remake"]) + ob * 2 * m * n + 8 * n * max(groups, 1)
            return {"bytes": int(b), "flops": 2 * m * n * k}
        b = tb * (m * k + 2 * used * k * n + 2 * m * n * case["keep"] + 2 * used * n * case["bias"]) + ob * m * n
        return {"bytes": int(b), "flops": 4 * m * n * k}
    if kind == "logprobs":
        # an element: its scaling, exponential, two sums and a comparison
        return {"bytes": tb * m * n + 20 * m + 12 * m * case["top"], "flops": 6 * m * n}
    k, top = case["k"], case["top"]
    if kind == "distill":
        return {"bytes": tb * (m * k + n * k) + 16 * m * top + 8 * m, "flops": 2 * m * n * k}
    return {"bytes": 2 * tb * (m * k + n * k) + 16 * m * top + 12 * m, "flops": 6 * m * n * k}


# ----------------------------------------------------------------------------- the definition, in 64 bits
def _act64(name, z):
    """(value, slope) of the activation."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        g = torch.sigmoid(z)
        return z * g, g + z * g * torch.sigmoid(-z)
    if name == "gelu":
        c = torch.special.ndtr(z)
        return z * c, c + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    # gelu_tanh: z sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
    u2 = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    g = torch.sigmoid(u2)
    return z * g, g + z * g * torch.sigmoid(-u2) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z.square())


def exact(case, seed):
    s = prepare(case, seed)
    kind, m, n = case["kind"], case["m"], case["n"]
    if kind in ("gated", "grouped_gated", "gated_grad"):
        groups = case.get("groups", 0)
        ends = s["offsets"].tolist() if groups else [0, m]
        both = 1 if kind == "gated_grad" else 2
        parts = [torch.zeros(m, n, dtype=torch.float64, device="cuda") for _ in range(both)]
        for e in range(len(ends) - 1):
            rows = slice(ends[e], ends[e + 1])
            if ends[e] == ends[e + 1]:
                continue
            a = s["A"][rows].double()
            for h in range(both):
                if case["tb"]:
                    parts[h][rows] = a.mm(s["B"][e, h * n:(h + 1) * n].double().T)
                else:
                    first = h * _up8(n)
                    parts[h][rows] = a.mm(s["B"][e, :, first:first + n].double())
                if both == 2 and case["bias"]:
                    parts[h][rows] += s["biases"][h, e].double()
        if both == 2:
            g, u = parts
            r = {"D": _act64(case["act"], g)[0].mul_(u)}
            if case["keep"]:
                r["G"], r["U"] = g, u
            return r
        g = s["kept"][:, :n].double()
        u = s["kept"][:, _up8(n):_up8(n) + n].double()
        value, slope = _act64(case["act"], g)
        dg, du = parts[0] * u * slope, parts[0] * value
        sums = torch.stack([torch.stack([d[ends[e]:ends[e + 1]].sum(0) for d in (dg, du)]) for e in range(len(ends) - 1)])
        r = {"dG": dg, "dU": du, "dbias": sums}
        if case["remake"]:
            r["H"] = value * u
        return r
    if kind == "logprobs":
        out = {"logprob": [], "lse": [], "entropy": [], "top_index": [], "top_logprob": []}
        for r0 in range(0, m, 1024):   # blocks of rows: a stable sort of all of them would not fit three times
            raw = s["Z"][r0:r0 + 1024].double()
            z = raw * case["alpha"]
            lp = z - torch.logsumexp(z, 1, keepdim=True)
            p = lp.exp()
            out["lse"].append(torch.logsumexp(z, 1))
            out["logprob"].append(lp.gather(1, s["target"][r0:r0 + 1024, None])[:, 0])
            out["entropy"].append(-torch.special.xlogy(p, p).sum(1))
            if case["top"]:
                at = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :case["top"]].clone()
                out["top_index"].append(at)
                out["top_logprob"].append(lp.gather(1, at))
        return {name: torch.cat(v) for name, v in out.items() if v}
    x, w = s["X"].double(), s["W"].double()
    logits = x.mm(w.T)
    lse = torch.logsumexp(logits, 1)
    row, entry = (s["index"] >= 0).nonzero(as_tuple=True)
    col = s["index"][row, entry]
    log_q = torch.full(s["logit"].shape, -math.inf, dtype=torch.float64, device="cuda")
    log_q[row, entry] = s["logit"][row, entry].double() * TEACHER
    if case["mass"] == "given":
        log_q -= s["teacher_lse"].double()[:, None]
    else:
        some = torch.zeros(m, dtype=torch.bool, device="cuda")
        some[row] = True
        log_q[some] = torch.log_softmax(log_q[some], 1)
    q = log_q.exp()
    picked = torch.zeros_like(q)
    picked[row, entry] = logits[row, col]
    loss = torch.zeros_like(lse).index_add_(0, row, q[row, entry] * (log_q[row, entry] - logits[row, col] + lse[row]))
    r = {"loss": loss, "lse": lse, "picked": picked}
    if kind == "distill_train":
        logits.sub_(lse[:, None]).exp_()
        logits.mul_(q.sum(1, keepdim=True))
        logits[row, col] -= q[row, entry]
        logits.mul_(s["g"].double()[:, None])
        r["dX"], r["dW"] = logits.mm(w), logits.T.mm(x)
    return r
