"""The operators of language models that are built on the matrix product, as cases that can be timed.

Three families of calls, each in its forward and its backward direction:

  epilogue       D = act(alpha op(A) op(B) + bias) + beta C, with the value before the activation
                 kept for the backward pass; single tokens (m = 1) up to whole batches.
  epilogue_grad  dZ = act'(Z) * (alpha op(A) op(B)) and the bias gradient (column sums of dZ).
  grouped        D[r] = act(A[r] op(B_e) + bias_e), rows r of expert e given by offsets on the
                 device; ragged, some experts without rows.
  grouped_bwd    the gradients of a grouped product: dZ = act'(Z) * (A op(B_e)), the bias
                 gradients of each expert, and a weights' gradient dV_e = A_e^T X_e.
  loss           softmax cross entropy of X W^T over a large vocabulary, without keeping the logits.
  loss_train     the same with the gradients of X and W.

Where ``own`` is false the operators are computed in their plain form (elementary torch operations
in 32 bits); where it is true by the library's entry points."""
import math

import torch

own = False

F = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a square projection: serving, where latency counts
        dict(name="epi_one_token", kind="epilogue", m=1, n=4096, k=4096, type="bf16", out="bf16", ta=False, tb=True,
             act="silu", bias=True, aux=False, beta=1.0),
        # a few dozen tokens of odd count, odd widths
        dict(name="epi_odd_small", kind="epilogue", m=37, n=5000, k=1001, type="f16", out="f32", ta=False, tb=False,
             act="gelu_tanh", bias=True, aux=False, beta=0.0),
        # the widening half of a feed-forward block over a batch, keeping Z for the backward pass
        dict(name="epi_batch", kind="epilogue", m=8192, n=8192, k=2048, type="bf16", out="bf16", ta=False, tb=True,
             act="gelu", bias=True, aux=True, beta=0.0),
        # the narrowing half's gradient through the activation, ragged sizes
        dict(name="epi_grad_ragged", kind="epilogue_grad", m=5000, n=3000, k=1000, type="f16", out="f16", ta=False,
             tb=True, act="gelu_tanh"),
        # the same over a batch
        dict(name="epi_grad_batch", kind="epilogue_grad", m=4096, n=8192, k=4096, type="bf16", out="bf16", ta=False,
             tb=False, act="silu"),
        # experts while serving: a few rows for each, all weights read
        dict(name="grouped_tokens", kind="grouped", rows=64, groups=32, n=1408, k=2048, type="bf16", out="bf16",
             tb=True, act="silu", bias=False, aux=False, skew=0.5),
        # experts over a prompt or a training batch
        dict(name="grouped_batch", kind="grouped", rows=16384, groups=64, n=2816, k=2048, type="bf16", out="bf16",
             tb=True, act="silu", bias=True, aux=True, skew=0.5),
        # few experts, odd sizes, strongly uneven, some without rows
        dict(name="grouped_odd", kind="grouped", rows=1999, groups=7, n=1490, k=1003, type="f16", out="f32", tb=False,
             act="none", bias=True, aux=False, skew=2.0),
        # gradients of a grouped product
        dict(name="grouped_bwd_batch", kind="grouped_bwd", rows=8192, groups=16, n=4096, k=2048, type="bf16",
             out="bf16", tb=False, act="silu", skew=0.5),
        # log-likelihood of a few tokens: the head's weights are read once
        dict(name="loss_few_tokens", kind="loss", m=8, n=32000, k=4096, type="bf16", ignored=0.0),
        # evaluation with an odd vocabulary
        dict(name="loss_odd", kind="loss", m=2047, n=50021, k=1000, type="f16", ignored=0.1),
        # a training step of the head
        dict(name="loss_train_batch", kind="loss_train", m=4096, n=128000, k=4096, type="bf16", ignored=0.1),
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; two in five are odd ones, the others multiples of 8 where they can be."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 16 and rng.random() < 0.6:
        v = v // 8 * 8
    return max(lo, min(hi, v))


def draw(rng):
    kind = rng.choice(["epilogue", "epilogue", "epilogue_grad", "grouped", "grouped", "grouped_bwd", "loss", "loss_train"])
    t = rng.choice(["bf16", "f16"])
    out = rng.choice([t, t, "f32"])
    acts = ["none", "relu", "gelu", "gelu_tanh", "silu"]
    if kind in ("epilogue", "epilogue_grad"):
        c = dict(kind=kind, m=_log(rng, 1 if kind == "epilogue" else 16, 8192), n=_log(rng, 256, 8192),
                 k=_log(rng, 64, 4096), type=t, out=out, ta=rng.random() < 0.2, tb=rng.random() < 0.6, act=rng.choice(acts))
        if kind == "epilogue":
            c.update(bias=rng.random() < 0.7, aux=rng.random() < 0.4, beta=rng.choice([0.0, 0.0, 1.0, 0.5]))
        return c
    if kind in ("grouped", "grouped_bwd"):
        c = dict(kind=kind, rows=_log(rng, 8 if kind == "grouped" else 64, 16384), groups=_log(rng, 2, 64),
                 n=_log(rng, 128, 4096), k=_log(rng, 128, 2048), type=t, out=out, tb=rng.random() < 0.6,
                 act=rng.choice(acts), skew=rng.choice([0.0, 0.5, 2.0]))
        if kind == "grouped":
            c.update(bias=rng.random() < 0.5, aux=rng.random() < 0.4)
        return c
    big = kind == "loss_train"
    return dict(kind=kind, m=_log(rng, 16 if big else 1, 4096), n=_log(rng, 2000, 128000), k=_log(rng, 256, 4096), type=t,
                ignored=rng.choice([0.0, 0.1, 0.5]))


# ----------------------------------------------------------------------------- inputs
def _matrix(rows, cols, dtype, gen, scale=1.0):
    """rows x cols random normal values in rows of whole 16-byte blocks, as the library's alignment asks."""
    return (torch.randn(rows, -(-cols // 8) * 8, device="cuda", generator=gen) * scale).to(dtype)[:, :cols]


def _experts(case, seed):
    """Rows of each expert: a draw from uneven shares, as a router's choices are."""
    gen = torch.Generator().manual_seed(seed + 7919)
    share = torch.softmax(case["skew"] * torch.randn(case["groups"], generator=gen), 0)
    where = torch.multinomial(share, case["rows"], replacement=True, generator=gen)
    counts = torch.bincount(where, minlength=case["groups"])
    ends = counts.cumsum(0)
    return torch.cat([torch.zeros(1, dtype=torch.int64), ends]), int(counts.max())


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    t = F[case["type"]]
    kind = case["kind"]
    if kind in ("epilogue", "epilogue_grad"):
        m, n, k = case["m"], case["n"], case["k"]
        s["A"] = _matrix(k, m, t, gen) if case["ta"] else _matrix(m, k, t, gen)
        s["B"] = _matrix(n, k, t, gen, k ** -0.5) if case["tb"] else _matrix(k, n, t, gen, k ** -0.5)
        s["alpha"] = 1.0
        if kind == "epilogue":
            s["bias_v"] = torch.randn(n, device="cuda", generator=gen).mul(0.5).to(t) if case["bias"] else None
            s["C"] = _matrix(m, n, F[case["out"]], gen) if case["beta"] else None
        else:
            s["Z"] = _matrix(m, n, t, gen)
    elif kind in ("grouped", "grouped_bwd"):
        rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
        offsets, s["most"] = _experts(case, seed)
        s["offsets"] = offsets.to(torch.int32).cuda()
        s["A"] = _matrix(rows, k, t, gen)
        shape = (n, k) if case["tb"] else (k, n)
        s["B"] = _matrix(groups * shape[0], shape[1], t, gen, k ** -0.5).unflatten(0, (groups, shape[0]))
        if kind == "grouped":
            s["bias_v"] = torch.randn(groups, n, device="cuda", generator=gen).mul(0.5).to(t) if case["bias"] else None
        else:
            s["Z"] = _matrix(rows, n, t, gen)
            s["X"] = _matrix(rows, n, t, gen)   # the product's other operand for the weights' gradient
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["X"] = _matrix(m, k, t, gen)
        s["W"] = _matrix(n, k, t, gen, 2.0 * k ** -0.5)
        target = torch.randint(0, n, (m,), device="cuda", generator=gen)
        out = torch.rand(m, device="cuda", generator=gen) < case["ignored"]
        s["target"] = torch.where(out, torch.full_like(target, -100), target)
        # the gradient that comes in: that of a mean over the rows that count, with the usual
        # loss scale where fp16 needs one
        g = (65536.0 if case["type"] == "f16" else 1.0) / max(1, m * (1 - case["ignored"]))
        s["g"] = torch.full((m,), g, device="cuda")
    return s


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


def _op(x, t):
    x = x.float()
    return x.t() if t else x


def _rows_of(s):
    """Expert and place within it of every row."""
    row = torch.arange(s["rows"], device="cuda")
    e = torch.bucketize(row, s["offsets"][1:].long(), right=True)
    return e, row - s["offsets"].long()[e]


def _spread(s, e, place, x):
    """Rows gathered by expert, short ones filled with zeros: groups x most x columns, in 32 bits."""
    y = torch.zeros(s["groups"], s["most"], x.shape[1], device="cuda")
    y[e, place] = x.float()
    return y


def _plain(s):
    kind = s["kind"]
    if kind == "epilogue":
        z = s["alpha"] * (_op(s["A"], s["ta"]) @ _op(s["B"], s["tb"]))
        if s["bias"]:
            z = z + s["bias_v"].float()
        d = _act(s["act"], z)
        if s["beta"]:
            d = d + s["beta"] * s["C"].float()
        r = {"D": d.to(F[s["out"]])}
        if s["aux"]:
            r["Z"] = z.to(F[s["type"]])
        return r
    if kind == "epilogue_grad":
        d = s["alpha"] * (_op(s["A"], s["ta"]) @ _op(s["B"], s["tb"])) * _act_slope(s["act"], s["Z"].float())
        return {"dZ": d.to(F[s["out"]]), "dbias": d.sum(0)}
    if kind in ("grouped", "grouped_bwd"):
        e, place = _rows_of(s)
        b = s["B"].float()
        z = torch.bmm(_spread(s, e, place, s["A"]), (b.transpose(1, 2) if s["tb"] else b).contiguous())[e, place]
        if kind == "grouped":
            if s["bias"]:
                z = z + s["bias_v"].float()[e]
            r = {"D": _act(s["act"], z).to(F[s["out"]])}
            if s["aux"]:
                r["Z"] = z.to(F[s["type"]])
            return r
        d = z * _act_slope(s["act"], s["Z"].float())
        db = torch.zeros(s["groups"], s["n"], device="cuda").index_add_(0, e, d)
        dv = torch.bmm(_spread(s, e, place, s["A"]).transpose(1, 2).contiguous(), _spread(s, e, place, s["X"]))
        return {"dZ": d.to(F[s["out"]]), "dbias": db, "dV": dv.to(F[s["out"]])}
    x, w = s["X"].float(), s["W"].float()
    counts = (s["target"] >= 0)
    at = torch.where(counts, s["target"], torch.zeros_like(s["target"]))[:, None]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(1, keepdim=True)
    lse = top + torch.log(total)
    r = {"loss": torch.where(counts, (lse - logits.gather(1, at))[:, 0], torch.zeros_like(lse[:, 0])), "lse": lse[:, 0]}
    if kind == "loss_train":
        p = p / total
        p.scatter_add_(1, at, torch.full_like(lse, -1.0))
        p = p * (s["g"] * counts)[:, None]
        r["dX"] = (p @ w).to(F[s["type"]])
        r["dW"] = (p.t() @ x).to(F[s["type"]])
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
    return torch.empty(rows, -(-cols // 8) * 8, device="cuda", dtype=dtype)[:, :cols]


def _own(s):
    mp, h = _library()
    kind, t = s["kind"], s["type"]
    if kind == "epilogue":
        m, n, k = s["m"], s["n"], s["k"]
        d = _new(m, n, F[s["out"]])
        z = _new(m, n, F[t]) if s["aux"] else None
        epi = mp.Epilogue(act=s["act"], bias=s["bias_v"], bias_type=t, aux=z, ld_aux=z.stride(0) if s["aux"] else 0)
        c = s["C"]
        mp.mpgemm_run_epilogue(h, s["ta"], s["tb"], m, n, k, s["alpha"], s["A"], t, s["A"].stride(0), s["B"], t,
                               s["B"].stride(0), epi, s["beta"], c, s["out"], d.stride(0), d, s["out"], d.stride(0))
        return {"D": d, "Z": z} if s["aux"] else {"D": d}
    if kind == "epilogue_grad":
        m, n, k = s["m"], s["n"], s["k"]
        d = _new(m, n, F[s["out"]])
        db = torch.empty(n, device="cuda")
        size = mp.mpgemm_epilogue_grad_workspace_size(1, m, n)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        mp.mpgemm_run_epilogue_grad(h, s["ta"], s["tb"], m, n, k, s["alpha"], s["A"], t, s["A"].stride(0), s["B"], t,
                                    s["B"].stride(0), s["act"], s["Z"], s["Z"].stride(0), d, s["out"], d.stride(0), db,
                                    ws, size)
        return {"dZ": d, "dbias": db}
    if kind == "grouped":
        rows, groups, n, k = s["rows"], s["groups"], s["n"], s["k"]
        d = _new(rows, n, F[s["out"]])
        z = _new(rows, n, F[t]) if s["aux"] else None
        epi = mp.Epilogue(act=s["act"], bias=s["bias_v"], bias_type=t, aux=z, ld_aux=z.stride(0) if s["aux"] else 0,
                          bias_stride=n)
        mp.mpgemm_run_grouped(h, s["tb"], groups, rows, n, k, 1.0, s["A"], t, s["A"].stride(0), s["offsets"], s["B"], t,
                              s["B"].stride(1), s["B"].stride(0), epi, d, s["out"], d.stride(0))
        return {"D": d, "Z": z} if s["aux"] else {"D": d}
    if kind == "grouped_bwd":
        rows, groups, n, k = s["rows"], s["groups"], s["n"], s["k"]
        d = _new(rows, n, F[s["out"]])
        db = torch.empty(groups, n, device="cuda")
        size = mp.mpgemm_epilogue_grad_workspace_size(groups, rows, n)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        mp.mpgemm_run_grouped_grad(h, s["tb"], groups, rows, n, k, 1.0, s["A"], t, s["A"].stride(0), s["offsets"],
                                   s["B"], t, s["B"].stride(1), s["B"].stride(0), s["act"], s["Z"], s["Z"].stride(0), d,
                                   s["out"], d.stride(0), db, ws, size)
        dv = _new(groups * k, n, F[s["out"]])
        mp.mpgemm_run_grouped_wgrad(h, groups, rows, k, n, 1.0, s["A"], t, s["A"].stride(0), s["X"], t,
                                    s["X"].stride(0), s["offsets"], 0.0, dv, s["out"], dv.stride(0), k * dv.stride(0))
        return {"dZ": d, "dbias": db, "dV": dv.unflatten(0, (groups, k))}
    m, n, k = s["m"], s["n"], s["k"]
    x, w = s["X"], s["W"]
    loss, lse = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    train = kind == "loss_train"
    size = mp.mpgemm_linear_ce_workspace_size(m, n, k, t, train)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    mp.mpgemm_run_linear_ce(h, m, n, k, 1.0, x, t, x.stride(0), w, w.stride(0), s["target"], loss, lse, ws, size)
    if not train:
        return {"loss": loss, "lse": lse}
    dx, dw = _new(m, k, F[t]), _new(n, k, F[t])
    mp.mpgemm_run_linear_ce_grad(h, m, n, k, 1.0, x, t, x.stride(0), w, w.stride(0), s["target"], lse, s["g"], dx,
                                 dx.stride(0), dw, dw.stride(0), ws, size)
    return {"loss": loss, "lse": lse, "dX": dx, "dW": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- what cannot be done without
def work(case):
    tb = 2
    ob = {"bf16": 2, "f16": 2, "f32": 4}[case.get("out", case["type"])]
    kind = case["kind"]
    if kind in ("epilogue", "epilogue_grad"):
        m, n, k = case["m"], case["n"], case["k"]
        b = tb * (m * k + k * n) + ob * m * n
        if kind == "epilogue":
            b += tb * n * case["bias"] + tb * m * n * case["aux"] + ob * m * n * bool(case["beta"])
        else:
            b += tb * m * n + 4 * n
        return {"bytes": b, "flops": 2 * m * n * k}
    if kind in ("grouped", "grouped_bwd"):
        rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
        used = groups * (1 - math.exp(-rows / groups))   # experts that have rows, where the shares are even
        b = tb * (rows * k + used * k * n) + ob * rows * n + 4 * groups
        if kind == "grouped":
            return {"bytes": int(b + tb * used * n * case["bias"] + tb * rows * n * case["aux"]), "flops": 2 * rows * n * k}
        return {"bytes": int(b + tb * 2 * rows * n + 4 * groups * n + ob * groups * k * n), "flops": 4 * rows * n * k}
    m, n, k = case["m"], case["n"], case["k"]
    if kind == "loss":
        return {"bytes": tb * (m * k + n * k) + 16 * m, "flops": 2 * m * n * k}
    return {"bytes": 2 * tb * (m * k + n * k) + 20 * m, "flops": 6 * m * n * k}


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
    kind = case["kind"]
    if kind in ("epilogue", "epilogue_grad"):
        a = s["A"].double().T if case["ta"] else s["A"].double()
        b = s["B"].double().T if case["tb"] else s["B"].double()
        z = a.mm(b)
        if kind == "epilogue_grad":
            d = z * _act64(case["act"], s["Z"].double())[1]
            return {"dZ": d, "dbias": d.sum(0)}
        if case["bias"]:
            z += s["bias_v"].double()
        d = _act64(case["act"], z)[0]
        if case["beta"]:
            d = d + case["beta"] * s["C"].double()
        return {"D": d, "Z": z} if case["aux"] else {"D": d}
    if kind in ("grouped", "grouped_bwd"):
        ends = s["offsets"].tolist()
        n, k, groups = case["n"], case["k"], case["groups"]
        d = torch.zeros(case["rows"], n, dtype=torch.float64, device="cuda")
        z = torch.zeros_like(d)
        db = torch.zeros(groups, n, dtype=torch.float64, device="cuda")
        dv = torch.zeros(groups, k, n, dtype=torch.float64, device="cuda") if kind == "grouped_bwd" else None
        for e in range(groups):
            r = slice(ends[e], ends[e + 1])
            if ends[e] == ends[e + 1]:
                continue
            a, b = s["A"][r].double(), s["B"][e].double()
            z[r] = a.mm(b.T if case["tb"] else b)
            if kind == "grouped":
                if case["bias"]:
                    z[r] += s["bias_v"][e].double()
                d[r] = _act64(case["act"], z[r])[0]
            else:
                d[r] = z[r] * _act64(case["act"], s["Z"][r].double())[1]
                db[e] = d[r].sum(0)
                dv[e] = a.T.mm(s["X"][r].double())
        if kind == "grouped":
            return {"D": d, "Z": z} if case["aux"] else {"D": d}
        return {"dZ": d, "dbias": db, "dV": dv}
    x, w, t = s["X"].double(), s["W"].double(), s["target"]
    logits = x.mm(w.T)
    lse = torch.logsumexp(logits, 1)
    row = torch.arange(case["m"], device="cuda")[t >= 0]
    loss = torch.zeros_like(lse)
    loss[row] = lse[row] - logits[row, t[row]]
    if kind == "loss":
        return {"loss": loss, "lse": lse}
    logits.sub_(lse[:, None]).exp_()
    logits[row, t[row]] -= 1
    weight = torch.zeros_like(lse)
    weight[row] = s["g"][row].double()
    logits.mul_(weight[:, None])
    return {"loss": loss, "lse": lse, "dX": logits.mm(w), "dW": logits.T.mm(x)}
