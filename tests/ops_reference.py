"""The products of language models in 64 bits, with bounds of what 32-bit sums and one rounding to
the output's type may add, and the buffers the GPU tests run them on.

Bounds.  Products of 16-bit values are exact in FP32; a sum of k of them by blocks of eight is
off by at most (2^-21 + (k / 8 + 4) 2^-24) S, S the sum of the products' magnitudes: 24 fraction
bits below a block's largest product, cut, and one rounding per block.  An activation's slope is
at most 1.13; exp2 and the reciprocal are off by one unit (2^-23), arguments of exponentials by
2^-24 of up to about 100, polynomials by 5e-7: 2^-17 of the value covers them, 2^-19 the slopes
(which are of order one).  A rounding to the output's type adds eps / 2 of the value (or half the
smallest subnormal)."""
import math

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SENTINEL = 77.0


def padded(rows, cols, dtype, fill, extra=0, device="cuda"):
    """A rows x cols view into rows of whole 16-byte blocks (and `extra` elements more), the rest
    of the buffer filled with `fill`; two rows of it follow the last one."""
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    ld = -(-max(cols, 1) // unit) * unit + extra
    buf = torch.full((rows + 2, ld), fill, dtype=dtype, device=device)
    return buf, buf[:rows, :cols]


def matrix(gen, rows, cols, t, scale=1.0, extra=8):
    """Random normal values; what lies past the rows' ends is NaN."""
    _, view = padded(rows, cols, TYPES[t], float("nan"), extra)
    view.copy_((torch.randn(rows, cols, generator=gen) * scale).to(TYPES[t]))
    return view


def output(rows, cols, t, extra=8):
    return padded(rows, cols, TYPES[t], SENTINEL, extra)


def untouched(buf, rows, cols):
    """Nothing but the rows x cols view of the buffer has been written."""
    rest = buf.clone()
    rest[:rows, :cols] = SENTINEL
    return bool((rest == SENTINEL).all())


# ----------------------------------------------------------------------------- activations
def act64(name, z):
    """(value, slope) in 64 bits; slopes of infinite z are their limits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z), (z > 0).double()
    c = z.clamp(-40, 40)
    if name == "silu":
        g = torch.sigmoid(c)
        return z * torch.sigmoid(z), g + c * g * torch.sigmoid(-c)
    if name == "gelu":
        return (z * torch.special.ndtr(z),
                torch.special.ndtr(c) + c * torch.exp(-c * c / 2) / math.sqrt(2 * math.pi))
    k = math.sqrt(8 / math.pi)
    g = torch.sigmoid(k * (c + 0.044715 * c ** 3))
    return (z * torch.sigmoid(k * (z + 0.044715 * z ** 3)),
            g + c * g * (1 - g) * k * (1 + 0.134145 * c * c))


# ----------------------------------------------------------------------------- bounds
def sum_error(k, magnitude):
    return (2.0 ** -21 + (k / 8 + 4) * 2.0 ** -24) * magnitude


def rounding(value, t):
    f = torch.finfo(TYPES[t])
    return value.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def product64(a, b, k, alpha=1.0):
    """(a b alpha, bound of its FP32 form's error)."""
    a, b = a.double().cpu(), b.double().cpu()
    z = alpha * (a @ b)
    return z, sum_error(k, abs(alpha) * (a.abs() @ b.abs())) + 2.0 ** -23 * z.abs()


def forward64(z, z_err, act, bias=None, beta=0.0, c=None):
    """(D, error before its rounding, Z, its error)."""
    if bias is not None:
        z = z + bias.double().cpu()
        z_err = z_err + 2.0 ** -23 * z.abs()
    d = act64(act, z)[0]
    err = 1.13 * z_err + (2.0 ** -17 * d.abs() + 1e-30 if act not in ("none", "relu") else 0.0)
    if beta:
        d = d + beta * c.double().cpu()
        err = err + 2.0 ** -23 * (d.abs() + abs(beta) * c.double().cpu().abs())
    return d, err, z, z_err


def slope64(z, z_err, act, kept):
    """(D, error before its rounding) of the gradient through an activation."""
    if act == "none":
        return z, z_err
    s = act64(act, kept.double().cpu())[1]
    exact = act == "relu"
    return z * s, 1.13 * z_err + (0.0 if exact else 2.0 ** -19) * z.abs()


def column_sums64(d, err):
    return d.sum(0), err.sum(0) + d.shape[0] * 2.0 ** -24 * d.abs().sum(0)


def assert_within(got, want, bound, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    if bool(bad.any()):
        at = tuple(int(v[0]) for v in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {at}: "
                             f"{float(got[at])} for {float(want[at])}, bound {float(bound[at])}")


# ----------------------------------------------------------------------------- cross entropy
def cross_entropy64(x, w, target, alpha, k):
    """(loss, lse, bound of both, logits, bound of the logits)."""
    z, z_err = product64(x, w.t(), k, alpha)
    n = z.shape[1]
    lse = torch.logsumexp(z, 1)
    t = target.cpu()
    counts = (t >= 0) & (t < n)
    at = torch.where(counts, t, torch.zeros_like(t))[:, None]
    loss = torch.where(counts, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    # the exponentials and their sums are off by 2^-18 together: relative in the sum, so absolute here
    err = z_err.max(1).values + 2.0 ** -18 + 2.0 ** -21 * lse.abs()
    loss_err = err + z_err.gather(1, at)[:, 0] + 2.0 ** -21 * z.gather(1, at)[:, 0].abs()
    return loss, lse, torch.where(counts, loss_err, torch.zeros_like(err)), err, z, z_err


def cross_entropy_grad64(x, w, target, grad, alpha, k, t):
    """(dX, bound, dW, bound), the logits' gradient rounded to the type for the products."""
    _, lse, _, lse_err, z, z_err = cross_entropy64(x, w, target, alpha, k)
    m, n = z.shape
    tt = target.cpu()
    counts = ((tt >= 0) & (tt < n))
    p = torch.exp(z - lse[:, None])
    p_err = p * (z_err + lse_err[:, None] + 2.0 ** -18)
    rows = torch.arange(m)[counts]
    p[rows, tt[counts]] -= 1
    weight = torch.where(counts, grad.double().cpu(), torch.zeros(m, dtype=torch.float64))
    p, p_err = p * weight[:, None], p_err * weight.abs()[:, None]
    # the rounding; FP16's weights are brought to 2^13 first, so that its smallest step (2^-24, half
    # of it off) stands for max |weight| 2^-37
    step = 2.0 ** -38 * float(weight.abs().max()) if t == "f16" and m else 0.0
    p_err = p_err + torch.finfo(TYPES[t]).eps / 2 * (p.abs() + p_err) + step + 2.0 ** -23 * p.abs()
    xd, wd = x.double().cpu(), w.double().cpu()
    dx, dw = alpha * (p @ wd), alpha * (p.t() @ xd)
    dx_err = abs(alpha) * (p_err @ wd.abs()) + sum_error(n + 256, abs(alpha) * (p.abs() @ wd.abs())) + 2.0 ** -22 * dx.abs()
    dw_err = abs(alpha) * (p_err.t() @ xd.abs()) + sum_error(m, abs(alpha) * (p.abs().t() @ xd.abs())) + 2.0 ** -22 * dw.abs()
    return dx, dx_err + rounding(dx, t), dw, dw_err + rounding(dw, t)
