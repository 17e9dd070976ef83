"""Gated products in 64 bits with bounds of what 32-bit sums and one rounding to the output's type may
add (as in tests/ops_reference.py), and the pairs of matrices the GPU tests run them on."""
import math

import torch

from tests import ops_reference as ref


def pair(gen, rows, cols, t, layout, scale=1.0):
    """(whole buffer, first, second, elements between them): two rows x cols matrices of random values, side by
    side in each row or one after the other; everything that is not theirs is NaN."""
    c8 = -(-max(cols, 1) // 8) * 8
    if layout == "beside":
        buf = torch.full((rows + 2, 2 * c8 + 24), float("nan"), dtype=ref.TYPES[t], device="cuda")
        a, b, stride = buf[:rows, :cols], buf[:rows, c8 + 8:c8 + 8 + cols], c8 + 8
    else:
        buf = torch.full((2 * rows + 5, c8 + 8), float("nan"), dtype=ref.TYPES[t], device="cuda")
        a, b, stride = buf[:rows, :cols], buf[rows + 3:2 * rows + 3, :cols], (rows + 3) * (c8 + 8)
    for x in (a, b):
        x.copy_((torch.randn(rows, cols, generator=gen) * scale).to(ref.TYPES[t]))
    return buf, a, b, stride


def pair_out(rows, cols, t, layout):
    """The same for outputs, filled with the sentinel."""
    c8 = -(-max(cols, 1) // 8) * 8
    if layout == "beside":
        buf = torch.full((rows + 2, 2 * c8 + 24), ref.SENTINEL, dtype=ref.TYPES[t], device="cuda")
        return buf, buf[:rows, :cols], buf[:rows, c8 + 8:c8 + 8 + cols], c8 + 8
    buf = torch.full((2 * rows + 5, c8 + 8), ref.SENTINEL, dtype=ref.TYPES[t], device="cuda")
    return buf, buf[:rows, :cols], buf[rows + 3:2 * rows + 3, :cols], (rows + 3) * (c8 + 8)


def pair_untouched(buf, *views):
    """Nothing but the views of the buffer has been written."""
    rest = torch.ones_like(buf, dtype=torch.bool)
    for v in views:
        torch.as_strided(rest, v.shape, v.stride(), v.storage_offset() - buf.storage_offset()).fill_(False)
    return bool((buf[rest] == ref.SENTINEL).all())


def act64(name, z):
    """ref.act64 with GELU's tail by erfc: torch's ndtr has 1e-16 of absolute error there (at -7.7 6.83e-15 for
    6.80e-15), which is more than the bounds below allow of values that the other factor brings back."""
    if name != "gelu":
        return ref.act64(name, z)
    c = z.clamp(-40, 40)
    phi = 0.5 * torch.erfc(-c / math.sqrt(2))
    return z * phi, phi + c * torch.exp(-c * c / 2) / math.sqrt(2 * math.pi)


def _act(act, g, g_err):
    """(act(g), error) -- slopes are at most 1.13; the value's own 2^-17 where it is not exact."""
    a = act64(act, g)[0]
    return a, 1.13 * g_err + (2.0 ** -17 * a.abs() + 1e-30 if act not in ("none", "relu") else 0.0)


def forward64(a, bg, bu, k, act, bias_g=None, bias_u=None, alpha=1.0):
    """((D, error), (G, error), (U, error)), errors before the rounding to the output's type."""
    out = []
    for b, bias in ((bg, bias_g), (bu, bias_u)):
        z, err = ref.product64(a, b, k, alpha)
        if bias is not None:
            z = z + bias.double().cpu()
            err = err + 2.0 ** -23 * z.abs()
        out.append((z, err))
    (g, g_err), (u, u_err) = out
    v, v_err = _act(act, g, g_err)
    d = v * u
    return (d, v_err * u.abs() + v.abs() * u_err + v_err * u_err + 2.0 ** -23 * d.abs()), out[0], out[1]


def grad64(e, e_err, g, u, act):
    """((dG, error), (dU, error), (H, error)) from E and the kept factors."""
    g, u = g.double().cpu(), u.double().cpu()
    value, slope = act64(act, g)
    if act in ("silu", "gelu_tanh", "gelu"):
        value = torch.where(g == -math.inf, torch.zeros_like(value), value)   # the limit
    exact = act in ("none", "relu")
    # two roundings of products beside the slope's own error, which is one of numbers of order one
    dg = e * u * slope
    dg_err = (1.13 * e_err + (0.0 if exact else 2.0 ** -19) * e.abs()) * u.abs() + 2.0 ** -22 * dg.abs()
    v_err = torch.zeros_like(value) if exact else 2.0 ** -17 * value.abs() + 1e-30
    du = e * value
    h = value * u
    return ((dg, dg_err), (du, e_err * value.abs() + v_err * (e.abs() + e_err) + 2.0 ** -23 * du.abs()),
            (h, v_err * u.abs() + 2.0 ** -23 * h.abs()))


def check(got, want, err, t, what):
    ref.assert_within(got, want, err + ref.rounding(want.abs() + err, t), what)
