"""Plain forms, in 64 bits and from the formulas, of the operators beside the
GEMV: the oracle of tests/test_operators.py. Nothing here uses the library."""
import numpy as np
import torch

F64 = torch.float64


def quantize_i8(x):
    """q [n, inp] as float64 whole numbers and scale a / 127 of x [n, inp]."""
    x = x.to(F64)
    a = x.abs().amax(1, keepdim=True)
    q = torch.round(127 * x / a)
    q = torch.where(torch.isfinite(a) & (a > 0), q, 0.0)
    scale = torch.where(torch.isfinite(a), a / 127, torch.nan)
    return q, scale[:, 0]


def rounded4(x, group):
    """Codes, scale and lowest value of x [..., dim]: float64 [..., ng, group] / [..., ng]."""
    g = x.to(F64).unflatten(-1, (x.shape[-1] // group, group))
    fine = torch.isfinite(g).all(-1)
    lo, hi = g.amin(-1), g.amax(-1)
    s = torch.where(fine, (hi - lo) / 15, 0.0).to(x.dtype).to(F64)
    u = torch.round((g - lo[..., None]) / s[..., None]).clamp(0, 15)
    u = torch.where(fine[..., None] & (s[..., None] > 0), u, 0.0)
    return u, torch.where(fine, s, torch.nan), torch.where(fine, lo, torch.nan)


def values4(x, group):
    """The values that x stands for once it is in the cache."""
    u, s, lo = rounded4(x, group)
    return (lo[..., None] + s[..., None] * u).flatten(-2)


def code_bytes(u, which):
    """Packed row bytes [rows, dim / 2] of codes u [rows, dim] (float64 or int):
    channel by channel, from the documented places."""
    u = u.to(torch.int64).cpu().numpy()
    rows, dim = u.shape
    out = np.zeros((rows, dim // 2), np.uint8)
    for c in range(dim):
        j, r = divmod(c, 32)
        if which == 0:
            t, i = divmod(r, 8)
            at = t * dim // 8 + 4 * j + i // 2
        else:
            g, i = divmod(r, 4)
            at = g * dim // 16 + 2 * j + i // 2
        out[:, at] |= (u[:, c] << (4 * (i & 1))).astype(np.uint8)
    return out


def attention(q, k, v, lens, n_new, scale):
    """q [batch, n_new, q_heads, dim]; k, v [batch, tokens, heads, dim] (values,
    float64). Returns out like q, mass [batch, heads, tokens], and bounds on
    what fp32 arithmetic may change: in out, per row, and in mass.

    The bound: a score is a sum of dim products, each with a few roundings of
    2^-24; with the sums' own roundings its error is below 2^-20 sum |q| |k|.
    exp multiplies it into a relative error of p (and 2^-21 for exp2 itself);
    numerator and denominator double it, and the sums over the tokens add 2^-20.
    A mass is a sum of such p's: each adds its own error and a rounding of the
    sum, which stays below the row count."""
    b, n, qh, dim = q.shape
    heads = k.shape[2]
    per = qh // heads
    out = torch.zeros(q.shape, dtype=F64)
    mass = torch.zeros(b, heads, k.shape[1], dtype=F64)
    bound = torch.zeros(b, n, qh, dtype=F64)
    mass_bound = torch.zeros_like(mass)
    q = q.to(F64)
    for i in range(b):
        for j in range(n):
            m = int(lens[i]) - (n - 1 - j)
            if m <= 0:
                continue
            for h in range(qh):
                kk, vv = k[i, :m, h // per], v[i, :m, h // per]
                s = scale * (kk @ q[i, j, h])
                p = torch.softmax(s, 0)
                out[i, j, h] = p @ vv
                mass[i, h // per, :m] += p
                err = 2.0 ** -20 * float((kk.abs() @ q[i, j, h].abs()).max()) * abs(scale) + 2.0 ** -20
                bound[i, j, h] = 2 * err * float(vv.abs().max())
                mass_bound[i, h // per, :m] += (2 * err + n * per * 2.0 ** -24) * p
    return out, mass, bound, mass_bound


def keep(mass, length, budget, recent):
    """Kept positions of one head: a plain loop."""
    if length <= budget:
        return list(range(length))
    old = length - recent
    order = sorted(range(old), key=lambda i: (-np.inf if np.isnan(mass[i]) else -float(mass[i]), not np.isnan(mass[i]), i))
    return sorted(order[:budget - recent]) + list(range(old, length))
