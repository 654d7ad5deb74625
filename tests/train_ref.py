"""Plain binary64 references of the training operators (numpy and torch on the
CPU; none of the library's code), and the bounds of their errors.

Bounds count roundings: one rounding to a type t is off by at most
finfo(t).eps / 2 relative to the value. A binary32 sum of terms t_i formed as
running sums of L terms joined by a tree of depth D is off by at most about
(L + D) 2^-24 sum |t_i|; the matrix instructions are granted 2^-23 a step,
in case they truncate.
"""
from __future__ import annotations

import numpy as np
import torch

GROUP = 32
FP8_MAX = {0: 448.0, 1: 57344.0}
U = 2.0 ** -24


def half(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def floor_of(dtype) -> float:
    """Half of the smallest step of a type (its subnormals' spacing)."""
    return float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps / 2


# ------------------------------------------------------------- checkpoints ---

def decode_table(fmt: int) -> np.ndarray:
    """The 256 values of a format, from its definition (NaN for NaN codes)."""
    mbits, bias = (3, 7) if fmt == 0 else (2, 15)
    out = np.empty(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 0x80 else 1.0), (c & 0x7F) >> mbits, c & ((1 << mbits) - 1)
        if fmt == 0 and (c & 0x7F) == 0x7F:
            v = np.nan
        elif fmt == 1 and e == 31:
            v = np.inf if m == 0 else np.nan
        elif e == 0:
            v = m * 2.0 ** (1 - bias - mbits)
        else:
            v = (1 + m / (1 << mbits)) * 2.0 ** (e - bias)
        out[c] = sign * v
    return out


def encode(x: np.ndarray, fmt: int) -> np.ndarray:
    """Nearest code of each binary64 value by search over the table: ties to
    the even code, beyond the range to the largest, NaN to 0x7F | sign."""
    top = 0x7E if fmt == 0 else 0x7B
    mag = decode_table(fmt)[:top + 1]
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), mag[-1])
    hi = np.clip(np.searchsorted(mag, a, side="left"), 0, top)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - mag[lo], mag[hi] - a
    code = np.where(dhi < dlo, hi, np.where(dlo < dhi, lo, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def checkpoint_save(x: np.ndarray, fmt: int):
    """(codes, scale bytes) of a binary32-representable matrix, group by group."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, groups), np.uint8)
    for g in range(groups):
        part = x[:, g * GROUP:(g + 1) * GROUP].astype(np.float64)
        amax = np.abs(part).max(axis=1)
        e = np.zeros(rows)
        fine = np.isfinite(amax) & (amax > 0)
        for r in np.nonzero(fine)[0]:
            k = -126
            while amax[r] > FP8_MAX[fmt] * 2.0 ** k:
                k += 1
            e[r] = k
        codes[:, g * GROUP:(g + 1) * GROUP] = encode(part * (2.0 ** -e)[:, None], fmt)
        scales[:, g] = (e + 127).astype(np.uint8)
    return codes, scales


def checkpoint_values(codes: np.ndarray, scales: np.ndarray, fmt: int) -> np.ndarray:
    s = np.repeat(2.0 ** (scales.astype(np.float64) - 127), GROUP, axis=1)[:, :codes.shape[1]]
    return decode_table(fmt)[codes] * s


# ------------------------------------------------------------------- norms ---

def norm_forward(x, w, b, eps, centered):
    """(y, mean, rstd, bound of y before its rounding), all binary64."""
    x = x.double()
    mu = x.mean(1, keepdim=True) if centered else torch.zeros_like(x[:, :1])
    xc = x - mu
    rstd = 1 / torch.sqrt(xc.square().mean(1, keepdim=True) + eps)
    y = xc * rstd * w
    # mu: sums of at most 32 terms a lane, joined over 6 + 16 levels; the variance likewise,
    # and the roundings of x - mu, rstd and the products: 128 steps cover their sum
    near = w.abs() * rstd * (xc.abs() + (x.abs().mean(1, keepdim=True) if centered else 0))
    if b is not None:
        y = y + b
        near = near + b.abs()
    return y, mu[:, 0], rstd[:, 0], 128 * U * near


def norm_backward(dy, x, w, mu, rstd, centered):
    """(dx, dweight, dbias, bound of dx before its rounding, of dweight, of dbias)."""
    dy, x, rstd = dy.double(), x.double(), rstd.double()[:, None]
    xh = (x - mu.double()[:, None] if centered else x) * rstd
    g = dy * w
    c1 = g.mean(1, keepdim=True) if centered else torch.zeros_like(g[:, :1])
    c2 = (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2)
    near = rstd * (g.abs() + (g.abs().mean(1, keepdim=True) if centered else 0)
                   + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    # column sums: at most rows / 512 + 1 terms a lane, four waves, 16 partial sums a thread, 32 threads
    steps = (dy.shape[0] / 512 + 64) * U + 4 * U
    return (dx, (dy * xh).sum(0), dy.sum(0), 128 * U * near, steps * (dy * xh).abs().sum(0),
            steps * dy.abs().sum(0))


# ------------------------------------------------------ gated feed-forward ---

def act_parts(g, name):
    """act(g), act'(g) and a bound of |act''| in binary64."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), 0.5
    if name == "gelu":
        phi = 0.5 * torch.erfc(-g / 2 ** 0.5)
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / (2 * np.pi) ** 0.5, 0.8
    c = (2 / np.pi) ** 0.5
    z = c * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(2 * z)
    return g * s, s + 2 * g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g), 1.0


def ffn(x, wg, wu, act, dh=None, dtype=torch.float16):
    """Products and gradients in binary64 with the bounds of their errors before the last rounding, as dicts."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    K = x.shape[1]
    g, u = x.mm(wg.t()), x.mm(wu.t())
    eg, eu = 2 * U * (K + 8) * x.abs().mm(wg.abs().t()), 2 * U * (K + 8) * x.abs().mm(wu.abs().t())
    a, d, curve = act_parts(g, act)
    # elementary functions: a handful of units in the last place of a and d (which are O(1 + |g|) in their terms)
    ea = d.abs() * eg + 0.5 * curve * eg * eg + 16 * U * (a.abs() + g.abs() * 0.1)
    ed = curve * eg + 32 * U * (1 + g.abs())
    val, err = {"h": a * u}, {"h": ea * u.abs() + (a.abs() + ea) * eu + 4 * U * (a * u).abs()}
    if dh is None:
        return val, err
    dh = dh.double()
    r = half(dtype)
    tiny = floor_of(dtype)
    du, dg = dh * a, dh * u * d
    # rounded to dtype, as operands of the matrix instructions
    edu = dh.abs() * ea + 4 * U * du.abs()
    edu = edu + r * (du.abs() + edu) + tiny
    edg = dh.abs() * (u.abs() * ed + (d.abs() + ed) * eu) + 8 * U * dg.abs()
    edg = edg + r * (dg.abs() + edg) + tiny
    F, T = wg.shape[0], x.shape[0]
    val["dx"] = dg.mm(wg) + du.mm(wu)
    mag = (dg.abs() + edg).mm(wg.abs()) + (du.abs() + edu).mm(wu.abs())
    err["dx"] = edg.mm(wg.abs()) + edu.mm(wu.abs()) + 2 * U * (2 * F + 16) * mag
    for name, v, e in (("dw_gate", dg, edg), ("dw_up", du, edu)):
        val[name] = v.t().mm(x)
        err[name] = e.t().mm(x.abs()) + 2 * U * (T + 16) * (v.abs() + e).t().mm(x.abs())
    return val, err


def assert_near(got: torch.Tensor, ref: torch.Tensor, bound: torch.Tensor, what: str) -> None:
    """|got - ref| <= bound + one rounding to got's type."""
    dt = got.dtype
    d = (got.detach().cpu().double() - ref).abs()
    tol = bound + half(dt) * (ref.abs() + bound) + floor_of(dt)
    assert torch.isfinite(d).all(), what + ": not finite"
    worst = (d / tol.clamp_min(1e-300)).max().item() if d.numel() else 0.0
    assert worst <= 1.0, "%s: off by %.3g of the bound" % (what, worst)
