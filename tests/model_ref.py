"""Plain binary64 references of the operators at the ends of a model and between
its tokens (torch on the CPU; none of the library's code), and the bounds of
their errors before the last rounding, in the terms of train_ref: U = 2^-24 is
half a step of binary32; exponentials, reciprocals and logarithms are granted
one unit in the last place (2 U)."""
from __future__ import annotations

import math

import torch

from tests.train_ref import U, assert_near, floor_of, half  # noqa: F401

CHUNK = 32


# --------------------------------------------------------------- embedding ---

def embedding_forward(ids, weight, scale):
    """(y, bound): one product."""
    w = torch.cat([weight.double(), torch.zeros(1, weight.shape[1], dtype=torch.float64)])
    ids = ids.long()
    y = w[torch.where((ids >= 0) & (ids < weight.shape[0]), ids, weight.shape[0])] * scale
    return y, U * y.abs()


def embedding_backward(dy, ids, vocab, scale, base=None):
    """(dweight, bound): a sum of n rows in any order, a product, with base one more addition."""
    ids = ids.long()
    live = (ids >= 0) & (ids < vocab)
    dw = torch.zeros(vocab, dy.shape[1], dtype=torch.float64)
    mag, n = torch.zeros_like(dw), torch.zeros(vocab, 1, dtype=torch.float64)
    dw.index_add_(0, ids[live], dy[live].double())
    mag.index_add_(0, ids[live], dy[live].double().abs())
    n.index_add_(0, ids[live], torch.ones(int(live.sum()), 1, dtype=torch.float64))
    dw, bound = dw * scale, (n + 2) * U * mag * abs(scale)
    return (dw, bound) if base is None else (dw + base.double(), bound + U * (base.double().abs() + mag * abs(scale)))


# -------------------------------------------------------------- recurrence ---

def gates(gate):
    """a, 1 - a and bounds of their relative errors. e^-|g| is off by 2 U |g| (a constant and a product in the
    exponent) and one unit; the sum, the reciprocal and the product follow. The larger of the two holds e
    times that error, and e |g| < 1."""
    g = gate.double()
    # beyond 1,000 e^-|g| is 0 in binary64 and so is every bound it takes part in (0 times an infinite |g| is not)
    g = g.clamp(-1000, 1000)
    small, big = (2 * g.abs() + 8) * U, torch.full_like(g, 8 * U)
    return (torch.sigmoid(g), torch.sigmoid(-g), torch.where(g >= 0, big, small), torch.where(g >= 0, small, big))


def recurrence_forward(x, gate, h0=None, lengths=None):
    """h before and after each step [B, T + 1, C] (steps behind a length repeat the last), and its bound.

    Every step adds the errors of a and 1 - a and a few roundings (products, the sum, and where spans of steps are
    joined, of partial results no larger than the recurrence of the magnitudes): 8 U of that recurrence."""
    x = x.double()
    a, keep, ea, ek = gates(gate)
    B, T, C = x.shape
    h = torch.zeros(B, C, dtype=torch.float64) if h0 is None else h0.double()
    mag, err = h.abs(), torch.zeros_like(h)
    hs, errs = [h], [err]
    for t in range(T):
        m = a[:, t] * mag + keep[:, t] * x[:, t].abs()
        e = a[:, t] * err + a[:, t] * ea[:, t] * mag + keep[:, t] * ek[:, t] * x[:, t].abs() + 8 * U * m
        n = a[:, t] * h + keep[:, t] * x[:, t]
        live = torch.ones(B, 1, dtype=torch.bool) if lengths is None else (t < lengths.long())[:, None]
        h, mag, err = torch.where(live, n, h), torch.where(live, m, mag), torch.where(live, e, err)
        hs.append(h)
        errs.append(err)
    return torch.stack(hs, 1), torch.stack(errs, 1)


def recurrence_backward(dy, x, gate, states, dh_last=None, lengths=None):
    """{"dx", "dgate", "dh0"} and bounds: h from the saved states, then the gradients backward in time."""
    dy, x = dy.double(), x.double()
    a, keep, ea, ek = gates(gate)
    B, T, C = x.shape
    before, eb = torch.zeros_like(x), torch.zeros_like(x)
    for t0 in range(0, T, CHUNK):
        hs, errs = recurrence_forward(x[:, t0:t0 + CHUNK], gate[:, t0:t0 + CHUNK], states[:, t0 // CHUNK])
        before[:, t0:t0 + CHUNK], eb[:, t0:t0 + CHUNK] = hs[:, :-1], errs[:, :-1]
    carry = torch.zeros(B, C, dtype=torch.float64) if dh_last is None else dh_last.double()
    mag, err = carry.abs(), torch.zeros_like(carry)
    val = {"dx": torch.zeros_like(x), "dgate": torch.zeros_like(x)}
    bound = {"dx": torch.zeros_like(x), "dgate": torch.zeros_like(x)}
    for t in range(T - 1, -1, -1):
        live = torch.ones(B, 1, dtype=torch.bool) if lengths is None else (t < lengths.long())[:, None]
        lam, lmag = dy[:, t] + carry, dy[:, t].abs() + mag
        lerr = err + 8 * U * lmag
        at, kt, xt, ht = a[:, t], keep[:, t], x[:, t], before[:, t]
        val["dx"][:, t], bound["dx"][:, t] = kt * lam, kt * lerr + kt * (ek[:, t] + 4 * U) * lmag
        val["dgate"][:, t] = lam * (ht - xt) * at * kt
        bound["dgate"][:, t] = at * kt * (lerr * (ht - xt).abs() + lmag * (eb[:, t] + U * (ht.abs() + xt.abs()))
                                          + lmag * (ht - xt).abs() * (ea[:, t] + ek[:, t] + 8 * U))
        carry = torch.where(live, at * lam, carry)
        err = torch.where(live, at * lerr + at * (ea[:, t] + 4 * U) * lmag, err)
        mag = torch.where(live, at * lmag, mag)
    val["dh0"], bound["dh0"] = carry, err
    return val, bound


# ------------------------------------------------------------------ losses ---

def _softmax(z, tau):
    """largest, sum, q and the relative bound of the sum and of each exponential. (z - largest) / tau as an exponent
    of 2 is off by 4 U of itself; a sum of V terms is formed by at least 256 lanes of 8 terms at a time."""
    z = z.double()
    largest = z.amax(1, keepdim=True) if z.shape[1] else torch.full((z.shape[0], 1), -math.inf, dtype=torch.float64)
    d = torch.where(z == -math.inf, torch.full_like(z, -1e4 * tau), z - torch.where(largest == -math.inf, 0.0, largest))
    e = torch.where(z == -math.inf, 0.0, torch.exp(d / tau))
    s = e.sum(1, keepdim=True)
    each = (4 * d.abs() / tau + 4) * U
    total = (e * each).sum(1, keepdim=True) / s.clamp_min(1e-300) + (z.shape[1] / 256 + 64) * U
    return largest, s, e / s.clamp_min(1e-300), d / tau, each + total + 4 * U, total


def distill(logits, ids, teacher, tau, dloss=None):
    """{"loss", "stats", "dlogits"} and bounds; rows without entries or without a finite logit are left out."""
    rows, vocab = logits.shape
    largest, s, q, dz, eq, es = _softmax(logits, tau)
    ids, t = ids.long(), teacher.double()
    entry = (ids >= 0) & (ids < vocab) & (t > -math.inf)
    named = entry.any(1, keepdim=True)
    live = named & (largest > -math.inf)
    t = torch.where(entry, t, -math.inf)
    top = t.amax(1, keepdim=True)
    dt = torch.where(entry, (t - torch.where(named, top, 0.0)) / tau, 0.0)
    w = torch.where(entry, torch.exp(dt), 0.0)
    st = w.sum(1, keepdim=True).clamp_min(1e-300)
    p, k = w / st, t.shape[1]
    each = (4 * dt.abs() + 4) * U
    et = (p * each).sum(1, keepdim=True) + (k + 4) * U
    ep = p * (each + et)
    at = ids.clamp(0, max(vocab - 1, 0))
    log_p, log_q = dt - torch.log(st), dz.gather(1, at) - torch.log(s.clamp_min(1e-300))
    diff = torch.where(p > 0, log_p - log_q, 0.0)
    eln = (each * dt.abs().clamp_min(1) + et + 4 * U * torch.log(st).abs()
           + 4 * U * dz.gather(1, at).abs() + es + 4 * U * torch.log(s.clamp_min(1e-300)).abs() + 8 * U)
    loss = tau ** 2 * (p * diff).sum(1, keepdim=True)
    eloss = tau ** 2 * (ep * diff.abs() + p * eln + (k + 8) * U * p * diff.abs()).sum(1, keepdim=True)
    g = torch.ones(rows, 1, dtype=torch.float64) if dloss is None else dloss.double()[:, None]
    pc, epc = torch.zeros_like(q), torch.zeros_like(q)
    pc.scatter_add_(1, at, torch.where(entry, p, 0.0))
    epc.scatter_add_(1, at, torch.where(entry, ep + k * U * p, 0.0))
    dl = g * tau * (q - pc)
    edl = (g * tau).abs() * (q * eq + epc + 6 * U * (q + pc))
    zero = torch.zeros_like
    val = {"loss": torch.where(live, loss, 0.0)[:, 0], "dlogits": torch.where(live, dl, zero(dl)),
           "stats": torch.where(named, torch.cat([largest, torch.where(live, s, 0.0)], 1), 0.0)}
    err = {"loss": torch.where(live, eloss, 0.0)[:, 0], "dlogits": torch.where(live, edl, zero(dl)),
           "stats": torch.where(live, torch.cat([zero(s), s * es], 1), 0.0)}
    return val, err


def policy(logits, actions, old, adv, tau, ref=None, kl=0.0, low=0.2, high=0.2, dloss=None):
    """{"loss", "logp", "stats", "dlogits"} and bounds; the ratio's distance from its bounds is "clear"."""
    rows, vocab = logits.shape
    largest, s, q, dz, eq, es = _softmax(logits, tau)
    act = actions.long()
    named = (act >= 0) & (act < vocab)
    live = named & (largest[:, 0] > -math.inf)
    at = act.clamp(0, max(vocab - 1, 0))[:, None]
    lp = (dz.gather(1, at) - torch.log(s.clamp_min(1e-300)))[:, 0]
    elp = U * dz.gather(1, at)[:, 0].abs() + es[:, 0] + 2 * U
    old, adv = old.double(), adv.double()
    d = lp - old
    r = torch.exp(d)
    er = elp + U * d.abs() + 4 * U
    over = (adv > 0) & (r > 1 + high)
    under = (adv < 0) & (r < 1 - low)
    away = torch.zeros_like(lp) if ref is None or kl == 0 else ref.double() - lp
    first = torch.where(adv == 0, 0.0, torch.where(over, 1 + high, torch.where(under, 1 - low, r)) * adv)
    more = torch.expm1(away)
    loss = kl * (more - away) - first
    eaway = elp + U * away.abs()
    eloss = (torch.where(over | under, 4 * U * first.abs(), (er + 4 * U) * first.abs())
             + abs(kl) * (more.abs() * eaway + 4 * U * (more.abs() + away.abs())) + 4 * U * loss.abs()
             + abs(kl) * eaway * eaway * torch.exp(away))
    moving = torch.where(over | under | (adv == 0), 0.0, r * adv)
    g = -kl * more - moving
    eg = moving.abs() * (er + 4 * U) + abs(kl) * (torch.exp(away) * eaway + 4 * U * more.abs()) + 2 * U * g.abs()
    w = (torch.ones(rows, dtype=torch.float64) if dloss is None else dloss.double()) / tau
    hot = torch.zeros_like(q)
    if vocab:
        hot.scatter_(1, at, 1.0)
    dl = (w * g)[:, None] * (hot - q)
    edl = (w.abs() * (eg + 6 * U * g.abs()))[:, None] * (hot - q).abs() + (w * g).abs()[:, None] * (q * eq + 4 * U * (q + hot))
    keep = lambda v: torch.where(live, v, 0.0)  # noqa: E731
    wide = lambda v: torch.where(live[:, None], v, 0.0)  # noqa: E731
    val = {"loss": keep(loss), "logp": keep(lp), "dlogits": wide(dl),
           "stats": torch.where(named[:, None], torch.cat([largest, torch.where(live[:, None], s, 0.0)], 1), 0.0)}
    err = {"loss": keep(eloss), "logp": keep(elp), "dlogits": wide(edl),
           "stats": wide(torch.cat([torch.zeros_like(s), s * es], 1))}
    clear = torch.where(live, torch.minimum((r / (1 + high) - 1).abs(), (r - (1 - low)).abs()), 1.0)
    return val, err, clear
