"""Measured cases of the operators at the two ends of a model and between its
tokens: embedding lookup and its gradient, the gated linear recurrence (forward
and backward), distillation from a teacher's top logits, and the clipped policy
loss with a KL term (losses and gradients).

`run` computes one pass of a case: through the library where `own` is true,
otherwise in its plain form, elementary torch operations in binary32 (the policy
loss's values of a row in binary64: its clip is a border) with one rounding at
the end. `exact` gives the same outputs from the definitions in binary64.

  embedding      y[t] = scale W[id_t];  dW[v] = scale sum over {t: id_t = v} of dy[t]
                 (an id outside [0, vocab) is padding: a row of zeros, no gradient)
  recurrence     a = 1 / (1 + e^-gate);  h_t = a_t h_{t-1} + (1 - a_t) x_t;  y = h
                 (states: h before every 32nd step, what the backward pass starts from)
  distillation   p = softmax(teacher's listed logits / tau), q = softmax(z / tau):
                 loss = tau^2 sum p (log p - log q) over the listed ids (one of -1 is absent)
  policy         lp = log softmax(z / tau)[action], r = e^(lp - old):
                 loss = -min(r A, clip(r, 1 - lo, 1 + hi) A) + kl (e^(ref - lp) - (ref - lp) - 1)
                 (an action of -1 is a masked row: loss and gradient 0)
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
CHUNK = 32  # steps between two saved states


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one decoded position of 16 GPT-2-small sequences: launch latency
        dict(name="embedding_fwd_token", op="embedding_fwd", rows=16, vocab=50257, cols=768, pad=0, dtype="f16",
             scale=1.0, padding=0.0),
        # four 4,096-token sequences of the Llama-2-7B shape, scaled by the root of the width
        dict(name="embedding_fwd", op="embedding_fwd", rows=16384, vocab=32000, cols=4096, pad=0, dtype="bf16",
             scale=64.0, padding=0.0),
        # its gradient: dense, binary32, as the optimizer step's quantize takes it
        dict(name="embedding_bwd", op="embedding_bwd", rows=16384, vocab=32000, cols=4096, pad=0, dtype="bf16",
             scale=64.0, padding=0.0, accumulate=False),
        # an odd width and a padded batch, added to the output projection's gradient of the same (tied) weight
        dict(name="embedding_bwd_tied", op="embedding_bwd", rows=5003, vocab=50257, cols=1027, pad=0, dtype="f16",
             scale=1.0, padding=0.2, accumulate=True),
        # one decoded token of 64 sequences, the state carried along: launch latency
        dict(name="recurrence_token", op="recurrence_fwd", batch=64, time=1, channels=4096, pad=0, dtype="bf16",
             state=True, ragged=False),
        # four 4,096-token sequences of 4,096 channels, keeping the states of the backward pass
        dict(name="recurrence_fwd", op="recurrence_fwd", batch=4, time=4096, channels=4096, pad=0, dtype="bf16",
             state=False, ragged=False),
        # its backward pass
        dict(name="recurrence_bwd", op="recurrence_bwd", batch=4, time=4096, channels=4096, pad=0, dtype="bf16",
             state=False, ragged=False),
        # long sequences of different lengths, few channels and an odd number of them, with gradients of the states
        dict(name="recurrence_bwd_long", op="recurrence_bwd", batch=2, time=16411, channels=999, pad=0, dtype="f16",
             state=True, ragged=True),
        # a few rows of the Llama-2 vocabulary, as a short prompt gives: latency
        dict(name="distill_small", op="distill", rows=16, vocab=32000, top=20, pad=0, dtype="bf16", tau=2.0,
             mode="fused"),
        # two 4,096-token sequences, loss and gradient in one call
        dict(name="distill", op="distill", rows=8192, vocab=32000, top=64, pad=0, dtype="bf16", tau=2.0, mode="fused"),
        # four 1,024-token rollouts over the GPT-2 vocabulary, whose rows start on no whole 16 bytes
        dict(name="policy", op="policy", rows=4096, vocab=50257, pad=0, dtype="bf16", tau=1.0, kl=0.05, mode="fused"),
        # binary32 logits over a long vocabulary: the gradient alone, from the statistics the forward pass kept
        dict(name="policy_bwd", op="policy", rows=500, vocab=131072, pad=0, dtype="f32", tau=0.7, kl=0.0, mode="bwd"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _size(rng, lo, hi):
    """Spread over the logarithm; half of the sizes are multiples of 64, the others any number."""
    n = _log(rng, lo, hi)
    return max(lo, n // 64 * 64) if n >= 64 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["embedding_fwd", "embedding_bwd", "recurrence_fwd", "recurrence_bwd", "distill", "policy"])
    case = dict(op=op, dtype=rng.choice(["f32", "f16", "bf16"]), pad=rng.choice([0, 0, 0, 8, 3]))
    wide = BYTES[case["dtype"]] // 2
    if op.startswith("embedding"):
        vocab = _size(rng, 64, 131072)
        cols = _size(rng, 32, min(8192, max(32, 32000 * 4096 // vocab)))
        rows = _size(rng, 1, max(1, min(65536, 16384 * 4096 // (wide * cols))))
        case.update(rows=rows, vocab=vocab, cols=cols, scale=rng.choice([1.0, round(cols ** 0.5, 3)]),
                    padding=rng.choice([0.0, 0.0, 0.3]))
        if op == "embedding_bwd":
            case.update(accumulate=rng.random() < 0.3)
    elif op.startswith("recurrence"):
        most = 4 * 4096 * 4096 // wide
        time = _size(rng, 1, 65536)
        channels = _size(rng, 1, min(8192, most // time))
        case.update(batch=_log(rng, 1, max(1, min(64, most // (time * channels)))), time=time, channels=channels,
                    state=rng.random() < 0.5, ragged=time > 1 and rng.random() < 0.3)
    else:
        vocab = _size(rng, 100, 262144)
        case.update(vocab=vocab, rows=_size(rng, 1, max(1, min(16384, 8192 * 32000 // (wide * vocab)))),
                    tau=rng.choice([1.0, 1.0, 2.0, 0.7]), mode=rng.choice(["fused", "fused", "fwd", "bwd"]))
        if op == "distill":
            case.update(top=_log(rng, 1, 100))
        else:
            case.update(kl=rng.choice([0.0, 0.05]))
    return case


def _distinct(rows, vocab):
    """Expected number of different ids among `rows` of _tokens()."""
    edge = torch.log(torch.arange(1, vocab + 2, dtype=torch.float64)) / math.log(vocab + 1)
    return float((1 - (1 - (edge[1:] - edge[:-1])) ** rows).sum())


def work(case):
    """Bytes and operations no implementation can do without: every input read once, every output written once."""
    b, op = BYTES[case["dtype"]], case["op"]
    if op.startswith("embedding"):
        live = case["rows"] * (1 - case["padding"])
        rows = _distinct(live, case["vocab"])
        if op == "embedding_fwd":
            return {"bytes": 8 * case["rows"] + case["cols"] * b * (rows + case["rows"]),
                    "flops": float(case["rows"] * case["cols"])}
        out = 8 * rows if case["accumulate"] else 4 * case["vocab"]
        return {"bytes": 8 * case["rows"] + case["cols"] * (b * live + out), "flops": 2.0 * live * case["cols"]}
    if op.startswith("recurrence"):
        lines = case["batch"] * case["channels"]
        n = lines * case["time"] * (0.75 if case["ragged"] else 1)  # _lengths()'s mean
        states = 4 * n / CHUNK if case["time"] > 1 else 0
        ends = 8 * lines if case["state"] else 0
        if op == "recurrence_fwd":
            return {"bytes": 3 * b * n + states + ends, "flops": 8.0 * n}
        return {"bytes": 5 * b * n + states + ends, "flops": 20.0 * n}
    n = case["rows"] * case["vocab"]
    side = case["rows"] * (4 + (12 * case["top"] if op == "distill" else 20))
    return {"bytes": n * b * (1 if case["mode"] == "fwd" else 2) + side, "flops": 5.0 * n}


# ------------------------------------------------------------------ inputs ---

def _rows(rows, cols, pad, dtype, make):
    """A [rows, cols] view of rows `cols + pad` long."""
    t = torch.empty(rows, cols + pad, dtype=dtype, device="cuda")
    t[:, :cols] = make
    return t[:, :cols]


def _cube(case, make):
    """A [batch, time, channels] view of steps `channels + pad` long."""
    b, t, c = case["batch"], case["time"], case["channels"]
    return _rows(b * t, c, case["pad"], DTYPES[case["dtype"]], make).unflatten(0, (b, t))


def _tokens(rows, vocab, padding, gen):
    """Ids with frequencies that fall as 1 / rank, ranks spread over the vocabulary; some of them padding."""
    u = torch.rand(rows, device="cuda", generator=gen, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1)
    ids = torch.randperm(vocab, device="cuda", generator=gen)[rank]
    return torch.where(torch.rand(rows, device="cuda", generator=gen) < padding, -1, ids)


def _lengths(case, gen):
    """From half of the steps to all of them, the first sequence having all."""
    t = case["time"]
    n = (t - torch.randint(0, t // 2 + 1, (case["batch"],), device="cuda", generator=gen)).int()
    n[0] = t
    return n


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 29)
    dt, op = DTYPES[case["dtype"]], case["op"]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if op.startswith("embedding"):
        rows, vocab, cols = case["rows"], case["vocab"], case["cols"]
        s["ids"] = _tokens(rows, vocab, case["padding"], gen)
        if op == "embedding_fwd":
            s["weight"] = _rows(vocab, cols, case["pad"], dt, randn(vocab, cols).mul_(0.02))
            s["y"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        else:
            s["dy"] = _rows(rows, cols, case["pad"], dt, randn(rows, cols).mul_(0.02))
            # the output projection's gradient where it is added to
            s["dweight"] = randn(vocab, cols) if case["accumulate"] else torch.empty(vocab, cols, device="cuda")
        return s
    if op.startswith("recurrence"):
        b, t, c = case["batch"], case["time"], case["channels"]
        # channels that forget within a step or two up to some that remember hundreds
        memory = 7 * torch.rand(c, device="cuda", generator=gen) - 1
        s["x"] = _cube(case, randn(b * t, c))
        s["gate"] = _cube(case, randn(b * t, c).add_(memory))
        s["lengths"] = _lengths(case, gen) if case["ragged"] else None
        s["h0"] = randn(b, c).mul_(0.5) if case["state"] else None
        if op == "recurrence_fwd":
            s["y"] = torch.zeros(b, t, c, dtype=dt, device="cuda")
            s["h_last"] = torch.empty(b, c, device="cuda") if case["state"] else None
            # a decoded token needs no backward pass
            s["states"] = torch.zeros(b, -(-t // CHUNK), c, device="cuda") if t > 1 else None
        else:
            h = _states(s)[1]
            s["states"] = h[:, ::CHUNK].contiguous()  # as the forward pass kept them
            s["dy"] = _cube(case, randn(b * t, c).mul_(0.02))
            s["dh_last"] = randn(b, c).mul_(0.02) if case["state"] else None
            s["dh0"] = torch.empty(b, c, device="cuda") if case["state"] else None
            s["dx"] = torch.zeros(b, t, c, dtype=dt, device="cuda")
            s["dgate"] = torch.zeros(b, t, c, dtype=dt, device="cuda")
        return s
    rows, vocab, tau = case["rows"], case["vocab"], case["tau"]
    z = randn(rows, vocab).mul_(2.5)
    s["logits"] = _rows(rows, vocab, case["pad"], dt, z)
    z.copy_(s["logits"])
    s["dloss"] = torch.full((rows,), 1024.0 / rows, device="cuda")  # a mean over the rows, times a loss scale
    if op == "distill":
        s["teacher"], s["ids"] = z.add(randn(rows, vocab)).topk(case["top"], 1)
        if case["top"] > 1:  # rows for which the teacher gave fewer
            s["ids"][::5, -1] = -1
        s["loss"] = torch.empty(rows, device="cuda")
    else:
        s["actions"] = (z / tau - torch.log(-torch.log(torch.rand(rows, vocab, device="cuda", generator=gen)
                                                       .clamp_(1e-9, 1 - 1e-7)))).argmax(1)
        lp = (z / tau).gather(1, s["actions"][:, None])[:, 0] - torch.logsumexp(z / tau, 1)
        s["old"], s["ref"] = lp + 0.15 * randn(rows), lp + 0.3 * randn(rows)
        s["advantages"] = randn(rows)
        s["actions"][3::7] = -1  # the prompt's rows
        s["loss"], s["logp"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    if case["mode"] == "bwd":
        top = z.amax(1)
        z.sub_(top[:, None]).div_(tau)
        s["stats"] = torch.stack([top, z.exp_().sum(1, dtype=torch.float64).float()], 1)
    elif case["mode"] == "fwd":
        s["stats"] = torch.empty(rows, 2, device="cuda")
    if case["mode"] != "fwd":
        s["dlogits"] = torch.empty(rows, vocab, dtype=dt, device="cuda")
    return s


# -------------------------------------------------------------- plain form ---

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0, along dimension 1: spans of steps joined two by two, twice as long
    each time."""
    d, n = 1, a.shape[1]
    while d < n:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _gates(gate):
    """a = 1 / (1 + e^-gate) and 1 - a, each from its own exponential."""
    g = gate.float()
    return 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))


def _states(s):
    """h after each step and before each step."""
    a, keep = _gates(s["gate"])
    b = keep * s["x"].float()
    first = torch.zeros_like(b[:, 0]) if s["h0"] is None else s["h0"]
    b[:, 0] += a[:, 0] * first
    h = _scan(a, b)
    return h, torch.cat([first[:, None], h[:, :-1]], 1)


def _inside(s):
    """[batch, time, 1]: which steps belong to their sequences."""
    t = torch.arange(s["x"].shape[1], device="cuda")
    return (t[None] < s["lengths"][:, None])[:, :, None]


def _plain_recurrence(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    last = None if s["lengths"] is None else (s["lengths"].long() - 1)[:, None, None]
    if case["op"] == "recurrence_fwd":
        h, before = _states(s)
        out = {"y": h.to(dt) if last is None else torch.where(_inside(s), h.to(dt), s["y"])}
        if case["state"]:
            out["h_last"] = h[:, -1] if last is None else h.gather(1, last.expand(-1, -1, h.shape[2]))[:, 0]
        if s["states"] is not None:
            kept = before[:, ::CHUNK]
            out["states"] = kept if last is None else torch.where(_inside(s)[:, ::CHUNK], kept, s["states"])
        return out
    before = _states({**s, "h0": s["states"][:, 0]})[1]
    a, keep = _gates(s["gate"])
    dy = s["dy"].float()
    if last is not None:
        dy = torch.where(_inside(s), dy, 0.0)
    if case["state"]:
        end = s["dh_last"][:, None]
        if last is None:
            dy = torch.cat([dy[:, :-1], dy[:, -1:] + end], 1)
        else:
            dy = dy.scatter_add(1, last.expand(-1, -1, dy.shape[2]), end)
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    lam = _scan(after.flip(1), dy.flip(1)).flip(1)
    dx, dgate = keep * lam, lam * (before - s["x"].float()) * a * keep
    out = {"dx": dx.to(dt), "dgate": dgate.to(dt)}
    if last is not None:
        out = {k: torch.where(_inside(s), v, s[k]) for k, v in out.items()}
    if case["state"]:
        out["dh0"] = a[:, 0] * lam[:, 0]
    return out


def _plain_loss(s):
    case, dt, tau = s["case"], DTYPES[s["case"]["dtype"]], s["case"]["tau"]
    z = s["logits"].float()
    if case["mode"] == "bwd":
        top, total = s["stats"][:, :1], s["stats"][:, 1:].double()
        e = torch.exp((z - top) / tau)
    else:
        top = z.amax(1, keepdim=True)
        e = torch.exp((z - top) / tau)
        total = e.sum(1, keepdim=True, dtype=torch.float64)
    out = {}
    if case["mode"] == "fwd":
        out["stats"] = torch.cat([top, total.float()], 1)
    if case["op"] == "distill":
        live = s["ids"] >= 0
        ids = s["ids"].clamp_min(0)
        t = torch.where(live, s["teacher"], -math.inf)
        t = (t - t.amax(1, keepdim=True)) / tau
        p = torch.exp(t)
        sum_p = p.sum(1, keepdim=True)
        p = p / sum_p
        if case["mode"] != "bwd":
            log_p, log_q = t - torch.log(sum_p), (z.gather(1, ids) - top) / tau - torch.log(total).float()
            out["loss"] = tau * tau * torch.where(p > 0, p * (log_p - log_q), 0.0).sum(1)
        if case["mode"] != "fwd":
            q = (e / total.float()).scatter_add(1, ids, torch.where(live, -p, 0.0))
            out["dlogits"] = (q * (tau * s["dloss"][:, None])).to(dt)
        return out
    live = s["actions"] >= 0
    ids = s["actions"].clamp_min(0)[:, None]
    lp = ((z.gather(1, ids) - top).double() / tau - torch.log(total))[:, 0]
    adv, away = s["advantages"].double(), s["ref"].double() - lp
    r = torch.exp(lp - s["old"].double())
    beyond = ((adv > 0) & (r > 1.2)) | ((adv < 0) & (r < 0.8))
    if case["mode"] != "bwd":
        loss = -torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv) + case["kl"] * (torch.exp(away) - away - 1)
        out["loss"], out["logp"] = torch.where(live, loss, 0.0).float(), torch.where(live, lp, 0.0).float()
    if case["mode"] == "fwd":
        out["stats"] = torch.where(live[:, None], out["stats"], 0.0)
    else:
        dlp = torch.where(beyond, 0.0, -adv * r) + case["kl"] * (1 - torch.exp(away))
        dlp = (torch.where(live, dlp, 0.0) * s["dloss"] / tau).float()[:, None]
        out["dlogits"] = (-dlp * (e / total.float())).scatter_add(1, ids, dlp).to(dt)
    return out


def _plain(s):
    case = s["case"]
    if case["op"] == "embedding_fwd":
        live = (s["ids"] >= 0)[:, None]
        y = s["weight"][s["ids"].clamp_min(0)].float() * case["scale"]
        return {"y": torch.where(live, y, 0.0).to(DTYPES[case["dtype"]])}
    if case["op"] == "embedding_bwd":
        live = s["ids"] >= 0
        if not case["accumulate"]:
            s["dweight"].zero_()
        s["dweight"].index_add_(0, s["ids"][live], s["dy"][live].float() * case["scale"])
        return {"dweight": s["dweight"]}
    return _plain_recurrence(s) if case["op"].startswith("recurrence") else _plain_loss(s)


# ------------------------------------------------------ the library's calls ---

def _own(s):
    import bit_adamw_optimizer_amd as M

    case = s["case"]
    op = case["op"]
    if op == "embedding_fwd":
        M.embedding_forward(s["ids"], s["weight"], s["y"], scale=case["scale"])
        return {"y": s["y"]}
    if op == "embedding_bwd":
        M.embedding_backward(s["dy"], s["ids"], s["dweight"], scale=case["scale"], accumulate=case["accumulate"])
        return {"dweight": s["dweight"]}
    if op == "recurrence_fwd":
        M.recurrence_forward(s["x"], s["gate"], s["y"], h0=s["h0"], h_last=s["h_last"], states=s["states"],
                             lengths=s["lengths"])
        return {k: s[k] for k in ("y", "h_last", "states") if s[k] is not None}
    if op == "recurrence_bwd":
        M.recurrence_backward(s["dy"], s["x"], s["gate"], s["states"], s["dx"], s["dgate"], dh_last=s["dh_last"],
                              dh0=s["dh0"], lengths=s["lengths"])
        return {k: s[k] for k in ("dx", "dgate", "dh0") if s[k] is not None}
    mode, tau = case["mode"], case["tau"]
    more = {} if mode == "fwd" else dict(dlogits=s["dlogits"], dloss=s["dloss"])
    if mode == "fwd":
        more["stats"] = s["stats"]
    if op == "distill":
        if mode == "bwd":
            M.distill_loss_backward(s["dloss"], s["logits"], s["ids"], s["teacher"], s["stats"], s["dlogits"],
                                    temperature=tau)
            return {"dlogits": s["dlogits"]}
        M.distill_loss_forward(s["logits"], s["ids"], s["teacher"], s["loss"], temperature=tau, **more)
        return {k: s[k] for k in ("loss", "stats" if mode == "fwd" else "dlogits")}
    ref = s["ref"] if case["kl"] else None
    if mode == "bwd":
        M.policy_loss_backward(s["dloss"], s["logits"], s["actions"], s["old"], s["advantages"], s["stats"],
                               s["dlogits"], ref_logp=ref, kl=case["kl"], clip_low=0.2, clip_high=0.2, temperature=tau)
        return {"dlogits": s["dlogits"]}
    M.policy_loss_forward(s["logits"], s["actions"], s["old"], s["advantages"], s["loss"], logp=s["logp"],
                          ref_logp=ref, kl=case["kl"], clip_low=0.2, clip_high=0.2, temperature=tau, **more)
    return {k: s[k] for k in ("loss", "logp", "stats" if mode == "fwd" else "dlogits")}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------- definitions, 64 ---

def _exact_loss(s):
    """The losses from torch's log-softmax, their gradients by differentiation."""
    case, tau, rows = s["case"], s["case"]["tau"], s["case"]["rows"]
    z = s["logits"].double().requires_grad_(case["mode"] != "fwd")
    log_q = torch.log_softmax(z / tau, 1)
    pick = torch.arange(rows, device="cuda")
    if case["op"] == "distill":
        live = s["ids"] >= 0
        t = (s["teacher"].double() / tau).masked_fill(~live, -math.inf)
        log_p = torch.log_softmax(t, 1).masked_fill(~live, 0.0)
        p = log_p.exp() * live
        loss = tau ** 2 * (p * (log_p - log_q[pick[:, None], s["ids"].clamp_min(0)])).sum(1)
        out = {"loss": loss.detach()}
    else:
        live = s["actions"] >= 0
        lp = log_q[pick, s["actions"].clamp_min(0)]
        ratio, adv = (lp - s["old"].double()).exp(), s["advantages"].double()
        away = s["ref"].double() - lp
        loss = -torch.min(ratio * adv, ratio.clamp(0.8, 1.2) * adv) + case["kl"] * (torch.expm1(away) - away)
        loss = loss * live
        out = {"loss": loss.detach(), "logp": (lp * live).detach()}
    if case["mode"] == "fwd":
        top = z.amax(1)
        stats = torch.stack([top, torch.exp((z - top[:, None]) / tau).sum(1)], 1)
        return {**out, "stats": stats * live[:, None] if case["op"] == "policy" else stats}
    if case["mode"] == "bwd":
        out = {}
    return {**out, "dlogits": torch.autograd.grad(loss, z, s["dloss"].double())[0]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embedding_fwd":
        table = torch.cat([s["weight"].double(), torch.zeros(1, case["cols"], dtype=torch.float64, device="cuda")])
        return {"y": table[s["ids"]] * case["scale"]}  # -1 takes the zeros at the end
    if case["op"] == "embedding_bwd":
        order = torch.argsort(s["ids"], stable=True)
        sums = torch.zeros(case["vocab"] + 1, case["cols"], dtype=torch.float64, device="cuda")
        sums.index_put_((s["ids"][order],), s["dy"][order].double() * case["scale"], accumulate=True)
        return {"dweight": sums[:-1] + (s["dweight"].double() if case["accumulate"] else 0)}
    if not case["op"].startswith("recurrence"):
        return _exact_loss(s)
    # the recurrence, step by step
    n = case["time"]
    x, g = s["x"].double(), s["gate"].double()
    a, keep = torch.sigmoid(g), torch.sigmoid(-g)
    back = case["op"] == "recurrence_bwd"
    first = s["states"][:, 0] if back else s["h0"]
    h = torch.zeros_like(x[:, 0]) if first is None else first.double()
    hs = [h]
    for t in range(n):
        new = a[:, t] * h + keep[:, t] * x[:, t]
        h = new if s["lengths"] is None else torch.where((t < s["lengths"])[:, None], new, h)
        hs.append(h)
    hs = torch.stack(hs, 1)
    inside = torch.ones_like(x, dtype=torch.bool) if s["lengths"] is None else _inside(s).expand_as(x)
    if not back:
        out = {"y": torch.where(inside, hs[:, 1:], s["y"].double())}
        if case["state"]:
            out["h_last"] = hs[:, -1]
        if s["states"] is not None:
            out["states"] = torch.where(inside[:, ::CHUNK], hs[:, :-1:CHUNK], s["states"].double())
        return out
    dy = s["dy"].double()
    carry = torch.zeros_like(x[:, 0]) if s["dh_last"] is None else s["dh_last"].double()
    dx, dgate = s["dx"].double(), s["dgate"].double()
    for t in range(n - 1, -1, -1):
        lam = dy[:, t] + carry
        slope = (hs[:, t] - x[:, t]) * a[:, t] * keep[:, t]
        dx[:, t] = torch.where(inside[:, t], keep[:, t] * lam, dx[:, t])
        dgate[:, t] = torch.where(inside[:, t], lam * slope, dgate[:, t])
        carry = torch.where(inside[:, t], a[:, t] * lam, carry)
    out = {"dx": dx, "dgate": dgate}
    if case["state"]:
        out["dh0"] = carry
    return out
