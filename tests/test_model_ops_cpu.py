"""Embedding, gated recurrence and losses without a GPU: the C ABI refuses bad
arguments before anything is enqueued, empty calls are accepted, the binding's
own checks, and the references that the GPU tests compare with against
differentiation and differences."""
import ctypes

import pytest
import torch

import bit_adamw_optimizer_amd as M
from tests import model_ref as R

P = ctypes.c_void_p
F32, F16, BF16 = 0, 1, 2


def _err():
    return M.lib().msamp_last_error().decode()


# --------------------------------------------------------------- embedding ---

def _efwd(rows=4, vocab=9, cols=64, ids=0x10000, ib=8, w=0x20000, ldw=64, dt=F16, y=0x30000, ldy=64, scale=1.0):
    return M.lib().msamp_embedding_forward(rows, vocab, cols, P(ids), ib, P(w), ldw, dt, P(y), ldy, scale, None)


def _ebwd(rows=4, vocab=9, cols=64, ids=0x10000, ib=8, dy=0x20000, lddy=64, dt=F16, dw=0x30000, ldw=64, scale=1.0,
          ws=0x40000, n=None):
    need = M.lib().msamp_embedding_backward_workspace(max(rows, 0), max(vocab, 0), max(cols, 0))
    return M.lib().msamp_embedding_backward(rows, vocab, cols, P(dy), lddy, dt, P(ids), ib, P(dw), ldw, scale, 0, P(ws),
                                            need if n is None else n, None)


def test_embedding_refuses():
    assert _efwd(rows=-1) == 1 and "negative" in _err()
    assert _efwd(rows=1 << 31) == 1 and _efwd(vocab=(1 << 30) + 1) == 1 and _efwd(cols=(1 << 22) + 1, ldw=1 << 23, ldy=1 << 23) == 1
    assert _efwd(ib=2) == 1 and "id_bytes" in _err()
    assert _efwd(dt=3) == 1 and _efwd(scale=float("nan")) == 1 and _efwd(scale=1e39) == 1 and "scale" in _err()
    assert _efwd(ids=0) == 1 and "ids is NULL" in _err()
    assert _efwd(w=0) == 1 and _efwd(y=0) == 1 and _efwd(ldy=63) == 1 and _efwd(ldw=-1) == 1
    assert _efwd(ids=0x10004) == 2 and _efwd(w=0x20001) == 2 and _efwd(y=0x30001) == 2
    for kw, what in ((dict(y=0x20000), "weight and y"), (dict(y=0x10010), "ids and y")):
        assert _efwd(**kw) == 1 and what + " overlap" in _err()
    assert _efwd(rows=0, ids=0, y=0) == 0 and _efwd(cols=0, w=0, y=0) == 0
    assert _ebwd(dy=0) == 1 and _ebwd(dw=0) == 1 and _ebwd(ids=0) == 1 and _ebwd(ldw=63) == 1 and _ebwd(scale=float("inf")) == 1
    assert _ebwd(ws=0) == 1 and "workspace" in _err()
    assert _ebwd(ws=0x40008) == 2 and _ebwd(n=8) == 1 and "needed" in _err()
    assert _ebwd(dw=0x30002) == 2
    for kw, what in ((dict(dw=0x20100), "dy and dweight"), (dict(ws=0x30010), "dweight and workspace"),
                     (dict(dw=0x10000), "ids and dweight"), (dict(ws=0x20000), "dy and workspace")):
        assert _ebwd(**kw) == 1 and what + " overlap" in _err()
    assert _ebwd(vocab=0, dw=0) == 0 and _ebwd(cols=0, dy=0, dw=0) == 0
    W = M.lib().msamp_embedding_backward_workspace
    assert W(-1, 4, 4) == -1 and W(4, 4, 1 << 23) == -1 and W(0, 0, 0) >= 0 and W(1 << 20, 4, 64) > 4 << 20


# -------------------------------------------------------------- recurrence ---

def _rec(**kw):
    """[4, 40, 64] in float16, everything at places of its own."""
    a = dict(batch=4, time=40, channels=64, dtype=F16, length_bytes=4, lengths=None, states=0x300000, h0=0x310000, ld_h0=64,
             h_last=0x320000, ld_h_last=64, dh_last=0x330000, ld_dh_last=64, dh0=0x340000, ld_dh0=64)
    for i, k in enumerate(("x", "gate", "y", "dy", "dx", "dgate")):
        a.update({k: 0x100000 + 0x10000 * i, k + "_batch": 40 * 64, k + "_time": 64})
    a.update(kw)
    s = M._Recurrence()
    for k, v in a.items():
        setattr(s, k, v)
    return s


def _rrun(which, ws=0x900000, n=1 << 30, **kw):
    return getattr(M.lib(), "msamp_recurrence_" + which)(ctypes.byref(_rec(**kw)), P(ws), n, None)


BOTH = ("forward", "backward")


@pytest.mark.parametrize("which", BOTH)
def test_recurrence_refuses(which):
    assert getattr(M.lib(), "msamp_recurrence_" + which)(None, None, 0, None) == 1
    for bad in (dict(batch=-1), dict(time=-1), dict(channels=-1), dict(time=1 << 31), dict(dtype=3), dict(x=0), dict(gate=0),
                dict(x_time=-1), dict(gate_batch=-1), dict(lengths=0x800000, length_bytes=2),
                dict(batch=1 << 23, x_batch=0, gate_batch=0), dict(x_batch=1 << 60)):
        assert _rrun(which, **bad) == 1, bad
        W = getattr(M.lib(), "msamp_recurrence_%s_workspace" % which)
        assert W(ctypes.byref(_rec(**bad))) == -1, bad
    for bad in (dict(x=0x100001), dict(gate=0x110001), dict(states=0x300002), dict(lengths=0x800002)):
        assert _rrun(which, **bad) == 2, bad
    assert _rrun(which, batch=0, x=0, gate=0, y=0, dy=0, dx=0, dgate=0, states=0, h0=0, h_last=0, dh_last=0, dh0=0) == 0


def test_recurrence_refuses_outputs():
    for bad in (dict(y=0), dict(y_time=63), dict(y_batch=64), dict(ld_h_last=63), dict(ld_h0=-1), dict(y_batch=39 * 64 + 63)):
        assert _rrun("forward", **bad) == 1, bad
    for bad in (dict(dy=0), dict(dx=0), dict(dgate=0), dict(states=0), dict(dx_time=63), dict(dgate_batch=64), dict(ld_dh0=63)):
        assert _rrun("backward", **bad) == 1, bad


def test_recurrence_memory_that_is_shared():
    def refused(which, what, **kw):
        assert _rrun(which, **kw) == 1 and what + " overlap" in _err(), (kw, _err())

    refused("forward", "x and y", y=0x100002)
    refused("forward", "x and y", y=0x100000, y_time=65, y_batch=65 * 40)
    refused("forward", "x and y", y=0x100000, y_batch=64 * 41)
    refused("forward", "gate and states", states=0x110000)
    refused("forward", "y and h_last", h_last=0x120000)
    refused("forward", "h0 and h_last", h_last=0x310004)
    refused("forward", "y and h0", h0=0x120000)
    refused("forward", "lengths and y", lengths=0x120000)
    refused("backward", "dx and dgate", dgate=0x140000)
    refused("backward", "dx and dgate", dx=0x130000, dgate=0x130000)  # both written over dy
    refused("backward", "states and dx", states=0x140000)
    refused("backward", "dh_last and dh0", dh0=0x330004)
    refused("backward", "dgate and dh0", dh0=0x150000)
    # halves of one buffer are apart, and overlapping by one element are not
    halves = dict(dx=0x400000, dx_time=128, dx_batch=128 * 40, dgate=0x400000 + 128, dgate_time=128, dgate_batch=128 * 40)
    refused("backward", "dx and dgate", **{**halves, "dgate": 0x400000 + 126})
    # time-major halves likewise
    major = dict(dx=0x400000, dx_time=128 * 4, dx_batch=128, dgate=0x400000 + 128, dgate_time=128 * 4, dgate_batch=128)
    refused("backward", "dx and dgate", **{**major, "dgate": 0x400000 + 126})
    # a state of the same shape and place as one step of x is still x
    refused("forward", "x and h_last", time=1, dtype=F32, h0=0, h_last=0x100000, ld_h_last=64, x_batch=64, y_batch=64, gate_batch=64)


def test_recurrence_parts_of_one_buffer_that_share_a_step_or_an_element():
    def refused(**kw):
        for which, what in (("forward", "x and y"), ("backward", "dx and dgate")):
            a, b = ("x", "y") if which == "forward" else ("dx", "dgate")
            args = {a + "_batch": kw["batch"], b + "_batch": kw["batch"], a + "_time": kw["time"], b + "_time": kw["time"],
                    a: 0x400000, b: 0x400000 + kw["apart"]}
            assert _rrun(which, **args) == 1 and what + " overlap" in _err(), (kw, _err())

    step, seq = 64 * 2, 40 * 64 * 2
    for pad in (0, 3):  # time halves
        long = 80 * 64 + pad
        for apart in (2, step, seq - step, seq - 2, 2 * long + seq - 2, 2 * long + step):
            refused(batch=long, time=64, apart=apart)
        # column halves of sequences that start anywhere
        for apart in (2, step - 2, 39 * 2 * step + step - 2, 2 * long + step - 2):
            refused(batch=long, time=128, apart=apart)
    # time-major halves
    refused(batch=64, time=8 * 64, apart=4 * step - 2)
    refused(batch=64, time=8 * 64, apart=3 * step)


# ------------------------------------------------------------------ losses ---

def _loss(**kw):
    a = dict(rows=4, vocab=100, dtype=F16, id_bytes=8, logits=0x100000, ld_logits=100, ids=0x110000, ld_ids=5, temperature=1.0,
             loss=0x120000, stats=0x130000, dloss=0x140000, dlogits=0x150000, ld_dlogits=100, top=5, teacher=0x160000,
             ld_teacher=5, teacher_dtype=F32, old_logp=0x170000, ref_logp=0x180000, advantages=0x190000, logp=0x1A0000,
             clip_low=0.2, clip_high=0.2, kl=0.1)
    a.update(kw)
    s = M._VocabLoss()
    for k, v in a.items():
        setattr(s, k, v)
    return s


def _lrun(which, back=False, ws=0x900000, **kw):
    a = ctypes.byref(_loss(**kw))
    if back:
        return getattr(M.lib(), "msamp_%s_backward" % which)(a, None)
    return getattr(M.lib(), "msamp_%s_forward" % which)(a, P(ws), 1 << 30, None)


@pytest.mark.parametrize("which", ("distill", "policy"))
def test_losses_refuse(which):
    assert getattr(M.lib(), "msamp_%s_forward" % which)(None, None, 0, None) == 1
    assert getattr(M.lib(), "msamp_%s_backward" % which)(None, None) == 1
    W = getattr(M.lib(), "msamp_%s_forward_workspace" % which)
    assert W(None) == -1 and W(ctypes.byref(_loss())) >= 0
    for bad in (dict(rows=-1), dict(vocab=-1), dict(rows=1 << 31), dict(vocab=(1 << 29) + 1), dict(dtype=3), dict(id_bytes=1),
                dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=1e39),
                dict(temperature=1e-39), dict(logits=0), dict(ids=0), dict(ld_logits=-1), dict(ld_dlogits=99)):
        for back in (False, True):
            assert _lrun(which, back, **bad) == 1, (bad, back)
        assert W(ctypes.byref(_loss(**bad))) == -1
    for bad in (dict(logits=0x100001), dict(ids=0x110004), dict(stats=0x130002), dict(dlogits=0x150001)):
        for back in (False, True):
            assert _lrun(which, back, **bad) == 2, (bad, back)
    assert _lrun(which, loss=0) == 1 and "loss is NULL" in _err()
    assert _lrun(which, True, stats=0) == 1 and _lrun(which, True, dlogits=0) == 1
    for kw, what in ((dict(dlogits=0x100002), "logits and dlogits"), (dict(loss=0x150000), "loss and dlogits"),
                     (dict(stats=0x120000), "loss and stats"), (dict(dloss=0x150010), "dlogits and dloss"),
                     (dict(dlogits=0x100000, ld_dlogits=101), "logits and dlogits")):
        assert _lrun(which, **kw) == 1 and what + " overlap" in _err(), (kw, _err())
    assert _lrun(which, rows=0, logits=0, ids=0, loss=0, stats=0, dlogits=0, dloss=0, teacher=0, old_logp=0, ref_logp=0,
                 advantages=0, logp=0) == 0
    assert _lrun(which, True, rows=0, logits=0, ids=0, loss=0, stats=0, dlogits=0, dloss=0, teacher=0, old_logp=0, ref_logp=0,
                 advantages=0, logp=0) == 0


@pytest.mark.parametrize("which", ("distill", "policy"))
def test_losses_refuse_a_temperature_whose_exponents_are_infinite(which):
    for back in (False, True):  # 1 / 4e-39 is finite in binary32, log2(e) / 4e-39 is not
        assert _lrun(which, back, temperature=4e-39) == 1 and "temperature" in _err()


def test_losses_refuse_their_own():
    for bad in (dict(top=-1), dict(top=1025, ld_ids=1025, ld_teacher=1025), dict(teacher=0), dict(teacher_dtype=3), dict(ld_teacher=-1)):
        assert _lrun("distill", **bad) == 1, bad
    assert _lrun("distill", teacher=0x160002) == 2
    assert _lrun("distill", loss=0x160000) == 1 and "teacher and loss overlap" in _err()
    for bad in (dict(old_logp=0), dict(advantages=0), dict(ref_logp=0), dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_high=-0.1),
                dict(clip_low=float("nan")), dict(kl=float("inf")), dict(kl=float("nan"))):
        assert _lrun("policy", **bad) == 1, bad
    assert _lrun("policy", logp=0x120000) == 1 and "overlap" in _err()


def test_binding_refuses():
    f16 = torch.float16
    x = torch.zeros(4, 64, dtype=f16)
    c = torch.zeros(2, 3, 4, dtype=f16)
    i = torch.zeros(4, dtype=torch.int64)
    v = torch.zeros(4)
    with pytest.raises(ValueError, match="not on a GPU"):
        M.embedding_forward(i, x, x)
    with pytest.raises(ValueError, match="not on a GPU"):
        M.embedding_backward(x, i, x.float())
    with pytest.raises(ValueError, match="not on a GPU"):
        M.recurrence_forward(c, c, c)
    with pytest.raises(ValueError, match="not on a GPU"):
        M.recurrence_backward(c, c, c, torch.zeros(2, 1, 4), c, c)
    with pytest.raises(TypeError):
        M.recurrence_backward(c, c, c, None, c, c)
    with pytest.raises(ValueError, match="not on a GPU"):
        M.distill_loss_forward(x, i[:, None], v[:, None], v)
    with pytest.raises(ValueError, match="not on a GPU"):
        M.policy_loss_forward(x, i, v, v, v)
    for f in (lambda: M.distill_loss_forward(x, i[:, None], v[:, None], None),
              lambda: M.distill_loss_backward(v, x, i[:, None], v[:, None], None, x),
              lambda: M.policy_loss_forward(x, i, v, v, None), lambda: M.policy_loss_backward(v, x, i, v, v, None, x)):
        with pytest.raises(TypeError):
            f()


def test_binding_checks_what_it_sends(monkeypatch):
    """Host tensors stand for the GPU's; what would go to the library is looked at instead of run."""
    sent = []
    monkeypatch.setattr(M, "_device_of", lambda t, name: t.get_device())
    monkeypatch.setattr(M, "_workspace", lambda n, dev: torch.empty(n + 16, dtype=torch.uint8))
    monkeypatch.setattr(M, "_run", lambda dev, entry, *args: sent.append(args))
    f16, B, T, C = torch.float16, 2, 70, 8
    p = torch.zeros(B, T, 2 * C, dtype=f16)
    y, st, h = torch.zeros(B, T, C, dtype=f16), M.new_recurrence_states(B, T, C, "cpu"), torch.zeros(B, C)
    assert st.shape == (B, 3, C)
    M.recurrence_forward(p[..., :C], p[..., C:], y, h0=h, h_last=h, states=st, lengths=torch.tensor([1, 70]))
    a = sent[-1][0]
    assert (a.batch, a.time, a.channels, a.dtype, a.length_bytes) == (B, T, C, F16, 8)
    assert (a.x, a.x_batch, a.x_time) == (p.data_ptr(), T * 2 * C, 2 * C) and a.gate == p.data_ptr() + 2 * C
    assert (a.h0, a.h_last, a.ld_h0, a.states, a.dy) == (h.data_ptr(), h.data_ptr(), C, st.data_ptr(), None)
    dx, dg = torch.zeros_like(y), torch.zeros(T, B, C, dtype=f16).transpose(0, 1)
    M.recurrence_backward(y, p[..., :C], p[..., C:], st, dx, dg, dh_last=h, dh0=h)
    a = sent[-1][0]
    assert (a.dy, a.dx, a.dgate_batch, a.dgate_time, a.dh_last, a.dh0) == (
        y.data_ptr(), dx.data_ptr(), C, B * C, h.data_ptr(), h.data_ptr()) and a.y is None and a.h0 is None
    bad = [dict(states=st[:, :2]), dict(states=st.half()), dict(lengths=torch.zeros(3, dtype=torch.int32)),
           dict(lengths=torch.zeros(B)), dict(h0=h.half()), dict(h_last=h[:1]), dict(h_last=h[:1].expand(B, C))]
    for kw in bad:
        with pytest.raises((TypeError, ValueError)):
            M.recurrence_forward(p[..., :C], p[..., C:], y, **kw)
    for x, g, out in ((p, p, y), (p[..., :C].float(), p[..., C:], y), (p[..., ::2], p[..., C:], y),
                      (p[..., :C], p[..., C:], y[:1].expand(B, T, C)), (p[..., :C], p[..., C:], y[:, :1].expand(B, T, C)),
                      (p[0, :, :C], p[..., C:], y), (p[..., :C], p[..., C:], y[0])):
        with pytest.raises((TypeError, ValueError)):
            M.recurrence_forward(x, g, out)

    z, ids, t, v = torch.zeros(4, 9, dtype=f16), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, 3), torch.zeros(4)
    M.distill_loss_forward(z, ids, t, v, temperature=2.0, dlogits=z, dloss=torch.ones(4))
    a = sent[-1][0]
    assert (a.rows, a.vocab, a.id_bytes, a.top, a.dlogits, a.temperature) == (4, 9, 4, 3, z.data_ptr(), 2.0)
    for f in (lambda: M.distill_loss_forward(z, ids, t, v, dloss=v), lambda: M.distill_loss_forward(z, ids, t[:, :2], v),
              lambda: M.distill_loss_forward(z, ids.float(), t, v), lambda: M.distill_loss_forward(z, ids, t.long(), v),
              lambda: M.distill_loss_forward(z, ids, t, v, stats=torch.zeros(4)), lambda: M.distill_loss_forward(z, ids[0], t, v),
              lambda: M.distill_loss_forward(z, ids, t, v, dlogits=z.float())):
        with pytest.raises((TypeError, ValueError)):
            f()
    act = torch.zeros(4, dtype=torch.int64)
    M.policy_loss_forward(z, act, v, v.clone(), torch.zeros(4), logp=torch.zeros(4), stats=torch.zeros(4, 2))
    a = sent[-1][0]
    assert (a.id_bytes, a.clip_low, a.clip_high, a.kl, a.ref_logp) == (8, 0.2, 0.2, 0.0, None)
    for f in (lambda: M.policy_loss_forward(z, act[:3], v, v, v), lambda: M.policy_loss_forward(z, act, v.double(), v, v),
              lambda: M.policy_loss_forward(z, act, v, v, v[::2]), lambda: M.policy_loss_forward(z, act, v, v, v, ref_logp=v[:2])):
        with pytest.raises((TypeError, ValueError)):
            f()

    w = torch.zeros(11, 9, dtype=f16)
    M.embedding_forward(act, w, z, scale=3.0)
    assert sent[-1][:5] == (4, 11, 9, act.data_ptr(), 8)
    M.embedding_backward(z, act.int(), w.float(), accumulate=True)
    for f in (lambda: M.embedding_forward(act[:3], w, z), lambda: M.embedding_forward(act, w.float(), z),
              lambda: M.embedding_forward(act, w[:, :8], z), lambda: M.embedding_forward(act.float(), w, z),
              lambda: M.embedding_backward(z, act, w), lambda: M.embedding_backward(z, act, w.float().t())):
        with pytest.raises((TypeError, ValueError)):
            f()


# -------------------------------------------------------------- references ---

def test_reference_embedding_gradient_agrees_with_autograd():
    torch.manual_seed(0)
    w = torch.randn(7, 5, dtype=torch.float64, requires_grad=True)
    ids = torch.tensor([3, 0, 3, -1, 6, 9, 3])
    dy = torch.randn(7, 5, dtype=torch.float64)
    y, _ = R.embedding_forward(ids, w, 1.5)
    assert (y[3] == 0).all() and (y[5] == 0).all() and torch.equal(y[0], w[3] * 1.5)
    (g,) = torch.autograd.grad(y, w, dy)
    assert torch.allclose(R.embedding_backward(dy, ids, 7, 1.5)[0], g, rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("lengths", [None, [70, 33, 0]])
def test_reference_recurrence_gradients_agree_with_autograd_and_differences(lengths):
    torch.manual_seed(1)
    B, T, C = 3, 70, 4
    x, g = torch.randn(B, T, C, dtype=torch.float64, requires_grad=True), torch.randn(B, T, C, dtype=torch.float64, requires_grad=True)
    h0 = torch.randn(B, C, dtype=torch.float64, requires_grad=True)
    dy, dl = torch.randn(B, T, C, dtype=torch.float64), torch.randn(B, C, dtype=torch.float64)
    n = None if lengths is None else torch.tensor(lengths)
    live = torch.ones(B, T, 1) if n is None else (torch.arange(T)[None] < n[:, None])[..., None]

    def total(x, g, h0):
        hs, _ = R.recurrence_forward(x, g, h0, n)
        return (hs[:, 1:] * dy * live).sum() + (hs[:, -1] * dl).sum()

    hs, _ = R.recurrence_forward(x, g, h0, n)
    val, _ = R.recurrence_backward(dy, x.detach(), g.detach(), hs[:, :-1:R.CHUNK].detach(), dl, n)
    for name, ref in zip(("dx", "dgate", "dh0"), torch.autograd.grad(total(x, g, h0), (x, g, h0))):
        got = val[name] * live if name != "dh0" else val[name]
        assert torch.allclose(got, ref, rtol=1e-10, atol=1e-12), name
    with torch.no_grad():
        for t, name in ((x, "dx"), (g, "dgate")):
            for at in ((0, 0, 0), (1, 32, 2), (0, 69, 3)):
                d = torch.zeros_like(t)
                d[at] = 1e-5
                args = [(t + s * d if u is t else u) for s in (1, -1) for u in (x, g, h0)]
                slope = (total(*args[:3]) - total(*args[3:])) / 2e-5
                assert abs(slope - val[name][at] * live[at[0], at[1], 0]) < 1e-8


def test_reference_losses_agree_with_autograd():
    torch.manual_seed(2)
    rows, vocab, tau = 6, 30, 1.7
    z = (2 * torch.randn(rows, vocab, dtype=torch.float64)).requires_grad_()
    w = torch.rand(rows, dtype=torch.float64) + 0.5
    ids = torch.stack([torch.randperm(vocab)[:4] for _ in range(rows)])
    ids[1, 2], ids[2, 1] = ids[1, 0], -1  # the same class twice; an absent entry
    t = torch.randn(rows, 4, dtype=torch.float64)
    lq = torch.log_softmax(z / tau, 1)
    lt = torch.log_softmax((t / tau).masked_fill(ids < 0, -torch.inf), 1).masked_fill(ids < 0, 0)
    loss = tau ** 2 * ((lt.exp() * (ids >= 0)) * (lt - lq.gather(1, ids.clamp_min(0)))).sum(1)
    val, _ = R.distill(z.detach(), ids, t, tau, w)
    assert torch.allclose(val["loss"], loss, rtol=1e-12, atol=1e-12)
    assert torch.allclose(val["dlogits"], torch.autograd.grad(loss, z, w)[0], rtol=1e-10, atol=1e-12)
    # one class is the cross-entropy
    val, _ = R.distill(z.detach(), ids[:, :1], t[:, :1], 1.0)
    assert torch.allclose(val["loss"], torch.nn.functional.cross_entropy(z, ids[:, 0], reduction="none"), rtol=1e-12)

    act = torch.tensor([3, 4, -1, 0, 29, 7])
    lp = torch.log_softmax(z / tau, 1).gather(1, act.clamp_min(0)[:, None])[:, 0]
    old, ref = (lp + torch.tensor([0.0, -0.4, 0.1, 0.4, -0.4, 0.4])).detach(), (lp + 0.3 * torch.randn(rows)).detach()
    adv = torch.tensor([1.0, 2.0, 1.0, -1.0, -2.0, 0.5], dtype=torch.float64)
    r = (lp - old).exp()
    loss = (-torch.min(r * adv, r.clamp(0.8, 1.3) * adv) + 0.2 * (torch.expm1(ref - lp) - (ref - lp))) * (act >= 0)
    val, _, _ = R.policy(z.detach(), act, old, adv, tau, ref, 0.2, 0.2, 0.3, w)
    assert torch.allclose(val["loss"], loss, rtol=1e-12, atol=1e-12)
    assert torch.allclose(val["dlogits"], torch.autograd.grad(loss, z, w)[0], rtol=1e-10, atol=1e-12)
    assert (val["loss"][2], val["logp"][2]) == (0, 0) and (val["stats"][2] == 0).all()
