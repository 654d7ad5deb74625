"""Training operators without a GPU: the C ABI refuses bad arguments before
anything is enqueued, empty calls are accepted, workspace sizes, the binding's
own checks, and the references the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import bit_adamw_optimizer_amd as M
from tests import train_ref as R

P = ctypes.c_void_p
F32, F16, BF16 = 0, 1, 2


def _err():
    return M.lib().msamp_last_error().decode()


def _ck(codes=0x10000, ld=64, scales=0x20000, lds=2, fmt=0):
    return ctypes.byref(M._Checkpoint(codes, ld, scales, lds, fmt))


def _save(rows=4, cols=64, x=0x30000, ldx=64, dtype=F16, ck=None):
    return M.lib().msamp_checkpoint_save(rows, cols, P(x), ldx, dtype, ck if ck is not None else _ck(), None)


def test_checkpoint_refuses():
    assert _save(rows=-1) == 1 and "negative" in _err()
    assert _save(cols=-1) == 1
    assert _save(cols=1 << 31) == 1
    assert _save(dtype=3) == 1 and "dtype" in _err()
    assert _save(x=0) == 1 and "x is NULL" in _err()
    assert _save(x=0x30001) == 2
    assert _save(x=0x30002, dtype=F32) == 2
    assert _save(ldx=-64) == 1
    assert _save(ldx=1 << 60) == 1
    assert _save(ck=_ck(fmt=2)) == 1
    assert _save(ck=_ck(codes=0)) == 1 and "ckpt.codes" in _err()
    assert _save(ck=_ck(scales=0)) == 1 and "ckpt.scales" in _err()
    assert _save(ck=_ck(ld=63)) == 1 and "less than a row" in _err()
    assert _save(ck=_ck(lds=1)) == 1
    assert M.lib().msamp_checkpoint_save(4, 64, P(0x30000), 64, F16, None, None) == 1
    L = M.lib().msamp_checkpoint_load
    assert L(4, 64, _ck(), P(0), 64, F16, None) == 1 and "out" in _err()
    assert L(4, 64, _ck(), P(0x30000), 63, F16, None) == 1
    assert L(4, 64, _ck(ld=-1), P(0x30000), 64, F16, None) == 1
    # nothing to do
    assert _save(rows=0, x=0) == 0 and _save(cols=0, x=0) == 0
    assert L(0, 64, _ck(codes=0, scales=0), P(0), 64, F16, None) == 0


def _fwd(rows=4, cols=64, x=0x30000, ldx=64, ck=None, dtype=F16, w=0x40000, b=0x50000, wd=F16, y=0x60000, ldy=64,
         mean=0x70000, rstd=0x80000, eps=1e-5, save=None):
    return M.lib().msamp_layernorm_forward(rows, cols, P(x), ldx, ck, dtype, P(w), P(b), wd, P(y), ldy, P(mean),
                                           P(rstd), eps, save, None)


def _bwd(rows=4, cols=64, dy=0x30000, x=0x90000, ck=None, dtype=F16, w=0x40000, wd=F16, mean=0x70000, rstd=0x80000,
         dx=0x60000, dw=0xA0000, db=0xB0000, ws=0xC0000, n=None, ldx=64):
    need = M.lib().msamp_layernorm_backward_workspace(max(rows, 0), max(cols, 0))
    return M.lib().msamp_layernorm_backward(rows, cols, P(dy), cols, P(x), ldx, ck, dtype, P(w), wd, P(mean), P(rstd),
                                            P(dx), cols, P(dw), P(db), 0, P(ws), need if n is None else n, None)


def test_norm_refuses():
    assert _fwd(rows=-1) == 1 and _fwd(cols=32769, ldx=40000, ldy=40000) == 1 and "32768" in _err()
    assert _fwd(dtype=7) == 1 and _fwd(wd=BF16) == 1 and "weight_dtype" in _err()
    assert _fwd(x=0) == 1 and _fwd(y=0) == 1 and _fwd(rstd=0) == 1
    assert _fwd(ldy=63) == 1 and _fwd(y=0x60001) == 2 and _fwd(w=0x40001) == 2 and _fwd(mean=0x70002) == 2
    assert _fwd(eps=-1e-9) == 1 and _fwd(eps=float("nan")) == 1 and _fwd(eps=float("inf")) == 1
    assert _fwd(ck=_ck()) == 1 and "both" in _err()
    assert _fwd(x=0, ck=_ck(), save=_ck()) == 1 and "save" in _err()
    assert _fwd(save=_ck(ld=1)) == 1
    assert _fwd(rows=0) == 0 and _fwd(cols=0) == 0
    assert _bwd(dy=0) == 1 and _bwd(dx=0) == 1 and _bwd(rstd=0) == 1 and _bwd(x=0) == 1
    assert _bwd(ws=0) == 1 and "workspace" in _err()
    assert _bwd(ws=0xC0008) == 2
    assert _bwd(n=8) == 1 and "needed" in _err()
    assert _bwd(ck=_ck()) == 1
    assert _bwd(rows=0, dw=0, db=0, dy=0, x=0, dx=0, rstd=0, mean=0) == 0
    W = M.lib().msamp_layernorm_backward_workspace
    assert W(-1, 4) == -1 and W(4, 40000) == -1 and W(0, 64) == 0 and W(1, 64) > 0


def _ffn(**kw):
    a = M._GatedFfn(4, 64, 96, F16, 0, 0x10000, 64, None, 0x20000, 64, 0x30000, 64, 0x40000, 96, 0x50000, 96,
                    0x60000, 64, 0x70000, 64, 0x80000, 64, F16, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _run(a, which, ws=0x100000, n=1 << 30):
    f = getattr(M.lib(), "msamp_gated_ffn_" + which)
    return f(ctypes.byref(a), P(ws), n, None)


def test_ffn_refuses():
    for which in ("forward", "backward"):
        W = getattr(M.lib(), "msamp_gated_ffn_%s_workspace" % which)
        assert W(ctypes.byref(_ffn())) >= 0 and W(ctypes.byref(_ffn(tokens=-1))) == -1 and W(None) == -1
        for bad in (dict(tokens=-1), dict(hidden=-1), dict(ffn=1 << 31), dict(dtype=F32), dict(act=3), dict(x=0),
                    dict(w_gate=0), dict(w_up=0), dict(ldx=-1), dict(ldh=95)):
            assert _run(_ffn(**bad), which) == 1, (which, bad)
        for bad in (dict(x=0x10001), dict(w_up=0x30001), dict(h=0x40001)):
            assert _run(_ffn(**bad), which) == 2, (which, bad)
        assert M.lib().msamp_gated_ffn_forward(None, None, 0, None) == 1
    assert _run(_ffn(h=0), "forward") == 1
    ck = M._Checkpoint(0x10000, 64, 0x20000, 2, 0)
    assert _run(_ffn(x=0, x_ckpt=ctypes.pointer(ck)), "forward") == 1 and "checkpoint" in _err()
    for bad in (dict(dh=0), dict(dx=0), dict(dw_gate=0), dict(dw_up=0), dict(lddx=63), dict(dw_dtype=BF16),
                dict(dw_accumulate=1), dict(x_ckpt=ctypes.pointer(ck))):
        assert _run(_ffn(**bad), "backward") == 1, bad
    assert _run(_ffn(dw_gate=0x70002, dw_dtype=F32), "backward") == 2
    assert _run(_ffn(), "backward", ws=0) == 1 and "workspace" in _err()
    assert _run(_ffn(), "backward", ws=0x100008) == 2
    assert _run(_ffn(), "backward", n=16) == 1 and "needed" in _err()
    # nothing to write
    assert _run(_ffn(tokens=0, x=0, h=0), "forward") == 0 and _run(_ffn(ffn=0, h=0), "forward") == 0


def test_shared_memory_is_refused():
    assert _save(x=0x10010) == 1 and "x and ckpt overlap" in _err()
    assert _save(x=0x20004) == 1
    L = M.lib().msamp_checkpoint_load
    assert L(4, 64, _ck(), P(0x10000 - 2), 64, F16, None) == 1 and "ckpt and out overlap" in _err()
    # a checkpoint whose scales lie in its codes' rows: apart behind the columns, not within them
    assert L(4, 64, _ck(scales=0x10020), P(0x1000A), 80, F16, None) == 1
    assert _save(ck=_ck(ld=66, scales=0x1003F, lds=66)) == 1 and "ckpt and ckpt overlap" in _err()
    for role, at in (("x and y", 0x30040), ("weight and y", 0x40000 - 64), ("y and mean", 0x70000), ("y and rstd", 0x80000)):
        assert _fwd(y=at) == 1 and role + " overlap" in _err(), role
    assert _fwd(mean=0x80000) == 1 and _fwd(save=_ck(codes=0x30000)) == 1 and _fwd(save=_ck(scales=0x60000)) == 1
    # y in x's place, but not with other rows
    assert _fwd(y=0x30000, ldy=65) == 1 and _fwd(y=0x30000, ldx=0) == 1
    # columns of one buffer whose rows have the same distance, overlapping by one
    assert _fwd(y=0x30000 + 126, ldx=128, ldy=128) == 1 and _fwd(y=0x30000 - 126, ldx=128, ldy=128) == 1
    for role, kw in (("dy and dx", dict(dx=0x30002)), ("x and dx", dict(dx=0x90002)), ("weight and dweight", dict(dw=0x40000)),
                     ("dweight and dbias", dict(db=0xA0000)), ("rstd and dbias", dict(db=0x80000)),
                     ("dx and workspace", dict(ws=0x60000))):
        assert _bwd(**kw) == 1 and role + " overlap" in _err(), role
    # one row may name any distance to the next
    assert _fwd(rows=1, ldx=1 << 62, ldy=1 << 62, y=0x30040) == 1 and "x and y overlap" in _err()
    for which in ("forward", "backward"):
        assert _run(_ffn(h=0x10000), which) == 1 and "x and h overlap" in _err()
        assert _run(_ffn(h=0x20000), which) == 1 and _run(_ffn(h=0x30002), which) == 1
    for kw in (dict(dx=0x10000), dict(dx=0x20000), dict(dw_gate=0x80000), dict(dw_up=0x30000), dict(dh=0x40000),
               dict(dx=0x50000)):
        assert _run(_ffn(**kw), "backward") == 1 and "overlap" in _err(), kw
    assert _run(_ffn(), "backward", ws=0x80000) == 1 and "workspace overlap" in _err()


def test_eps_beyond_binary32_is_refused():
    assert _fwd(eps=1e39) == 1 and "eps" in _err()


def test_sizes_beyond_the_matrix_kernels_are_refused():
    big = dict(hidden=1 << 22, ldx=1 << 22, ld_gate=1 << 22, ld_up=1 << 22, lddx=1 << 22, ld_dw_gate=1 << 22,
               ld_dw_up=1 << 22, tokens=100, ffn=96)
    assert M.lib().msamp_gated_ffn_forward_workspace(ctypes.byref(_ffn(**big))) == -1 and "2^22" in _err()
    assert M.lib().msamp_gated_ffn_backward_workspace(ctypes.byref(_ffn(**big))) == -1 and "2^22" in _err()
    wide = dict(ffn=1 << 21, ldh=1 << 21, lddh=1 << 21)
    assert M.lib().msamp_gated_ffn_backward_workspace(ctypes.byref(_ffn(**wide))) == -1 and "2^21" in _err()
    # as many rows as an int takes: a plan, or a refusal
    for t in (1 << 24, (1 << 31) - 1):
        for which in ("forward", "backward"):
            W = getattr(M.lib(), "msamp_gated_ffn_%s_workspace" % which)
            assert W(ctypes.byref(_ffn(tokens=t, ffn=1, ldh=1, lddh=1))) >= -1


def test_binding_refuses_host_tensors_and_bad_types():
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        M.checkpoint_save(x, None)
    with pytest.raises(ValueError):
        M.Checkpoint(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), 64)
    with pytest.raises(ValueError):
        M.layernorm_forward(x, None, None, x, None, x)
    with pytest.raises(ValueError):
        M.gated_ffn_forward(x, x, x, x)


def test_profile_kinds_have_names_in_order():
    for i, name in enumerate(M.KERNELS):
        assert M.lib().msamp_kernel_name(i).decode() == name


@pytest.mark.parametrize("fmt,dt", [(0, torch.float8_e4m3fn), (1, torch.float8_e5m2)])
def test_reference_codec_agrees_with_torch_in_range(fmt, dt):
    t = R.decode_table(fmt)
    codes = np.arange(256, dtype=np.uint8)
    v = torch.from_numpy(codes.copy()).view(dt).float().numpy()
    assert np.array_equal(t[~np.isnan(t)], v[~np.isnan(v)].astype(np.float64)) and np.array_equal(np.isnan(t), np.isnan(v))
    fine = np.isfinite(t)
    assert np.array_equal(R.encode(t[fine], fmt), codes[fine])
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * R.FP8_MAX[fmt] * 0.2
    x = np.clip(x, -R.FP8_MAX[fmt], R.FP8_MAX[fmt])
    assert np.array_equal(R.encode(x.astype(np.float64), fmt), torch.from_numpy(x).to(dt).view(torch.uint8).numpy())


@pytest.mark.parametrize("act", list(M.ACTIVATIONS))
def test_reference_gradients_agree_with_autograd(act):
    torch.manual_seed(3)
    x, wg, wu = (torch.randn(s, dtype=torch.float64, requires_grad=True) for s in ((5, 7), (9, 7), (9, 7)))
    dh = torch.randn(5, 9, dtype=torch.float64)
    if act == "silu":
        a = torch.nn.functional.silu(x @ wg.t())
    else:
        a = torch.nn.functional.gelu(x @ wg.t(), approximate="tanh" if act == "gelu_tanh" else "none")
    h = a * (x @ wu.t())
    grads = torch.autograd.grad(h, (x, wg, wu), dh)
    val, _ = R.ffn(x.detach(), wg.detach(), wu.detach(), act, dh)
    for name, ref in zip(("h", "dx", "dw_gate", "dw_up"), (h,) + grads):
        assert torch.allclose(val[name], ref, rtol=1e-12, atol=1e-12), name


@pytest.mark.parametrize("centered", [True, False])
def test_reference_norm_gradients_agree_with_autograd(centered):
    torch.manual_seed(4)
    x = torch.randn(6, 11, dtype=torch.float64, requires_grad=True)
    w, b = (torch.randn(11, dtype=torch.float64, requires_grad=True) for _ in range(2))
    dy = torch.randn(6, 11, dtype=torch.float64)
    y, mu, rstd, _ = R.norm_forward(x, w, b, 1e-5, centered)
    gx, gw, gb = torch.autograd.grad(y, (x, w, b), dy)
    dx, dw, db, *_ = R.norm_backward(dy, x.detach(), w.detach(), mu.detach(), rstd.detach(), centered)
    for got, ref in ((dx, gx), (dw, gw), (db, gb)):
        assert torch.allclose(got, ref, rtol=1e-12, atol=1e-12)


def _bytes(rows, cols):
    return torch.zeros(rows, cols, dtype=torch.uint8)


@pytest.mark.parametrize("call", ["save", "load", "norm saves", "norm reads", "norm backward", "block backward"])
def test_a_checkpoint_is_taken_as_its_fields_are_at_the_call(call, monkeypatch):
    """Host tensors stand for the GPU's; what would go to the library is looked at instead of run."""
    sent = []
    monkeypatch.setattr(M, "_device_of", lambda t, name: t.get_device())
    monkeypatch.setattr(M, "_workspace", lambda n, dev: torch.empty(n + 16, dtype=torch.uint8))
    monkeypatch.setattr(M, "_run", lambda dev, entry, *args: sent.append(args))
    rows, cols, f16 = 4, 64, torch.float16
    x, y, vec = torch.zeros(rows, cols, dtype=f16), torch.zeros(rows, cols, dtype=f16), torch.zeros(rows)
    w = torch.zeros(32, cols, dtype=f16)
    ck = M.Checkpoint(_bytes(rows, cols), _bytes(rows, 2), cols)

    def struct():
        del sent[:]
        if call == "save":
            M.checkpoint_save(x, ck)
        elif call == "load":
            M.checkpoint_load(ck, x)
        elif call == "norm saves":
            M.layernorm_forward(x, None, None, y, None, vec, save=ck)
        elif call == "norm reads":
            M.layernorm_forward(ck, None, None, y, None, vec)
        elif call == "norm backward":
            M.layernorm_backward(x, ck, None, None, vec, y, None, None)
        else:
            M.gated_ffn_backward(torch.zeros(rows, 32, dtype=f16), ck, w, w, y, w.clone(), w.clone())
        for a in sent[0]:
            a = getattr(a, "_obj", a)  # a byref
            if isinstance(a, M._GatedFfn):
                return a.x_ckpt.contents
            if isinstance(a, M._Checkpoint):
                return a
        raise AssertionError("no checkpoint among the arguments")

    def same():
        c = struct()
        return (c.codes, c.ld, c.scales, c.ld_scales, c.fmt) == (
            ck.codes.data_ptr(), ck.codes.stride(0), ck.scales.data_ptr(), ck.scales.stride(0), ck.fmt)

    first = ck.codes, ck.scales  # alive: no address is used twice
    assert same()
    ck.codes = _bytes(rows, cols + 5)
    assert same() and ck.codes.data_ptr() != first[0].data_ptr()
    ck.scales = _bytes(rows, 7)
    assert same()
    ck.codes.data = _bytes(rows, cols + 32)
    assert same()
    ck.codes.set_(_bytes(rows, cols + 64))
    assert same()
    ck.scales.resize_(rows, 100000)
    assert same()
    ck.fmt = M.E5M2
    assert same()
    # what no longer fits is refused, not read with the shape it had
    ck.codes = _bytes(rows + 1, cols)
    with pytest.raises(ValueError):
        struct()
    ck.codes = _bytes(rows, cols).expand(rows, cols)[:, :cols - 1]
    with pytest.raises(ValueError):
        struct()
    ck.codes, ck.scales = _bytes(1, cols).expand(rows, cols), _bytes(rows, 2)
    if call in ("save", "norm saves"):
        with pytest.raises(ValueError):
            struct()
    else:
        assert same()
    ck.codes, ck.cols = _bytes(rows, cols), 63
    with pytest.raises(ValueError):
        struct()
    ck.codes, ck.cols = torch.zeros(rows, cols, dtype=f16), cols
    with pytest.raises(TypeError):
        struct()
    ck.codes = first[0]
    assert same() and (ck.rows, ck.device) == (rows, -1)


@pytest.mark.parametrize("tokens,ffn,forward,backward", [
    (1 << 24, 1, True, True), (1 << 24, 96, True, True), (1 << 30, 1, True, True), (600000000, 96, True, True),
    # tiles of 256 rows: 2^23 - 1 of them, with those of the weights' gradients in the backward pass
    (((1 << 23) - 3) * 256, 1, True, True), (((1 << 23) - 3) * 256 + 1, 1, True, False),
    (((1 << 23) - 1) * 256, 96, True, False), ((1 << 31) - 1, 1, False, False), (1 << 30, 300, False, False)])
def test_how_many_tokens_are_planned(tokens, ffn, forward, backward):
    """The largest numbers of tokens are planned up to the limit the header states, and refused beyond it."""
    for which, fits in (("forward", forward), ("backward", backward)):
        a = _ffn(tokens=tokens, ffn=ffn, ldh=ffn, lddh=ffn)
        # far apart: nothing overlaps
        a.x, a.h, a.dh, a.dx = (i << 44 for i in range(1, 5))
        n = getattr(M.lib(), "msamp_gated_ffn_%s_workspace" % which)(ctypes.byref(a))
        plan = (ctypes.c_int32 * 6)()
        st = M.lib().msamp_gated_ffn_plan(ctypes.byref(a), int(which == "backward"), plan)
        assert (n >= 0, st == 0) == (fits, fits), (which, n, plan[:], _err())
        if not fits:
            assert n == -1 and "too many tiles" in _err()
        else:
            # the operands of the gradients' products, 64-column pieces of dg and du in 16 bits, and nothing
            # like it in the forward pass, whose operands here lie as they are read
            gates = tokens * 2 * (-(-ffn // 64) * 64) * 2 if which == "backward" else 0
            assert gates <= n <= gates + (1 << 28), (which, n)


@pytest.mark.parametrize("field", ["codes", "scales"])
def test_a_checkpoint_without_its_tensors_is_refused(field, monkeypatch):
    with monkeypatch.context() as m:
        m.setattr(M, "_device_of", lambda t, name: t.get_device())
        ck = M.Checkpoint(_bytes(4, 64), _bytes(4, 2), 64)
    setattr(ck, field, None)
    with pytest.raises(TypeError, match=field):
        ck._arg("ckpt", -1, (4, 64))
