"""The gated feed-forward block on the GPU, forward and backward, against the
binary64 reference (tests/train_ref.py), which also bounds the errors of the
binary32 sums and of the one intermediate rounding (dg and du to the 16-bit
type)."""
import pytest
import torch

import bit_adamw_optimizer_amd as M
from tests import train_ref as R

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# one token, a few, ragged, whole tiles and just beyond them; hidden sizes that are no multiple of anything
SHAPES = [(1, 64, 96, 0), (1, 1000, 129, 0), (3, 40, 7, 1), (16, 128, 256, 0), (17, 136, 264, 8), (65, 257, 130, 0),
          (128, 256, 512, 0), (129, 300, 513, 3), (256, 64, 256, 0), (300, 1, 33, 0), (31, 33, 1, 0)]


def matrix(rows, cols, dtype, pad, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * size
    buf = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = x.to(dtype)
    return buf[:, :cols]


def out(rows, cols, dtype, value=7.0):
    """A matrix inside a larger buffer, whose rest has to stay."""
    buf = torch.full((rows + 1, cols + 2), value, dtype=dtype, device="cuda")
    return buf, buf[:rows, :cols]


def untouched(buf, rows, cols, value=7.0):
    return bool((buf[rows:] == value).all() and (buf[:, cols:] == value).all())


def problem(t, k, f, dt, pad=0, seed=0):
    return (matrix(t, k, dt, pad, seed), matrix(f, k, dt, pad, seed + 1, 1.3 * k ** -0.5),
            matrix(f, k, dt, pad, seed + 2, 1.3 * k ** -0.5), matrix(t, f, dt, pad, seed + 3, 0.1))


def check(names, got, val, err, dt):
    for name in names:
        R.assert_near(got[name], val[name], err[name], name)
        # the roundings are as good as independent: in the 2-norm the last one is at most half a step of each
        # value, and those of dg, du before it weigh no more than it does each
        ref = val[name]
        rel = ((got[name].cpu().double() - ref).norm() / ref.norm().clamp_min(1e-300)).item()
        assert rel <= 3 * R.half(dt) + (err[name].norm() / ref.norm().clamp_min(1e-300)).item() * 0.25, (name, rel)


@pytest.mark.parametrize("act", list(M.ACTIVATIONS))
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("t,k,f,pad", SHAPES)
def test_forward(t, k, f, pad, dtype, act):
    dt = DT[dtype]
    x, wg, wu, _ = problem(t, k, f, dt, pad, seed=t + k)
    buf, h = out(t, f, dt)
    M.gated_ffn_forward(x, wg, wu, h, act=act)
    assert untouched(buf, t, f)
    val, err = R.ffn(x.cpu(), wg.cpu(), wu.cpu(), act, dtype=dt)
    check(["h"], {"h": h}, val, err, dt)


@pytest.mark.parametrize("act", list(M.ACTIVATIONS))
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("t,k,f,pad", SHAPES)
def test_backward(t, k, f, pad, dtype, act):
    dt = DT[dtype]
    x, wg, wu, dh = problem(t, k, f, dt, pad, seed=t + k)
    wide = (t + k + f) % 2 == 0  # binary32 or 16-bit weight gradients
    bufs = {"h": out(t, f, dt), "dx": out(t, k, dt), "dw_gate": out(f, k, torch.float32 if wide else dt),
            "dw_up": out(f, k, torch.float32 if wide else dt)}
    got = {n: v[1] for n, v in bufs.items()}
    M.gated_ffn_backward(dh, x, wg, wu, got["dx"], got["dw_gate"], got["dw_up"], act=act, h=got["h"])
    for n, (buf, v) in bufs.items():
        assert untouched(buf, *v.shape), n
    val, err = R.ffn(x.cpu(), wg.cpu(), wu.cpu(), act, dh.cpu(), dt)
    check(["h", "dx", "dw_gate", "dw_up"], got, val, err, dt)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("t,k,f", [(40, 96, 160), (130, 100, 257), (5, 1000, 64)])
def test_backward_from_a_checkpoint(t, k, f, dtype):
    """From the checkpoint: the same bits as from its values, in both formats."""
    dt = DT[dtype]
    x, wg, wu, dh = problem(t, k, f, dt, seed=k)
    for fmt in (M.E4M3, M.E5M2):
        ck = M.new_checkpoint(t, k, fmt)
        M.checkpoint_save(x, ck)
        xv = torch.empty_like(x)
        M.checkpoint_load(ck, xv)
        res = []
        for src in (ck, xv):
            h, dx = torch.empty(t, f, dtype=dt, device="cuda"), torch.empty(t, k, dtype=dt, device="cuda")
            a, b = torch.empty(f, k, device="cuda"), torch.empty(f, k, device="cuda")
            M.gated_ffn_backward(dh, src, wg, wu, dx, a, b, h=h)
            res.append((h, dx, a, b))
        assert all(torch.equal(p, q) for p, q in zip(*res))
        val, err = R.ffn(xv.cpu(), wg.cpu(), wu.cpu(), "silu", dh.cpu(), dt)
        check(["h", "dx", "dw_gate", "dw_up"], dict(zip(("h", "dx", "dw_gate", "dw_up"), res[0])), val, err, dt)


def test_accumulate_and_repeat():
    t, k, f = 200, 130, 140
    x, wg, wu, dh = problem(t, k, f, torch.float16)
    dx = torch.empty(t, k, dtype=torch.float16, device="cuda")
    a, b = torch.empty(f, k, device="cuda"), torch.empty(f, k, device="cuda")
    M.gated_ffn_backward(dh, x, wg, wu, dx, a, b)
    first = dx.clone()
    a2, b2 = torch.full_like(a, 0.5), torch.full_like(b, -2.0)
    M.gated_ffn_backward(dh, x, wg, wu, dx, a2, b2, accumulate=True)
    assert torch.equal(dx, first) and torch.equal(a2, 0.5 + a) and torch.equal(b2, -2.0 + b)


@pytest.mark.parametrize("t,k,f", [(1500, 200, 130), (3000, 72, 80), (40, 300, 700)])
def test_accumulate_over_split_sums_and_into_wide_rows(t, k, f):
    """Long sums over tokens are joined from parts before they are added; the gradients' rows lie apart."""
    x, wg, wu, dh = problem(t, k, f, torch.bfloat16)
    dx = torch.empty(t, k, dtype=torch.bfloat16, device="cuda")
    a, b = torch.empty(f, k, device="cuda"), torch.empty(f, k, device="cuda")
    M.gated_ffn_backward(dh, x, wg, wu, dx, a, b)
    val, err = R.ffn(x.cpu(), wg.cpu(), wu.cpu(), "silu", dh.cpu(), torch.bfloat16)
    check(["dx", "dw_gate", "dw_up"], {"dx": dx, "dw_gate": a, "dw_up": b}, val, err, torch.bfloat16)
    (buf, a2), (buf2, b2) = out(f, k, torch.float32, 0.5), out(f, k, torch.float32, -2.0)
    M.gated_ffn_backward(dh, x, wg, wu, dx, a2, b2, accumulate=True)
    assert torch.equal(a2, 0.5 + a) and torch.equal(b2, -2.0 + b)
    assert untouched(buf, f, k, 0.5) and untouched(buf2, f, k, -2.0)


def test_repeated_rows_of_dh_and_x():
    """Broadcast inputs (rows at distance 0): the sums of their gradients are the caller's."""
    t, k, f = 90, 136, 200
    x, wg, wu, dh = problem(t, k, f, torch.float16)
    xe, de = x[:1].expand(t, k), dh[:1].expand(t, f)
    dx, a, b = torch.empty_like(x), torch.empty(f, k, device="cuda"), torch.empty(f, k, device="cuda")
    M.gated_ffn_backward(de, xe, wg, wu, dx, a, b)
    val, err = R.ffn(xe.cpu(), wg.cpu(), wu.cpu(), "silu", de.cpu(), torch.float16)
    check(["dx", "dw_gate", "dw_up"], {"dx": dx, "dw_gate": a, "dw_up": b}, val, err, torch.float16)


def test_two_streams_at_once():
    """Calls that overlap have workspaces of their own."""
    dt = torch.bfloat16
    probs = [problem(400, 512, 1200, dt, seed=s) for s in (1, 2)]
    outs, want = [], []
    for x, wg, wu, dh in probs:
        o = (torch.empty_like(dh), torch.empty_like(x), torch.empty(1200, 512, device="cuda"), torch.empty(1200, 512, device="cuda"))
        M.gated_ffn_backward(dh, x, wg, wu, o[1], o[2], o[3], h=o[0])
        want.append([v.clone() for v in o])
        outs.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for s, (x, wg, wu, dh), o in zip(streams, probs, outs):
            with torch.cuda.stream(s):
                M.gated_ffn_backward(dh, x, wg, wu, o[1], o[2], o[3], h=o[0])
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(o, w))


def test_empty_calls():
    f16 = torch.float16
    e = lambda r, c: torch.empty(r, c, dtype=f16, device="cuda")  # noqa: E731
    full = lambda r, c: torch.full((r, c), 7.0, dtype=f16, device="cuda")  # noqa: E731
    M.gated_ffn_forward(e(0, 8), e(16, 8), e(16, 8), e(0, 16))
    M.gated_ffn_forward(e(4, 8), e(0, 8), e(0, 8), e(4, 0))
    h = full(4, 16)
    M.gated_ffn_forward(e(4, 0), e(16, 0), e(16, 0), h)  # sums of nothing
    assert not h.any()
    # no token: weight gradients of zero, or unchanged
    a, b = full(16, 8), full(16, 8)
    M.gated_ffn_backward(e(0, 16), e(0, 8), e(16, 8), e(16, 8), e(0, 8), a, b)
    assert not a.any() and not b.any()
    a, b = torch.full((16, 8), 7.0, device="cuda"), torch.full((16, 8), 7.0, device="cuda")
    M.gated_ffn_backward(e(0, 16), e(0, 8), e(16, 8), e(16, 8), e(0, 8), a, b, accumulate=True)
    assert (a == 7).all() and (b == 7).all()
    # no inner unit: no gradient of x
    dx = full(4, 8)
    M.gated_ffn_backward(e(4, 0), e(4, 8), e(0, 8), e(0, 8), dx, e(0, 8), e(0, 8))
    assert not dx.any()
    # no hidden unit
    h = full(4, 16)
    M.gated_ffn_backward(full(4, 16), e(4, 0), e(16, 0), e(16, 0), e(4, 0), e(16, 0), e(16, 0), h=h)
    assert not h.any()


def test_one_weight_for_gate_and_up_repeated_rows_and_views():
    dt = torch.bfloat16
    both = matrix(2 * 72, 80, dt, 0, 1, 0.1)  # gate and up as views of one tensor
    x = matrix(1, 80, dt, 0, 2).expand(50, 80)
    h, ref = torch.empty(50, 72, dtype=dt, device="cuda"), torch.empty(1, 72, dtype=dt, device="cuda")
    M.gated_ffn_forward(x, both[:72], both[72:], h)
    M.gated_ffn_forward(x[:1], both[:72].clone(), both[72:].clone(), ref)
    val, err = R.ffn(x.cpu(), both[:72].cpu(), both[72:].cpu(), "silu", dtype=dt)
    check(["h"], {"h": h}, val, err, dt)
    check(["h"], {"h": ref}, {"h": val["h"][:1]}, {"h": err["h"][:1]}, dt)
    M.gated_ffn_forward(x, both[:72], both[:72], h, act="gelu")  # the same weight twice
    val, err = R.ffn(x.cpu(), both[:72].cpu(), both[:72].cpu(), "gelu", dtype=dt)
    check(["h"], {"h": h}, val, err, dt)


@pytest.mark.parametrize("pads", [(0, 8), (8, 0), (0, 3), (16, 24)])
def test_weights_with_rows_of_different_length(pads):
    t, k, f = 70, 136, 200
    x, _, _, dh = problem(t, k, f, torch.float16)
    wg, wu = (matrix(f, k, torch.float16, pad, 5 + pad, 0.1) for pad in pads)
    got = {"h": torch.empty_like(dh), "dx": torch.empty_like(x),
           "dw_gate": torch.empty(f, k, device="cuda"), "dw_up": torch.empty(f, k, device="cuda")}
    M.gated_ffn_backward(dh, x, wg, wu, got["dx"], got["dw_gate"], got["dw_up"], h=got["h"])
    val, err = R.ffn(x.cpu(), wg.cpu(), wu.cpu(), "silu", dh.cpu(), torch.float16)
    check(["h", "dx", "dw_gate", "dw_up"], got, val, err, torch.float16)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("t,k,f,pads", [(1, 4242, 50, (0, 0, 0)), (2, 640, 33, (3, 0, 0)), (16, 777, 40, (0, 1, 5)),
                                        (17, 129, 70, (1, 1, 1)), (40, 1000, 31, (0, 3, 0)), (64, 65, 130, (7, 0, 2)),
                                        (5, 8192, 17, (8, 16, 24)), (60, 2000, 100, (1, 0, 0))])
def test_few_tokens_at_any_alignment(t, k, f, pads, dtype):
    dt = DT[dtype]
    x, wg, wu = (matrix(r, k, dt, pad, 3 * k + i, s) for i, (r, pad, s) in
                 enumerate(((t, pads[0], 1.0), (f, pads[1], k ** -0.5), (f, pads[2], k ** -0.5))))
    dh = matrix(t, f, dt, pads[0], 9, 0.1)
    val, err = R.ffn(x.cpu(), wg.cpu(), wu.cpu(), "silu", dh.cpu(), dt)
    buf, h = out(t, f, dt)
    M.gated_ffn_forward(x, wg, wu, h)
    assert untouched(buf, t, f)
    check(["h"], {"h": h}, val, err, dt)
    got = {"h": torch.empty_like(h), "dx": torch.empty(t, k, dtype=dt, device="cuda"),
           "dw_gate": torch.empty(f, k, device="cuda"), "dw_up": torch.empty(f, k, device="cuda")}
    M.gated_ffn_backward(dh, x, wg, wu, got["dx"], got["dw_gate"], got["dw_up"], h=got["h"])
    check(["h", "dx", "dw_gate", "dw_up"], got, val, err, dt)


def test_special_values_stay_in_their_token():
    """A token of NaN or infinity leaves the other tokens' rows as they are."""
    x, wg, wu, dh = problem(140, 200, 300, torch.bfloat16)
    outs = []
    for bad in (False, True):
        y = x.clone()
        if bad:
            y[3], y[77, 5] = float("nan"), float("inf")
        h, dx = torch.empty_like(dh), torch.empty_like(x)
        M.gated_ffn_backward(dh, y, wg, wu, dx, torch.empty_like(wg), torch.empty_like(wu), h=h)
        outs.append((h, dx))
    keep = [i for i in range(140) if i not in (3, 77)]
    for p, q in zip(*outs):
        assert torch.equal(p[keep], q[keep]) and torch.isnan(q[3]).all()


def test_large_gates_keep_their_limits():
    """Gates far out: act(g) is g or 0 there, its slope 1 or 0, and nothing overflows on the way."""
    dt = torch.bfloat16
    x = torch.tensor([[200.0], [-200.0], [30000.0], [-30000.0]], device="cuda").to(dt)
    one = torch.ones(8, 1, dtype=dt, device="cuda")
    up = torch.full((8, 1), 2.0 ** -7, dtype=dt, device="cuda")
    for act in M.ACTIVATIONS:
        h, dx = torch.empty(4, 8, dtype=dt, device="cuda"), torch.empty(4, 1, dtype=dt, device="cuda")
        a, b = torch.empty(8, 1, device="cuda"), torch.empty(8, 1, device="cuda")
        dh = torch.ones(4, 8, dtype=dt, device="cuda")
        M.gated_ffn_backward(dh, x, one, up, dx, a, b, act=act, h=h)
        xs = x.double().cpu()
        val, err = R.ffn(xs, one.cpu(), up.cpu(), act, dh.cpu(), dt)
        for name, g in (("h", h), ("dx", dx), ("dw_gate", a), ("dw_up", b)):
            R.assert_near(g, val[name], err[name], act + " " + name)


def test_gates_whose_powers_overflow():
    """g = 1e25: g^2 and g^3 leave binary32, the results do not."""
    dt = torch.bfloat16
    x = torch.tensor([[2.0 ** 83], [-2.0 ** 83]], device="cuda").to(dt)
    one = torch.ones(8, 1, dtype=dt, device="cuda")
    up = torch.full((8, 1), 2.0 ** -100, dtype=dt, device="cuda")
    dh = torch.full((2, 8), 2.0 ** -60, dtype=dt, device="cuda")
    for act in M.ACTIVATIONS:
        h, dx = torch.empty(2, 8, dtype=dt, device="cuda"), torch.empty(2, 1, dtype=dt, device="cuda")
        a, b = torch.empty(8, 1, device="cuda"), torch.empty(8, 1, device="cuda")
        M.gated_ffn_backward(dh, x, one, up, dx, a, b, act=act, h=h)
        # above: act(g) = g with slope 1; below: 0 with slope 0. All of it in powers of two.
        assert (h[0] == 2.0 ** 66).all() and (h[1] == 0).all(), act
        assert (a == 2.0 ** -77 * 2.0 ** 83).all() and (b == 2.0 ** 23 * 2.0 ** 83).all(), act
        assert dx[0, 0].item() == 8 * (2.0 ** -77 + 2.0 ** -77) and dx[1, 0].item() == 0, act


def test_refusals():
    x, wg, wu, dh = problem(4, 8, 16, torch.float16)
    h = torch.empty_like(dh)
    for bad in (dict(act="relu"),):
        with pytest.raises(ValueError):
            M.gated_ffn_forward(x, wg, wu, h, **bad)
    with pytest.raises(ValueError):
        M.gated_ffn_forward(x[:, :7], wg, wu, h)
    with pytest.raises(ValueError):
        M.gated_ffn_forward(x, wg, wu[:15], h)
    with pytest.raises(TypeError):
        M.gated_ffn_forward(x, wg, wu.bfloat16(), h)
    with pytest.raises(TypeError):
        M.gated_ffn_forward(x.float(), wg.float(), wu.float(), h.float())
    with pytest.raises(ValueError):
        M.gated_ffn_forward(x, wg, wu, h[:1].expand(4, 16))
    with pytest.raises(ValueError):
        M.gated_ffn_forward(x, torch.empty(8, 16, dtype=torch.float16, device="cuda").t(), wu, h)
    ck = M.new_checkpoint(4, 8)
    with pytest.raises(TypeError):
        M.gated_ffn_forward(ck, wg, wu, h)
    dx = torch.empty_like(x)
    with pytest.raises(TypeError):
        M.gated_ffn_backward(dh, x, wg, wu, dx, wg.clone(), wu.clone(), accumulate=True)
    with pytest.raises(TypeError):
        M.gated_ffn_backward(dh, x, wg, wu, dx, wg.clone(), wu.float())
    with pytest.raises(ValueError):
        M.gated_ffn_backward(dh, M.new_checkpoint(4, 9), wg, wu, dx, wg.clone(), wu.clone())


@pytest.mark.parametrize("t,k,f", [(3, 264, 520), (300, 264, 520)])
def test_gradients_against_differences(t, k, f):
    """Along one direction, against central differences of the binary64 product (the kernel's own forward pass
    is rounded to 16 bits, which differences would magnify)."""
    dt = torch.float16
    x, wg, wu, dh = problem(t, k, f, dt)
    dx = torch.empty_like(x)
    a, b = torch.empty(f, k, device="cuda"), torch.empty(f, k, device="cuda")
    M.gated_ffn_backward(dh, x, wg, wu, dx, a, b)
    v = [torch.randn(p.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(i)) * s
         for i, (p, s) in enumerate(((x, 1.0), (wg, k ** -0.5), (wu, k ** -0.5)))]
    p = [q.cpu().double() for q in (x, wg, wu)]
    step = 1e-5

    def f64(sign):
        y, g, u = (q + sign * step * d for q, d in zip(p, v))
        return (R.ffn(y, g, u, "silu")[0]["h"] * dh.cpu().double()).sum().item()

    diff = (f64(1) - f64(-1)) / (2 * step)
    terms = [(q.cpu().double() * d) for q, d in zip((dx, a, b), v)]
    along = sum(q.sum().item() for q in terms)
    val, err = R.ffn(*p, "silu", dh.cpu(), dt)
    bound = sum(((err[n] + R.half(dt) * val[n].abs() + R.floor_of(dt)) * d.abs()).sum().item()
                for n, d in zip(("dx", "dw_gate", "dw_up"), v))
    assert abs(diff - along) <= bound + 1e-6 * abs(diff)
    # and as independent roundings, of which there are three (dg or du, x's gradient, the sum)
    rms = sum(((R.half(dt) * val[n]) * d).square().sum().item() for n, d in zip(("dx", "dw_gate", "dw_up"), v)) ** 0.5
    assert abs(diff - along) <= 6 * 3 * rms + 1e-6 * abs(diff)


def test_in_a_graph_and_on_another_stream():
    dt = torch.float16
    x, wg, wu, dh = problem(70, 144, 200, dt)
    ck = M.new_checkpoint(70, 144)
    h, h2, dx = torch.empty_like(dh), torch.empty_like(dh), torch.empty_like(x)
    a, b = torch.empty(200, 144, device="cuda"), torch.empty(200, 144, device="cuda")

    def step():
        M.checkpoint_save(x, ck)
        M.gated_ffn_forward(x, wg, wu, h)
        M.gated_ffn_backward(dh, ck, wg, wu, dx, a, b, h=h2)

    outs = (h, h2, dx, a, b)
    step()
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs, want))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    for n in range(4):
        x.copy_(torch.randn(70, 144, device="cuda"))
        graphs[n % 2].replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, outs))


# sizes with tiles of 64 and 128 rows, sums over k in one part and in several (test_gpu_ffn_cuts.py: every cut)
@pytest.mark.parametrize("t,k,f,dtype,act", [(70, 2600, 200, "f16", "silu"), (1500, 200, 130, "bf16", "silu"),
                                             (200, 130, 2100, "f16", "gelu"), (300, 264, 9000, "bf16", "gelu_tanh"),
                                             (2050, 264, 4100, "bf16", "silu"), (64, 1500, 1030, "f16", "silu"),
                                             (33, 520, 270, "bf16", "gelu"), (2500, 1100, 1300, "f16", "silu")])
def test_every_cut(t, k, f, dtype, act):
    dt = DT[dtype]
    x, wg, wu, dh = problem(t, k, f, dt, seed=t + k)
    val, err = R.ffn(x.cpu(), wg.cpu(), wu.cpu(), act, dh.cpu(), dt)
    buf, h = out(t, f, dt)
    M.gated_ffn_forward(x, wg, wu, h, act=act)
    assert untouched(buf, t, f)
    check(["h"], {"h": h}, val, err, dt)
    for wide in (False, True):
        bufs = {"h": out(t, f, dt), "dx": out(t, k, dt), "dw_gate": out(f, k, torch.float32 if wide else dt),
                "dw_up": out(f, k, torch.float32 if wide else dt)}
        got = {n: v[1] for n, v in bufs.items()}
        M.gated_ffn_backward(dh, x, wg, wu, got["dx"], got["dw_gate"], got["dw_up"], act=act, h=got["h"])
        for n, (buf, v) in bufs.items():
            assert untouched(buf, *v.shape), n
        check(["h", "dx", "dw_gate", "dw_up"], got, val, err, dt)
        if wide:  # the parts are joined in one order
            first = {n: v.clone() for n, v in got.items()}
            M.gated_ffn_backward(dh, x, wg, wu, got["dx"], got["dw_gate"], got["dw_up"], act=act, h=got["h"])
            assert all(torch.equal(first[n], got[n]) for n in got)


@pytest.mark.parametrize("tokens", [41, 300])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("act", list(M.ACTIVATIONS))
def test_activations_keep_their_digits_in_the_tails(act, dtype, tokens):
    """Gates from -8 to 6, each exact (x = [gate, 1], one inner unit that copies the gate and has u = 1), so that h
    and du are act(g), and dg is act'(g), with bounds relative to their values."""
    dt = DT[dtype]
    g = torch.linspace(-8, 6, tokens, dtype=torch.float64).to(dt)
    x = torch.stack([g, torch.ones_like(g)], 1).cuda()
    one = torch.tensor([[1.0, 0.0]], dtype=dt, device="cuda")
    up = torch.tensor([[0.0, 1.0]], dtype=dt, device="cuda")
    dh = torch.ones(tokens, 1, dtype=dt, device="cuda")
    h, h2, dx = torch.empty_like(dh), torch.empty_like(dh), torch.empty_like(x)
    dw = torch.empty(1, 2, device="cuda"), torch.empty(1, 2, device="cuda")
    M.gated_ffn_forward(x, one, up, h, act=act)
    M.gated_ffn_backward(dh, x, one, up, dx, *dw, act=act, h=h2)
    g = g.double()
    a, d, _ = R.act_parts(g, act)
    if act == "gelu":
        # phi: two roundings of erfc's argument z, to which its value is g^2 + 2 times as sensitive, and 16 units
        # (32 U) for erfc itself. The density: |g|^2 / 2 loses one rounding, the exponential 2 |argument| + 4.
        phi, slope = a.abs() / g.abs().clamp_min(1e-300), (d - torch.where(g == 0, 0.5, a / g)).abs()
        ea = (2 * (g * g + 2) + 36) * R.U * a.abs()
        ed = (2 * (g * g + 2) + 36) * R.U * phi + (2 * g * g + 16) * R.U * slope + R.U * d.abs()
    else:
        # s = 1 / (1 + e^-E): E is off by at most 4 U relative, the exponential by 2 |E| + 4, reciprocal and
        # products by a few more; both terms of the slope carry them, the second through s (1 - s)
        E = g.abs() if act == "silu" else 1.6 * (g + 0.044715 * g ** 3).abs()
        s = torch.where(g == 0, 0.5, a / g)
        ea = (8 * E + 40) * R.U * a.abs()
        ed = (8 * E + 40) * R.U * (s + (d - s).abs()) + 4 * R.U * g.abs() * s * (1 + g * g)
    for name, got, ref, err in (("h", h[:, 0], a, ea), ("h again", h2[:, 0], a, ea), ("du", dx[:, 1], a, ea),
                                ("dg", dx[:, 0], d, ed)):
        R.assert_near(got, ref, err, act + " " + name)


@pytest.mark.parametrize("dtype,gate,dh,want", [
    ("f16", 64.0, 2.0 ** 9, 2.0 ** 15), ("f16", 64.0, 2.0 ** 10, float("inf")),
    ("bf16", 64.0, 2.0 ** 10, 2.0 ** 16), ("bf16", 64.0, 2.0 ** -40, 2.0 ** -34),
    # silu(0.5) = 0.311: of the smallest float16 it leaves less than half, of four of them 1.24
    ("f16", 0.5, 2.0 ** -24, 0.0), ("f16", 0.5, 2.0 ** -22, 2.0 ** -24)])
def test_gradients_of_gate_and_up_have_the_range_of_their_type(dtype, gate, dh, want):
    """du = dh act(g) is rounded to the type before it is summed, here into a binary32 gradient of one token."""
    dt = DT[dtype]
    x = torch.tensor([[gate, 1.0]], dtype=dt, device="cuda")
    wg = torch.tensor([[1.0, 0.0]], dtype=dt, device="cuda")
    wu = torch.tensor([[0.0, 2.0 ** -14]], dtype=dt, device="cuda")
    a, b = torch.empty(1, 2, device="cuda"), torch.empty(1, 2, device="cuda")
    M.gated_ffn_backward(torch.full((1, 1), dh, dtype=dt, device="cuda"), x, wg, wu, torch.empty_like(x), a, b)
    assert b[0, 1].item() == want
