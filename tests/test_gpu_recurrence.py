"""The gated linear recurrence on the GPU, forward and backward, against the
binary64 reference (tests/model_ref.py), whose bounds carry the gates' and the
sums' roundings along the sequence."""
import pytest
import torch

import bit_adamw_optimizer_amd as M
from tests import model_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def cube(shape, dtype, seed, size=1.0, offset=0.0, pad=0, behind=0):
    """[batch, time, channels] with `pad` elements behind each step and `behind` steps behind each sequence."""
    b, t, c = shape
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((b, t + behind, c + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :t, :c] = (torch.randn(b, t, c, generator=g) * size + offset).to(dtype)
    return buf[:, :t, :c]


def out_like(x, pad=1):
    b, t, c = x.shape
    buf = torch.full((b, t + 1, c + pad), 7.0, dtype=x.dtype, device="cuda")
    return buf, buf[:, :t, :c]


def untouched(buf, shape, lengths=None):
    b, t, c = shape
    ok = (buf[:, t:] == 7).all() and (buf[:, :, c:] == 7).all()
    if lengths is not None:
        for i, n in enumerate(lengths.tolist()):
            ok = ok and (buf[i, min(max(n, 0), t):] == 7).all()
    return bool(ok)


def mask(shape, lengths):
    if lengths is None:
        return torch.ones(shape[0], shape[1], 1, dtype=torch.bool)
    return (torch.arange(shape[1])[None] < lengths.cpu().long()[:, None])[:, :, None]


def check(x, g, h0=None, lengths=None, dy=None, dh_last=None, states=True):
    """One forward and one backward pass against the reference; returns what they gave."""
    shape = x.shape
    b, t, c = shape
    n = None if lengths is None else lengths.cpu()
    yb, y = out_like(x)
    st = M.new_recurrence_states(b, t, c).fill_(7) if states else None
    h_last = torch.full((b, c), 7.0, device="cuda")
    M.recurrence_forward(x, g, y, h0=h0, h_last=h_last, states=st, lengths=lengths)
    assert untouched(yb, shape, n)
    hs, errs = R.recurrence_forward(x.cpu(), g.cpu(), None if h0 is None else h0.cpu(), n)
    live = mask(shape, n)
    y0 = torch.where(live, y.cpu().double(), hs[:, 1:])  # behind a length there is nothing to compare
    R.assert_near(y0.to(x.dtype) if x.dtype != torch.float32 else y0.float(), hs[:, 1:], errs[:, 1:], "y")
    R.assert_near(h_last, hs[:, -1], errs[:, -1], "h_last")
    if not states:
        return y, h_last
    kept = live[:, ::R.CHUNK].expand_as(st)
    R.assert_near(st.cpu()[kept], hs[:, :-1:R.CHUNK][kept], errs[:, :-1:R.CHUNK][kept], "states")
    assert (st.cpu()[~kept] == 7).all()
    dy = cube(shape, x.dtype, 99, 0.1) if dy is None else dy
    dxb, dx = out_like(x)
    dgb, dg = out_like(x, 3)
    dh0 = torch.full((b, c), 7.0, device="cuda")
    M.recurrence_backward(dy, x, g, st, dx, dg, dh_last=dh_last, dh0=dh0, lengths=lengths)
    assert untouched(dxb, shape, n) and untouched(dgb, shape, n)
    clean = [torch.where(live, v.cpu().double(), 0.0) for v in (dy, x, g, st.repeat_interleave(R.CHUNK, 1)[:, :t])]
    val, err = R.recurrence_backward(*clean[:3], clean[3][:, ::R.CHUNK], None if dh_last is None else dh_last.cpu(), n)
    for name, got in (("dx", dx), ("dgate", dg)):
        sel = live.expand(shape)
        R.assert_near(got.cpu()[sel], val[name][sel], err[name][sel], name)
    R.assert_near(dh0, val["dh0"], err["dh0"], "dh0")
    return y, h_last, st, dx, dg, dh0


SHAPES = [(1, 1, 1), (2, 1, 70), (3, 2, 5), (1, 31, 3), (2, 32, 64), (1, 33, 129), (2, 63, 7), (1, 64, 2), (3, 65, 66), (1, 127, 130),
          (2, 128, 1), (1, 129, 63), (2, 255, 40), (1, 256, 65), (1, 257, 5), (1, 511, 3), (2, 513, 9), (1, 1025, 67)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype):
    dt = DT[dtype]
    b, t, c = shape
    x, g = cube(shape, dt, 1, pad=2, behind=1), cube(shape, dt, 2, 2.0, 1.5, pad=0)
    check(x, g)
    gen = torch.Generator().manual_seed(3)
    h0, dl = (torch.randn(b, c, generator=gen).cuda() for _ in range(2))
    check(x, g, h0, dh_last=dl, dy=cube(shape, dt, 4, 0.1, pad=1))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(5, 70, 33), (4, 300, 66), (6, 40, 2), (3, 1200, 5)])
def test_lengths(shape, dtype):
    """From none to all steps, and numbers beyond both ends; NaN behind every length."""
    dt = DT[dtype]
    b, t, c = shape
    n = torch.tensor([0, 1, t, 33, -3, t + 5][:b] if b <= 6 else None)
    n[2 % b] = t // 2
    x, g, dy = cube(shape, dt, 1), cube(shape, dt, 2, 2.0, 2.0), cube(shape, dt, 3, 0.1)
    for i, k in enumerate(n.tolist()):
        for v in (x, g, dy):
            v[i, max(k, 0):] = float("nan")
    gen = torch.Generator().manual_seed(4)
    h0, dl = (torch.randn(b, c, generator=gen).cuda() for _ in range(2))
    r64 = check(x, g, h0, n.cuda(), dy, dl)
    r32 = check(x, g, h0, n.int().cuda(), dy, dl)
    assert all(torch.equal(p.nan_to_num(), q.nan_to_num()) for p, q in zip(r64, r32))
    assert torch.equal(r64[1][0], h0[0]) and torch.equal(r64[5][0], dl[0])  # a sequence of no steps


@pytest.mark.parametrize("shape", [(1, 20000, 6), (1, 9001, 70), (2, 5000, 200), (3, 2600, 64)])
def test_long_sequences_of_few_channels(shape):
    """Gates that remember from one step to thousands."""
    b, t, c = shape
    x = cube(shape, torch.float32, 1)
    memory = torch.linspace(-1, 9, c).cuda()
    g = cube(shape, torch.float32, 2) + memory
    gen = torch.Generator().manual_seed(3)
    h0, dl = (torch.randn(b, c, generator=gen).cuda() for _ in range(2))
    got = check(x, g, h0, dh_last=dl)
    again = check(x, g, h0, dh_last=dl)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    n = torch.tensor([t - 1, t // 3, 17][:b], device="cuda")
    check(x, g, h0, n, dh_last=dl)


@pytest.mark.parametrize("dtype", list(DT))
def test_open_and_closed_gates(dtype):
    """Gates so far from 0 that one of a, 1 - a has no digits beside the other, and infinite ones."""
    dt = DT[dtype]
    shape = (2, 100, 12)
    x, g = cube(shape, dt, 1), cube(shape, dt, 2)
    g[..., 0], g[..., 1], g[..., 2], g[..., 3] = 20.0, -20.0, 300.0, -300.0
    g[..., 4], g[..., 5] = float("inf"), float("-inf")
    g[:, ::2, 6], g[:, 1::2, 6] = 12.0, -12.0
    y, h_last, *_ = check(x, g, torch.ones(2, 12, device="cuda"))
    assert (y[..., 4] == 1).all() and torch.equal(y[..., 5], x[..., 5])


def test_nan_stays_in_its_channel_and_sequence():
    shape = (3, 200, 10)
    x, g = cube(shape, torch.float32, 1), cube(shape, torch.float32, 2, offset=2)
    y0, h0, st0, dx0, dg0, dh0 = check(x, g)
    x[1, 50, 3] = float("nan")
    y = torch.empty_like(x)
    st = M.new_recurrence_states(*shape)
    M.recurrence_forward(x, g, y, states=st)
    bad = torch.isnan(y)
    assert bad[1, 50:, 3].all() and bad.sum() == 150
    assert torch.equal(y[~bad], y0[~bad])
    dy, dx, dg = cube(shape, torch.float32, 99, 0.1), torch.empty_like(x), torch.empty_like(x)
    M.recurrence_backward(dy, x, g, st, dx, dg)
    assert torch.equal(dx, dx0) and torch.isnan(dg[1, 50:, 3]).all() and torch.isnan(dg).sum() == 150


def test_layouts_in_place_and_repeated_inputs():
    B, T, C = 3, 140, 48
    f = torch.float16
    gen = torch.Generator().manual_seed(1)
    p = (torch.randn(B, T, 2 * C, generator=gen) + 0.5).to(f).cuda()
    x, g = p[..., :C], p[..., C:]  # halves of one projection's output
    y, h, st, dx, dg, dh0 = check(x, g)
    # time-major
    pt = p.transpose(0, 1).contiguous().transpose(0, 1)
    yt, st2 = torch.empty(T, B, C, dtype=f, device="cuda").transpose(0, 1), torch.empty_like(st)
    M.recurrence_forward(pt[..., :C], pt[..., C:], yt, states=st2)
    assert torch.equal(yt, y) and torch.equal(st, st2)
    dy = cube((B, T, C), f, 99, 0.1)
    dp = torch.empty_like(pt)
    M.recurrence_backward(dy, pt[..., :C], pt[..., C:], st, dp[..., :C], dp[..., C:])
    assert torch.equal(dp[..., :C], dx) and torch.equal(dp[..., C:], dg)
    # outputs over inputs
    for k in (0, C):
        q = p.clone()
        M.recurrence_forward(q[..., :C], q[..., C:], q[..., k:k + C])
        assert torch.equal(q[..., k:k + C], y)
    q = p.clone()
    M.recurrence_backward(dy, q[..., :C], q[..., C:], st, q[..., :C], q[..., C:])
    assert torch.equal(q[..., :C], dx) and torch.equal(q[..., C:], dg)
    q, d = p.clone(), dy.clone()
    M.recurrence_backward(d, q[..., :C], q[..., C:], st, q[..., C:], d)
    assert torch.equal(q[..., C:], dx) and torch.equal(d, dg)
    # one step's gate for all steps, one sequence's input for all sequences
    one, wide = g[:, :1].expand(B, T, C), x[:1].expand(B, T, C)
    ya, yb = torch.empty_like(y), torch.empty_like(y)
    M.recurrence_forward(wide, one, ya)
    M.recurrence_forward(wide.contiguous(), one.contiguous(), yb)
    assert torch.equal(ya, yb)


def test_tokens_one_at_a_time_give_the_sequence():
    """The state in place from call to call: within the roundings of whole sequences (float32 here)."""
    B, T, C = 5, 40, 77
    x, g = cube((B, T, C), torch.float32, 1), cube((B, T, C), torch.float32, 2, offset=1)
    hs, errs = R.recurrence_forward(x.cpu(), g.cpu())
    h = torch.zeros(B, C, device="cuda")
    y = torch.empty_like(x)
    for t in range(T):
        M.recurrence_forward(x[:, t:t + 1], g[:, t:t + 1], y[:, t:t + 1], h0=h, h_last=h)
    R.assert_near(y, hs[:, 1:], errs[:, 1:], "y")
    assert torch.equal(h, y[:, -1])
    # a finished sequence's state stays as it is
    before, n = h.clone(), torch.tensor([1, 0, 1, 0, 1], device="cuda")
    M.recurrence_forward(x[:, :1], g[:, :1], y[:, :1], h0=h, h_last=h, lengths=n)
    assert torch.equal(h[n == 0], before[n == 0]) and not torch.equal(h[n == 1], before[n == 1])


def test_sequences_in_two_calls():
    """The second half from the first one's last state; its gradient through dh_last and dh0."""
    B, T, C = 2, 320, 70
    x, g, dy = (cube((B, T, C), torch.float32, i, offset=i % 2) for i in (1, 2, 3))
    hs, errs = R.recurrence_forward(x.cpu(), g.cpu())
    h, y, cut = torch.zeros(B, C, device="cuda"), torch.empty_like(x), 160
    st = [M.new_recurrence_states(B, cut, C) for _ in range(2)]
    parts = [slice(0, cut), slice(cut, T)]
    for p, s in zip(parts, st):
        M.recurrence_forward(x[:, p], g[:, p], y[:, p], h0=h, h_last=h, states=s)
    R.assert_near(y, hs[:, 1:], errs[:, 1:], "y")
    dx, dg, d = torch.empty_like(x), torch.empty_like(x), torch.zeros(B, C, device="cuda")
    for p, s in reversed(list(zip(parts, st))):
        M.recurrence_backward(dy[:, p], x[:, p], g[:, p], s, dx[:, p], dg[:, p], dh_last=d, dh0=d)
    val, err = R.recurrence_backward(dy.cpu(), x.cpu(), g.cpu(), torch.cat(st, 1).cpu())
    for name, got in (("dx", dx), ("dgate", dg), ("dh0", d)):
        R.assert_near(got, val[name], err[name], name)


@pytest.mark.parametrize("shape", [(2, 5000, 70), (1, 9001, 600)])
def test_states_in_place_of_sequences_in_spans(shape):
    """The last state over the first one while other spans still start from it."""
    b, t, c = shape
    x, g, dy = (cube(shape, torch.float16, i, offset=i % 2) for i in (1, 2, 3))
    h0 = torch.linspace(-3, 3, b * c).view(b, c).cuda()
    y, y2, st = torch.empty_like(x), torch.empty_like(x), M.new_recurrence_states(*shape)
    last, h = torch.empty_like(h0), h0.clone()
    M.recurrence_forward(x, g, y, h0=h0, h_last=last, states=st)
    M.recurrence_forward(x, g, y2, h0=h, h_last=h)
    assert torch.equal(h, last) and torch.equal(y, y2)
    outs = [torch.empty_like(x) for _ in range(4)]
    dh0, d = torch.empty_like(h0), h0.clone()
    M.recurrence_backward(dy, x, g, st, outs[0], outs[1], dh_last=h0, dh0=dh0)
    M.recurrence_backward(dy, x, g, st, outs[2], outs[3], dh_last=d, dh0=d)
    assert torch.equal(d, dh0) and torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("channels", [1, 3, 63, 65, 127, 129])
def test_odd_channels_in_place(channels, dtype):
    """The last channel's lane reads its neighbour's too, and writes its own alone."""
    shape = (2, 300, channels)
    x, g = cube(shape, DT[dtype], 1, pad=1), cube(shape, DT[dtype], 2)
    y = torch.empty(shape, dtype=DT[dtype], device="cuda")
    M.recurrence_forward(x, g, y)
    M.recurrence_forward(x, g, x)
    assert torch.equal(x, y)


def test_empty_sizes():
    h0 = torch.ones(2, 3, device="cuda")
    h = torch.zeros(2, 3, device="cuda")
    none = torch.empty(2, 0, 3, device="cuda")
    M.recurrence_forward(none, none, none, h0=h0, h_last=h)
    assert torch.equal(h, h0)
    d = torch.zeros(2, 3, device="cuda")
    M.recurrence_backward(none, none, none, M.new_recurrence_states(2, 0, 3), none, none, dh_last=h0, dh0=d)
    assert torch.equal(d, h0)
    M.recurrence_backward(none, none, none, M.new_recurrence_states(2, 0, 3), none, none, dh0=d)
    assert not d.any()
    for shape in ((0, 4, 3), (2, 4, 0)):
        e = torch.empty(shape, device="cuda")
        M.recurrence_forward(e, e, torch.empty(shape, device="cuda"), states=M.new_recurrence_states(*shape))


def test_offsets_beyond_32_bits():
    """The last of many sequences of a tensor of more than 2^31 elements."""
    B, T, C = 2, 17000, 66000
    x = torch.zeros(B, T, C, dtype=torch.float16, device="cuda")
    assert x.numel() > 1 << 31
    x[:, :, -40:] = 1.0
    y = torch.empty_like(x)
    st = torch.empty(B, -(-T // 32), C, device="cuda")
    M.recurrence_forward(x, x, y, states=st)
    tail = x[:, :, -40:].contiguous()
    yt, stt = torch.empty_like(tail), torch.empty(B, -(-T // 32), 40, device="cuda")
    M.recurrence_forward(tail, tail, yt, states=stt)
    # the same to within the order of the joined spans: h climbs from 0 to 1
    assert (y[:, :, -40:].float() - yt.float()).abs().max() <= 2 * 2 ** -11 and not y[:, :, :100].any()
    M.recurrence_backward(x, x, x, st, y, x)  # dgate over x, in place
    dxt, dgt = torch.empty_like(tail), torch.empty_like(tail)
    M.recurrence_backward(tail, tail, tail, stt, dxt, dgt)
    assert (y[:, :, -40:].float() - dxt.float()).abs().max() <= 2 * 2 ** -11
    assert (x[:, :, -40:].float() - dgt.float()).abs().max() <= 2 * 2 ** -11


@pytest.mark.parametrize("shape", [(3, 1, 130), (2, 700, 40)])
def test_another_stream_and_replays(shape):
    b, t, c = shape
    x, g, dy = (cube(shape, torch.bfloat16, i) for i in (1, 2, 3))
    h0 = torch.ones(b, c, device="cuda")

    def outputs():
        return [torch.zeros_like(x) for _ in range(3)] + [M.new_recurrence_states(b, t, c), torch.zeros_like(h0)]

    def go(o):
        M.recurrence_forward(x, g, o[0], h0=h0, states=o[3])
        M.recurrence_backward(dy, x, g, o[3], o[1], o[2], dh_last=h0, dh0=o[4])

    want = outputs()
    go(want)
    other = outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(other)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(want, other))
    runs = []
    for _ in range(2):
        o, graph = outputs(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go(o)
        runs.append((graph, o))
    for _ in range(3):
        for _, o in runs:
            for v in o:
                v.fill_(5)
        for graph, _ in runs:
            graph.replay()
        torch.cuda.synchronize()
        for _, o in runs:
            assert all(torch.equal(p, q) for p, q in zip(want, o))
        go(other)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(2, 3, 6), (2, 33, 10), (3, 100, 33), (2, 300, 40), (1, 9001, 6)])
def test_backward_from_repeated_and_overlapping_steps(shape, dtype):
    """Gradients of a sum over time (one dy for all steps), inputs repeated over time or sequences, and steps that
    share elements, with and without lengths: what is behind the last step is not added again."""
    b, t, c = shape
    dt = DT[dtype]
    full = [cube(shape, dt, i, 0.5, offset=i % 2) for i in (1, 2, 3)]
    gen = torch.Generator().manual_seed(4)
    h0, dl = (torch.randn(b, c, generator=gen).cuda() for _ in range(2))
    shifted = cube((1, 1, b * c + 3 * t), dt, 5, 0.5).as_strided(shape, (c, 3, 1))
    for n in (None, torch.tensor([t - 1, t // 2 + 1, 1][:b], device="cuda")):
        check(full[0], full[1], h0, n, full[2][:, :1].expand(shape), dl)
        check(shifted, shifted, h0, n, shifted, dl)
        for i in range(3) if t < 1000 else ():
            args = [shifted if j == i else full[j] for j in range(3)]
            check(args[0], args[1], h0, n, args[2], dl)
        for which in (0, 1, 2, None):
            for v in ([p[:, :1].expand(shape) for p in full], [p[:1].expand(shape) for p in full]):
                args = [v[i] if which in (i, None) else full[i] for i in range(3)]
                outs = []
                for x, g, dy in (args, [p.contiguous() for p in args]):
                    st, y = M.new_recurrence_states(*shape).fill_(7), torch.full(shape, 7.0, dtype=dt, device="cuda")
                    M.recurrence_forward(x, g, y, h0=h0, states=st, lengths=n)
                    dx, dg, dh0 = torch.full_like(y, 7.0), torch.full_like(y, 7.0), torch.full_like(h0, 7.0)
                    M.recurrence_backward(dy, x, g, st, dx, dg, dh_last=dl, dh0=dh0, lengths=n)
                    outs.append((y, st, dx, dg, dh0))
                assert all(torch.equal(p, q) for p, q in zip(*outs)), (which, n)


def test_the_gradient_of_a_mean_over_time():
    """Open gates (a = 1/2) and dy = 1: l_t = 2 - 2^-(T - 1 - t), so that dx at the last step is 1/2."""
    for t in (33, 100, 300):
        x = torch.zeros(1, t, 2, device="cuda")
        dy, dx, dg = torch.ones(1, 1, 2, device="cuda").expand(1, t, 2), torch.empty_like(x), torch.empty_like(x)
        M.recurrence_backward(dy, x, x, M.new_recurrence_states(1, t, 2).zero_(), dx, dg)
        want = 1 - 0.5 ** (t - torch.arange(t, dtype=torch.float64))
        R.assert_near(dx[0, :, 0], want, 16 * R.U * want, "dx")


@pytest.mark.parametrize("pad", [0, 5])
def test_parts_of_one_buffer_that_are_apart(pad):
    """Time halves, and column halves of sequences that start anywhere: inputs and outputs share no element."""
    B, T, C = 3, 70, 24
    x, g, dy = (cube((B, T, C), torch.float32, i, offset=i % 2) for i in (1, 2, 3))
    y, st, dx, dg = torch.empty_like(x), M.new_recurrence_states(B, T, C), torch.empty_like(x), torch.empty_like(x)
    M.recurrence_forward(x, g, y, states=st)
    M.recurrence_backward(dy, x, g, st, dx, dg)
    for make in (lambda: torch.zeros(B, 2 * T * C + pad, device="cuda")[:, :2 * T * C].view(B, 2 * T, C).split(T, 1),
                 lambda: torch.zeros(B, 2 * T * C + pad, device="cuda")[:, :2 * T * C].view(B, T, 2 * C).split(C, 2),
                 lambda: torch.zeros(T, 2 * B * C + pad, device="cuda")[:, :2 * B * C].view(T, 2 * B, C).transpose(0, 1).split(B)):
        for src in (x, g):
            a, b = make()
            a.copy_(src)
            M.recurrence_forward(a if src is x else x, a if src is g else g, b)
            assert torch.equal(b, y) and torch.equal(a, src)
        a, b = make()
        M.recurrence_backward(dy, x, g, st, a, b)
        assert torch.equal(a, dx) and torch.equal(b, dg)


def test_the_largest_number_of_sequences():
    """2^22 sequences of 33 binary32 channels, in place: 2^23 workgroups."""
    B, T, C = 1 << 22, 129, 33
    g = cube((1, T, C), torch.float32, 1, offset=2.0)
    first, last = cube((1, T, C), torch.float32, 2), cube((1, T, C), torch.float32, 3)
    x = torch.ones(B, T, C, device="cuda")
    x[0], x[-1] = first[0], last[0]
    M.recurrence_forward(x, g.expand(B, T, C), x)
    y = torch.empty(3, T, C, device="cuda")
    M.recurrence_forward(torch.cat([first, torch.ones_like(first), last]), g.expand(3, T, C), y)
    # fewer waves side by side join their steps in another order: both within the bound
    for i, (at, v) in enumerate(((0, first), (B // 2 + 1, torch.ones_like(first)), (B - 1, last))):
        hs, errs = R.recurrence_forward(v.cpu(), g.cpu())
        R.assert_near(x[at:at + 1], hs[:, 1:], errs[:, 1:], "y")
        R.assert_near(y[i:i + 1], hs[:, 1:], errs[:, 1:], "y of three")
    assert torch.equal(x[1], x[B // 2 + 1]) and (x[1:-1].amax(0) == x[1]).all() and (x[1:-1].amin(0) == x[1]).all()


@pytest.mark.parametrize("time", [1, 17])
def test_every_gate_keeps_its_digits(time):
    """y = 1 - a from x = 1 and no state, and y = a from h0 = 1 and x = 0. e^-|g| comes from a power of 2 (two units of
    U), its product with what the exponent's rounding left (one), ln 2's own rounding (|g| U / 21); 1 + e, a reciprocal
    and a product (four) follow. The larger of the two is 1 less the smaller."""
    g = torch.cat([torch.linspace(-86, 86, 4001), torch.linspace(-1, 1, 1001)])[None, None].cuda()
    want = torch.sigmoid(-g.double())
    bound = (8 + g.double().abs() / 16) * R.U * torch.minimum(want, 1 - want) + torch.where(want > 0.5, R.U / 2, 0.0)
    shape = (1, time, g.shape[2])
    one = (torch.arange(time, device="cuda") == 0)[None, :, None].expand(shape)
    open_behind = torch.where(one, g, torch.full_like(g, 200.0)).contiguous()  # the later steps keep the state
    x, y = torch.where(one, 1.0, 0.0).contiguous(), torch.empty(shape, device="cuda")
    M.recurrence_forward(x, open_behind, y)
    assert ((y[:, -1:].double() - want).abs() <= bound).all()
    M.recurrence_forward(torch.zeros_like(x), torch.where(one, -g, open_behind).contiguous(), y, h0=torch.ones(1, shape[2], device="cuda"))
    assert ((y[:, -1:].double() - want).abs() <= bound).all()
