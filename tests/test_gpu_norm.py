"""Layer norm and RMS norm on the GPU, forward and backward, from matrices and
from 8-bit checkpoints, against the binary64 reference (tests/train_ref.py).
Tolerances are one rounding to the output type plus the bound of the binary32
arithmetic that the reference derives."""
import pytest
import torch

import bit_adamw_optimizer_amd as M
from tests import train_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
SHAPES = [(1, 1, 0), (2, 7, 0), (5, 64, 0), (9, 513, 1), (6, 768, 0), (3, 1000, 8), (4, 1025, 0), (5, 2048, 0),
          (3, 2049, 3), (2, 4096, 0), (3, 5120, 0), (2, 8200, 0), (2, 16385, 0), (1, 32768, 0)]


def matrix(rows, cols, dtype, pad, seed, size=1.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * size + offset
    buf = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = x.to(dtype)
    return buf[:, :cols]


def weights(cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.2 * torch.randn(cols, generator=g)).to(dtype).cuda(), (0.3 * torch.randn(cols, generator=g)).to(dtype).cuda())


def forward(x, w, b, centered, save=None, like=None):
    like = x if like is None else like
    rows, cols = like.shape
    y = torch.full((rows + 1, cols + 1), 7.0, dtype=like.dtype, device="cuda")
    mean = torch.empty(rows, device="cuda") if centered else None
    rstd = torch.empty(rows, device="cuda")
    M.layernorm_forward(x, w, b, y[:rows, :cols], mean, rstd, eps=EPS, save=save)
    assert (y[rows:] == 7).all() and (y[:, cols:] == 7).all()
    return y[:rows, :cols], mean, rstd


def check_forward(x, w, b, centered, y, mean, rstd):
    ones = torch.ones(x.shape[1], dtype=torch.float64)
    ry, rmu, rrs, bound = R.norm_forward(x.cpu(), ones if w is None else w.cpu().double(),
                                         None if b is None else b.cpu().double(), EPS, centered)
    R.assert_near(y, ry, bound, "y")
    if centered:
        R.assert_near(mean, rmu, 128 * R.U * x.cpu().double().abs().mean(1), "mean")
    # the variance's relative error is at most 128 steps, of which the square root halves; the mean's
    # error enters it squared
    R.assert_near(rstd, rrs, 128 * R.U * rrs, "rstd")


def backward(dy, x, w, mean, rstd, accumulate=False, dw=None, db=None):
    rows, cols = dy.shape
    dx = torch.full((rows + 1, cols + 1), 7.0, dtype=dy.dtype, device="cuda")
    dw = torch.full((cols,), 7.0, device="cuda") if dw is None else dw
    db = torch.full((cols,), 7.0, device="cuda") if db is None else db
    M.layernorm_backward(dy, x, w, mean, rstd, dx[:rows, :cols], dw, db, accumulate=accumulate)
    assert (dx[rows:] == 7).all() and (dx[:, cols:] == 7).all()
    return dx[:rows, :cols], dw, db


def check_backward(dy, x, w, mean, rstd, got):
    ones = torch.ones(dy.shape[1], dtype=torch.float64)
    ref = R.norm_backward(dy.cpu(), x.cpu(), ones if w is None else w.cpu().double(),
                          None if mean is None else mean.cpu(), rstd.cpu(), mean is not None)
    for name, g, r, e in zip(("dx", "dweight", "dbias"), got, ref[:3], ref[3:]):
        R.assert_near(g, r, e, name)


@pytest.mark.parametrize("centered", [True, False])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_forward_and_backward(rows, cols, pad, dtype, centered):
    dt = DT[dtype]
    x = matrix(rows, cols, dt, pad, seed=cols, size=2.0, offset=0.5)
    w, b = weights(cols, dt, seed=cols + 1)
    y, mean, rstd = forward(x, w, b if centered else None, centered)
    check_forward(x, w, b if centered else None, centered, y, mean, rstd)
    dy = matrix(rows, cols, dt, pad, seed=cols + 2, size=0.1)
    check_backward(dy, x, w, mean, rstd, backward(dy, x, w, mean, rstd))


@pytest.mark.parametrize("fmt", [M.E4M3, M.E5M2])
@pytest.mark.parametrize("centered", [True, False])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", [(5, 33), (7, 768), (2, 1001), (3, 4096), (2, 8224)])
def test_through_checkpoints(rows, cols, dtype, centered, fmt):
    """The forward pass saves its input; forward again and backward read it."""
    dt = DT[dtype]
    x = matrix(rows, cols, dt, 0, seed=cols, offset=0.2)
    w, b = weights(cols, torch.float32, seed=cols + 1)
    plain, saved = M.new_checkpoint(rows, cols, fmt), M.new_checkpoint(rows, cols, fmt)
    M.checkpoint_save(x, plain)
    y, mean, rstd = forward(x, w, b, centered, save=saved)
    check_forward(x, w, b, centered, y, mean, rstd)
    assert torch.equal(saved.codes[:, :cols], plain.codes[:, :cols]) and torch.equal(saved.scales, plain.scales)
    xv = torch.empty(rows, cols, device="cuda")
    M.checkpoint_load(saved, xv)
    dy = matrix(rows, cols, dt, 0, seed=cols + 2, size=0.1)
    check_backward(dy, xv, w, mean, rstd, backward(dy, saved, w, mean, rstd))
    y2, mean2, rstd2 = forward(saved, w, b, centered, like=x)
    check_forward(xv, w, b, centered, y2, mean2, rstd2)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols,pad", [(1, 128, 0), (33, 127, 1), (1000, 64, 0), (257, 33, 0), (15, 8, 8), (700, 129, 0),
                                           (50, 256, 0), (2, 255, 3), (1234, 200, 0)])
def test_short_rows(rows, cols, pad, dtype):
    """Several rows to a wave (up to 128 and 256 columns), numbers of rows that fill no workgroup."""
    dt = DT[dtype]
    x, dy = matrix(rows, cols, dt, pad, 1, offset=0.3), matrix(rows, cols, dt, pad, 2, size=0.1)
    w, b = weights(cols, dt, 3)
    for centered in (True, False):
        ck = M.new_checkpoint(rows, cols)
        y, mean, rstd = forward(x, w, b if centered else None, centered, save=ck)
        check_forward(x, w, b if centered else None, centered, y, mean, rstd)
        check_backward(dy, x, w, mean, rstd, backward(dy, x, w, mean, rstd))
        xv = torch.empty(rows, cols, device="cuda")
        M.checkpoint_load(ck, xv)
        check_backward(dy, xv, w, mean, rstd, backward(dy, ck, w, mean, rstd))


def test_no_weight_no_bias_and_one_gradient():
    x, dy = matrix(37, 300, torch.float16, 0, 1), matrix(37, 300, torch.float16, 0, 2)
    y, mean, rstd = forward(x, None, None, True)
    check_forward(x, None, None, True, y, mean, rstd)
    full = backward(dy, x, None, mean, rstd)
    check_backward(dy, x, None, mean, rstd, full)
    dx, dw, db = torch.empty_like(dy), torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    M.layernorm_backward(dy, x, None, mean, rstd, dx, dw, None)
    assert torch.equal(dx, full[0]) and torch.equal(dw, full[1])
    M.layernorm_backward(dy, x, None, mean, rstd, dx, None, db)
    assert torch.equal(dx, full[0]) and torch.equal(db, full[2])
    M.layernorm_backward(dy, x, None, mean, rstd, dx, None, None)
    assert torch.equal(dx, full[0])


@pytest.mark.parametrize("rows,cols", [(3000, 96), (1500, 1030), (700, 5000)])
def test_many_rows_accumulate_and_repeat(rows, cols):
    x, dy = matrix(rows, cols, torch.bfloat16, 0, 1, offset=1.0), matrix(rows, cols, torch.bfloat16, 0, 2)
    w, _ = weights(cols, torch.bfloat16, 3)
    _, mean, rstd = forward(x, w, None, True)
    first = backward(dy, x, w, mean, rstd)
    check_backward(dy, x, w, mean, rstd, first)
    again = backward(dy, x, w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(first, again))  # the same sums in the same order
    dw, db = torch.full((cols,), 2.0, device="cuda"), torch.full((cols,), -3.0, device="cuda")
    _, dw2, db2 = backward(dy, x, w, mean, rstd, True, dw, db)
    assert torch.equal(dw2, 2.0 + first[1]) and torch.equal(db2, -3.0 + first[2])


@pytest.mark.parametrize("rows,cols", [(1, 40), (20, 128), (4, 2048), (2, 4096), (1, 9000), (1, 20001)])
def test_one_workgroup_accumulates(rows, cols):
    x, dy = matrix(rows, cols, torch.float16, 0, 1, offset=1.0), matrix(rows, cols, torch.float16, 0, 2)
    w, _ = weights(cols, torch.float16, 3)
    _, mean, rstd = forward(x, w, None, True)
    first = backward(dy, x, w, mean, rstd)
    check_backward(dy, x, w, mean, rstd, first)
    dw, db = torch.full((cols,), 2.0, device="cuda"), torch.full((cols,), -3.0, device="cuda")
    _, dw2, db2 = backward(dy, x, w, mean, rstd, True, dw, db)
    assert torch.equal(dw2, 2.0 + first[1]) and torch.equal(db2, -3.0 + first[2])


@pytest.mark.parametrize("rows,cols", [(128, 64), (129, 64), (64, 250), (65, 250), (32, 500), (33, 500), (16, 768), (17, 768),
                                       (8, 2048), (9, 2048), (4, 4095), (5, 4095), (2, 8192), (3, 8192), (2, 20000)])
@pytest.mark.parametrize("ckpt", [False, True])
def test_on_both_sides_of_one_workgroup(rows, cols, ckpt):
    """Several turns of one workgroup, and the fewest rows that several share."""
    x, dy = matrix(rows, cols, torch.bfloat16, 0, 1, offset=0.5), matrix(rows, cols, torch.bfloat16, 0, 2, size=0.1)
    w, _ = weights(cols, torch.bfloat16, 3)
    ck = M.new_checkpoint(rows, cols)
    _, mean, rstd = forward(x, w, None, True, save=ck)
    if ckpt:
        x = torch.empty(rows, cols, device="cuda")
        M.checkpoint_load(ck, x)
    first = backward(dy, ck if ckpt else x, w, mean, rstd)
    check_backward(dy, x, w, mean, rstd, first)
    dw, db = torch.full((cols,), 2.0, device="cuda"), torch.full((cols,), -3.0, device="cuda")
    _, dw2, db2 = backward(dy, ck if ckpt else x, w, mean, rstd, True, dw, db)
    assert torch.equal(dw2, 2.0 + first[1]) and torch.equal(db2, -3.0 + first[2])


def test_empty_calls():
    dw, db = torch.full((40,), 7.0, device="cuda"), torch.full((40,), 7.0, device="cuda")
    none, r = torch.empty(0, 40, device="cuda"), torch.empty(0, device="cuda")
    M.layernorm_forward(none, dw, db, none, r, r)
    M.layernorm_backward(none, none, dw, r, r, none, dw, db, accumulate=True)
    assert (dw == 7).all() and (db == 7).all()
    M.layernorm_backward(none, none, None, r, r, none, dw, db)
    assert not dw.any() and not db.any()
    e, r = torch.empty(3, 0, device="cuda"), torch.empty(3, device="cuda")
    M.layernorm_forward(e, None, None, e, r, r)
    M.layernorm_backward(e, e, None, r, r, e, torch.empty(0, device="cuda"), None)


def test_special_values_stay_in_their_row():
    x = matrix(8, 700, torch.float32, 0, 1)
    clean, mean, rstd = forward(x, None, None, True)
    dy = matrix(8, 700, torch.float32, 0, 2)
    ref = backward(dy, x, None, mean, rstd)[0].clone()
    bad = x.clone()
    bad[2, 5], bad[4, 699], bad[6] = float("inf"), float("nan"), torch.finfo(torch.float32).max
    y, mean, rstd = forward(bad, None, None, True)
    keep = [0, 1, 3, 5, 7]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[2]).any() and torch.isnan(y[4]).all()
    dx = backward(dy, bad, None, mean, rstd)[0]
    assert torch.equal(dx[keep], ref[keep])


def test_constant_rows_and_large_offsets():
    """A variance far below the mean: taken around the mean, it keeps its digits."""
    x = torch.full((4, 1024), 1000.0, device="cuda")
    y, mean, rstd = forward(x, None, None, True)
    assert (mean == 1000).all() and not y.any()
    R.assert_near(rstd, torch.full((4,), EPS ** -0.5, dtype=torch.float64), torch.full((4,), 4 * R.U * EPS ** -0.5, dtype=torch.float64), "rstd")
    x = 1000 + 0.125 * torch.randint(-8, 9, (4, 1024), generator=torch.Generator().manual_seed(1)).float().cuda()
    y, mean, rstd = forward(x, None, None, True)
    check_forward(x, None, None, True, y, mean, rstd)


def test_repeated_rows_and_refusals():
    row, dy = torch.randn(1, 50, device="cuda"), torch.randn(4, 50, device="cuda")
    y, mean, rstd = forward(row.expand(4, 50), None, None, True)
    assert torch.equal(y, y[:1].expand(4, 50))
    got = backward(dy[:1].expand(4, 50), row.expand(4, 50), None, mean, rstd)
    check_backward(dy[:1].expand(4, 50), row.expand(4, 50), None, mean, rstd, got)
    r4 = torch.empty(4, device="cuda")
    with pytest.raises(ValueError):
        M.layernorm_forward(dy, None, None, row.expand(4, 50), None, r4)
    with pytest.raises(ValueError):
        M.layernorm_forward(dy, torch.ones(49, device="cuda"), None, dy, None, r4)
    with pytest.raises(TypeError):
        M.layernorm_forward(dy, torch.ones(50, device="cuda").half(), None, dy, None, r4)
    with pytest.raises(TypeError):
        M.layernorm_forward(dy.half(), None, None, dy, None, r4)
    with pytest.raises(ValueError):
        M.layernorm_forward(dy, None, None, dy, None, torch.empty(8, device="cuda")[::2])
    with pytest.raises(M.MsampError):
        big = torch.empty(1, 32769, device="cuda")
        M.layernorm_forward(big, None, None, big, None, r4[:1])
    with pytest.raises(M.MsampError):
        M.layernorm_forward(dy, None, None, dy, None, r4, eps=-1.0)


def test_more_rows_than_one_launch_takes():
    """2^22 wide rows: a launch of all of them would have 2^32 threads."""
    rows, cols = (1 << 22) + 5, 8200
    if torch.cuda.mem_get_info()[0] < rows * cols * 2 * 1.2:
        pytest.skip("needs 83 GB of GPU memory")
    row = matrix(1, cols, torch.float16, 0, 1)
    y = torch.empty(rows, cols, dtype=torch.float16, device="cuda")
    rstd = torch.zeros(rows, device="cuda")
    M.layernorm_forward(row.expand(rows, cols), None, None, y, None, rstd)
    one, r = torch.empty_like(row), torch.empty(1, device="cuda")
    M.layernorm_forward(row, None, None, one, None, r)
    assert (rstd == r).all()
    for at in (0, (1 << 21) - 2, (1 << 22) - 2, rows - 4):
        assert torch.equal(y[at:at + 4], one.expand(4, cols))
    del y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols,pad", [(300, 40, 0), (1000, 200, 3), (700, 513, 1), (600, 1030, 0), (530, 4096, 0), (300, 9001, 0)])
def test_in_place(rows, cols, pad, dtype):
    """y in x's place, dx in dy's and in x's: the bits of a call with outputs of their own."""
    dt = DT[dtype]
    x, dy = matrix(rows, cols, dt, pad, 1, offset=0.5), matrix(rows, cols, dt, pad, 2, size=0.1)
    w, b = weights(cols, dt, 3)
    y, mean, rstd = forward(x, w, b, True)
    ref = backward(dy, x, w, mean, rstd)

    def copy(t):
        buf = torch.full((rows, cols + pad), 7.0, dtype=dt, device="cuda")
        buf[:, :cols] = t
        return buf, buf[:, :cols]

    buf, at = copy(x)
    M.layernorm_forward(at, w, b, at, mean, rstd, eps=EPS)
    assert torch.equal(at, y) and (buf[:, cols:] == 7).all()
    for over in ("dy", "x"):
        buf, at = copy(dy if over == "dy" else x)
        dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        M.layernorm_backward(at if over == "dy" else dy, at if over == "x" else x, w, mean, rstd, at, dw, db)
        assert torch.equal(at, ref[0]) and torch.equal(dw, ref[1]) and torch.equal(db, ref[2])
        assert (buf[:, cols:] == 7).all()


def test_columns_of_one_buffer():
    """Input and output side by side in the rows of one buffer, the statistics behind them."""
    buf = torch.zeros(64, 80, device="cuda")
    x = matrix(64, 32, torch.float32, 0, 1)
    buf[:, 4:36] = x
    rstd = torch.empty(64, device="cuda")
    M.layernorm_forward(buf[:, 4:36], None, None, buf[:, 36:68], None, rstd, eps=EPS)
    y, _, r = forward(x, None, None, False)
    assert torch.equal(buf[:, 36:68], y) and torch.equal(rstd, r) and torch.equal(buf[:, 4:36], x)
    assert not buf[:, :4].any() and not buf[:, 68:].any()
    with pytest.raises(M.MsampError):
        M.layernorm_forward(buf[:, 4:36], None, None, buf[:, 35:67], None, rstd, eps=EPS)
    assert torch.equal(buf[:, 4:36], x)


def test_backward_against_differences():
    """dx and dweight against central differences of the kernel's own binary32 forward pass."""
    rows, cols, step = 3, 40, 2.0 ** -7
    x, dy = matrix(rows, cols, torch.float32, 0, 1), matrix(rows, cols, torch.float32, 0, 2)
    w, b = weights(cols, torch.float32, 3)
    _, mean, rstd = forward(x, w, b, True)
    dx, dw, db = backward(dy, x, w, mean, rstd)
    vx, vw, vb = matrix(rows, cols, torch.float32, 0, 4), *weights(cols, torch.float32, 5)
    up = forward(x + step * vx, w + step * vw, b + step * vb, True)[0].double()
    down = forward(x - step * vx, w - step * vw, b - step * vb, True)[0].double()
    diff = ((up - down) * dy.double()).sum().item() / (2 * step)
    along = (dx.double() * vx.double()).sum().item() + (dw.double() * vw.double()).sum().item() + (db.double() * vb.double()).sum().item()
    # rounding of y: 128 steps of |y| |dy| over 2 step; truncation: step^2 / 6 of a third derivative of order
    # |dy| |y| (rstd |v|)^3 for each value (rstd is about 1 and |v| below 4 here, so below 64)
    size = (up.abs() * dy.double().abs()).sum().item()
    assert abs(diff - along) <= 128 * R.U * size / step + step ** 2 / 6 * 64 * size


def test_in_a_graph_with_eager_work_between():
    x, dy = matrix(600, 520, torch.bfloat16, 0, 1), matrix(600, 520, torch.bfloat16, 0, 2)
    w, b = weights(520, torch.bfloat16, 3)
    ck = M.new_checkpoint(600, 520)
    y, mean, rstd = torch.empty_like(x), torch.empty(600, device="cuda"), torch.empty(600, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(520, device="cuda"), torch.empty(520, device="cuda")

    def step():
        M.layernorm_forward(x, w, b, y, mean, rstd, save=ck)
        M.layernorm_backward(dy, ck, w, mean, rstd, dx, dw, db)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):
        step()
    for k in range(4):
        x.copy_(torch.randn(600, 520, device="cuda") * 2.0 ** k)
        (g if k % 2 == 0 else other).replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, mean, rstd, dx, dw, db, ck.codes, ck.scales)]
        step()
        torch.cuda.synchronize()
        for p, q in zip(got, (y, mean, rstd, dx, dw, db, ck.codes, ck.scales)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", [(3, 8200), (300, 12007), (700, 16384), (3, 16392), (5, 16385), (256, 20001),
                                       (257, 24000), (600, 16390), (3, 32761), (300, 32768), (515, 32767)])
def test_wide_rows_over_several_workgroups(rows, cols, dtype):
    """Two and four pieces of 8 columns a lane, one and several rows a workgroup, sums joined from their parts: from a
    matrix and from a checkpoint, added to what is there."""
    dt = DT[dtype]
    x, dy = matrix(rows, cols, dt, 0, 1, offset=0.5), matrix(rows, cols, dt, 0, 2, size=0.1)
    w, _ = weights(cols, dt, 3)
    ck = M.new_checkpoint(rows, cols, M.E5M2 if rows % 2 else M.E4M3)
    for centered in (True, False):
        _, mean, rstd = forward(x, w, None, centered, save=ck)
        xv = torch.empty(rows, cols, device="cuda")
        M.checkpoint_load(ck, xv)
        for src, val in ((x, x), (ck, xv)):
            first = backward(dy, src, w, mean, rstd)
            check_backward(dy, val, w, mean, rstd, first)
            dw, db = torch.full((cols,), 2.0, device="cuda"), torch.full((cols,), -3.0, device="cuda")
            dx, dw2, db2 = backward(dy, src, w, mean, rstd, True, dw, db)
            assert torch.equal(dx, first[0]) and torch.equal(dw2, 2.0 + first[1]) and torch.equal(db2, -3.0 + first[2])


def test_rows_whose_squares_leave_binary32():
    """The sums are binary32's: where the sum of the squares exceeds it, rstd is 0, and so are y (without a bias) and
    dx. The other rows are as they are without it."""
    x, dy = matrix(8, 700, torch.float32, 0, 1), matrix(8, 700, torch.float32, 0, 2)
    _, b = weights(700, torch.float32, 3)
    keep = [0, 1, 3, 4, 5, 7]
    big = x.clone()
    big[2], big[6, 9] = torch.finfo(torch.float32).max, 1e20
    for bias in (None, b):
        clean, _, r = forward(x, None, bias, False)
        y, _, rstd = forward(big, None, bias, False)
        assert (rstd[[2, 6]] == 0).all() and torch.equal(rstd[keep], r[keep]) and torch.equal(y[keep], clean[keep])
        want = torch.zeros(700, device="cuda") if bias is None else bias
        assert torch.equal(y[2], want) and torch.equal(y[6], want)
    dx, dw, _ = backward(dy, big, None, None, rstd)
    ref = backward(dy, x, None, None, r)
    assert not dx[[2, 6]].any() and torch.equal(dx[keep], ref[0][keep]) and torch.isfinite(dw).all()
    # around the mean, as long as their sum is within binary32
    big[2] = torch.where(torch.arange(700, device="cuda") % 2 == 0, 1e20, -1e20)
    y, mean, rstd = forward(big, None, None, True)
    assert (rstd[[2, 6]] == 0).all() and torch.isfinite(mean).all() and not y[[2, 6]].any()
    assert not backward(dy, big, None, mean, rstd)[0][[2, 6]].any()
