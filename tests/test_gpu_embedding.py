"""Embedding lookup and its gradient on the GPU against the binary64 reference
(tests/model_ref.py), whose bounds count the sums' and products' roundings."""
import pytest
import torch

import bit_adamw_optimizer_amd as M
from tests import model_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# rows, vocabulary, columns, padding behind each row
SHAPES = [(1, 1, 1, 0), (2, 5, 3, 0), (7, 40, 33, 1), (64, 9, 64, 0), (65, 100, 100, 3), (300, 17, 257, 0), (129, 1000, 513, 8),
          (33, 6000, 65, 0), (10, 50, 1027, 1), (50, 30, 2052, 0), (3, 300, 4100, 0)]


def rows_of(rows, cols, pad, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = (torch.randn(rows, cols, generator=g) * size).to(dtype)
    return buf[:, :cols]


def ids_of(rows, vocab, seed, dtype=torch.int64, bad=True):
    """A few ids often, the others seldom; some outside the vocabulary."""
    g = torch.Generator().manual_seed(seed)
    ids = (torch.rand(rows, generator=g) ** 3 * vocab).long().clamp(0, vocab - 1)
    if bad and rows > 4:
        top = torch.iinfo(dtype)
        ids[1], ids[3], ids[rows // 2], ids[-1] = -1, vocab, top.min, top.max
    return ids.to(dtype).cuda()


def forward(ids, w, scale=1.0):
    rows, cols = ids.shape[0], w.shape[1]
    y = torch.full((rows + 1, cols + 1), 7.0, dtype=w.dtype, device="cuda")
    M.embedding_forward(ids, w, y[:rows, :cols], scale=scale)
    assert (y[rows:] == 7).all() and (y[:, cols:] == 7).all()
    return y[:rows, :cols]


def backward(dy, ids, vocab, scale=1.0, base=None):
    cols = dy.shape[1]
    dw = torch.full((vocab + 1, cols + 1), 7.0, device="cuda")
    if base is not None:
        dw[:vocab, :cols] = base
    M.embedding_backward(dy, ids, dw[:vocab, :cols], scale=scale, accumulate=base is not None)
    assert (dw[vocab:] == 7).all() and (dw[:, cols:] == 7).all()
    return dw[:vocab, :cols]


def check_backward(dy, ids, vocab, scale, got, base=None):
    ref, bound = R.embedding_backward(dy.cpu(), ids.cpu(), vocab, scale, None if base is None else base.cpu())
    R.assert_near(got, ref, bound, "dweight")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,vocab,cols,pad", SHAPES)
def test_forward_and_backward(rows, vocab, cols, pad, dtype):
    dt = DT[dtype]
    w, dy = rows_of(vocab, cols, pad, dt, 1), rows_of(rows, cols, pad, dt, 2, 0.1)
    for it in (torch.int64, torch.int32):
        ids = ids_of(rows, vocab, cols, it)
        y = forward(ids, w, 1.7)
        ref, bound = R.embedding_forward(ids.cpu(), w.cpu(), torch.tensor(1.7).double())
        R.assert_near(y, ref, bound, "y")
        check_backward(dy, ids, vocab, torch.tensor(1.7).double(), backward(dy, ids, vocab, 1.7))
    base = rows_of(vocab, cols, 0, torch.float32, 3)
    got = backward(dy, ids, vocab, 0.5, base)
    check_backward(dy, ids, vocab, 0.5, got, base)
    live = ids[(ids >= 0) & (ids < vocab)].long()
    absent = torch.ones(vocab, dtype=torch.bool, device="cuda")
    absent[live] = False
    assert torch.equal(got[absent], base[absent])


@pytest.mark.parametrize("rows,vocab,cols,hot", [
    (1000, 7, 40, 0.9), (5000, 300, 33, 0.5), (64, 3, 1030, 1.0), (65, 3, 1030, 1.0), (70000, 50, 9, 0.97), (66000, 70000, 8, 0.3),
    (140000, 11, 5, 0.6)])
def test_an_id_with_most_of_the_rows(rows, vocab, cols, hot):
    """Sums cut into pieces, whole and ended inside a piece; more rows to a piece for many rows."""
    g = torch.Generator().manual_seed(rows)
    ids = torch.randint(0, vocab, (rows,), generator=g)
    ids[torch.rand(rows, generator=g) < hot] = vocab // 2
    ids = ids.cuda()
    dy = rows_of(rows, cols, 0, torch.float16, 5, 0.1)
    got = backward(dy, ids, vocab)
    check_backward(dy, ids, vocab, 1.0, got)
    assert torch.equal(got, backward(dy, ids, vocab))  # in the rows' order, every time


def test_a_large_vocabulary_of_narrow_rows():
    rows, vocab, cols = 3000, 300001, 2
    ids, dy = ids_of(rows, vocab, 1), rows_of(rows, cols, 0, torch.bfloat16, 2)
    check_backward(dy, ids, vocab, 1.0, backward(dy, ids, vocab))


def test_all_padding_and_no_rows():
    dy = rows_of(5, 12, 0, torch.float32, 1)
    ids = torch.full((5,), -1, device="cuda")
    w = rows_of(4, 12, 0, torch.float32, 2)
    assert (forward(ids, w) == 0).all() and (backward(dy, ids, 4) == 0).all()
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert (backward(dy[:0], none, 4) == 0).all()
    M.embedding_forward(none, w, torch.empty(0, 12, device="cuda"))
    y = forward(torch.zeros(3, dtype=torch.int64, device="cuda"), w[:0])  # nothing in the vocabulary
    assert (y == 0).all()
    base = rows_of(4, 12, 0, torch.float32, 3)
    assert torch.equal(backward(dy[:0], none, 4, base=base), base)


def test_special_values_stay_in_their_rows():
    ids = torch.tensor([2, 0, 1, 0], device="cuda")
    dy = rows_of(4, 9, 0, torch.float16, 1)
    dy[0, 3], dy[2, 4] = float("inf"), float("nan")
    dw = backward(dy, ids, 4)
    assert torch.isinf(dw[2, 3]) and torch.isnan(dw[1, 4]) and torch.isfinite(dw).sum() == dw.numel() - 2
    w = rows_of(3, 9, 0, torch.float16, 2)
    w[1] = float("nan")
    y = forward(ids, w)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3]]).all()


def test_weights_and_gradients_beyond_32_bits_of_offset():
    vocab, cols = 70001, 32768
    w = torch.empty(vocab, cols, dtype=torch.float16, device="cuda")
    w[-1] = 3.0
    ids = torch.tensor([vocab - 1, vocab - 1], device="cuda")
    assert (forward(ids, w, 2.0) == 6).all()
    del w
    dw = torch.empty(vocab, cols, device="cuda")
    M.embedding_backward(torch.full((2, cols), 1.5, dtype=torch.float16, device="cuda"), ids, dw)
    assert (dw[-1] == 3).all() and not dw[:-1].any()


def test_another_stream_and_replays():
    rows, vocab, cols = 500, 40, 96
    w, dy, ids = rows_of(vocab, cols, 0, torch.float16, 1), rows_of(rows, cols, 0, torch.float16, 2), ids_of(rows, vocab, 3)
    want_y, want_dw = forward(ids, w, 2.0).clone(), backward(dy, ids, vocab, 2.0).clone()
    outs, graphs = [], []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, dw = torch.zeros(rows, cols, dtype=torch.float16, device="cuda"), torch.zeros(vocab, cols, device="cuda")
        M.embedding_forward(ids, w, y, scale=2.0)
        M.embedding_backward(dy, ids, dw, scale=2.0)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want_y) and torch.equal(dw, want_dw)
    for _ in range(2):  # two graphs, workspaces of their own
        y, dw = torch.zeros_like(want_y), torch.zeros(vocab, cols, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.embedding_forward(ids, w, y, scale=2.0)
            M.embedding_backward(dy, ids, dw, scale=2.0)
        graphs.append(g)
        outs.append((y, dw))
    for _ in range(3):
        for y, dw in outs:
            y.fill_(5), dw.fill_(5)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for y, dw in outs:
            assert torch.equal(y, want_y) and torch.equal(dw, want_dw)
        backward(dy, ids, vocab)  # eager work between the replays


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,vocab,cols", [
    (40, 3, 4100), (40, 3, 4157), (45, 3, 5000), (30, 2, 8196), (40000, 700, 132), (40000, 700, 190), (40000, 700, 252),
    (140000, 1100, 131)])
def test_ids_of_several_rows_whose_last_columns_do_not_fill_a_wave(rows, vocab, cols, dtype):
    """A wave reads its rows' numbers from all of its lanes, those without columns among them: as many rows of an id as
    a piece has (16, 64 of 40,000 rows, 256 of 140,000) and fewer, and ids of more than a piece."""
    g = torch.Generator().manual_seed(cols)
    ids = torch.randint(0, vocab, (rows,), generator=g)
    ids[rows // 2] = -1
    if rows > 1000:
        ids[ids >= vocab - 2] = 0
        ids[:64], ids[64:64 + 50] = vocab - 1, vocab - 2
    ids = ids.cuda()
    dy, base = rows_of(rows, cols, 1, DT[dtype], 7, 0.1), rows_of(vocab, cols, 0, torch.float32, 8)
    got = backward(dy, ids, vocab, 0.5)
    check_backward(dy, ids, vocab, 0.5, got)
    check_backward(dy, ids, vocab, 0.5, backward(dy, ids, vocab, 0.5, base), base)
    assert torch.equal(got, backward(dy, ids, vocab, 0.5))


@pytest.mark.parametrize("rows,vocab,cols", [(300, 4, 7), (1000, 50, 260), (20000, 9, 3)])
def test_the_order_of_the_sum(rows, vocab, cols):
    """In the rows' order up to a piece of them; beyond it pieces of the rows sorted by id, joined in order."""
    ids, dy = ids_of(rows, vocab, 3), rows_of(rows, cols, 0, torch.float32, 4)
    piece = 16
    while piece * 1024 < rows:
        piece *= 2
    i, v = ids.cpu(), dy.cpu()
    order = torch.argsort(torch.where((i < 0) | (i >= vocab), vocab, i), stable=True)
    want, at = torch.zeros(vocab, cols), 0
    for k in range(vocab):
        n = int((i == k).sum())
        cuts = [at, at + n] if n <= piece else [at, *range(at // piece * piece + piece, at + n, piece), at + n]
        total = torch.zeros(cols)
        for p0, p1 in zip(cuts, cuts[1:]):
            part = torch.zeros(cols)
            for r in order[p0:p1]:
                part += v[r]
            total = part if len(cuts) == 2 else total + part
        want[k], at = total, at + n
    assert torch.equal(backward(dy, ids, vocab).cpu(), want)


def test_more_rows_than_a_launch_has():
    """More than 2^20 workgroups: looked up in turns, gradients in slices of the vocabulary or of the rows."""
    n = (1 << 20) + 3
    ids = torch.arange(n, device="cuda") % 7
    w = rows_of(7, 520, 0, torch.float16, 1)
    y = torch.zeros(n, 520, dtype=torch.float16, device="cuda")
    M.embedding_forward(ids, w, y)
    assert torch.equal(y, w[ids])
    del y
    dw = torch.full((n, 2049), 7.0, device="cuda")
    few = torch.tensor([n - 1, 0, n - 1], device="cuda")
    M.embedding_backward(torch.ones(3, 2049, dtype=torch.float16, device="cuda"), few, dw)
    assert (dw[0] == 1).all() and (dw[-1] == 2).all() and not dw[1:-1].any()
    del dw
    dw = torch.ones(7, 2049, device="cuda")
    M.embedding_backward(torch.ones(n, 2049, dtype=torch.float16, device="cuda"), ids, dw, accumulate=True)
    assert torch.equal(dw[:, 0].cpu(), 1.0 + torch.bincount(ids.cpu(), minlength=7)) and (dw == dw[:, :1]).all()
