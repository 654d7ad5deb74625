"""Distillation and the clipped policy loss on the GPU, losses and gradients,
against the binary64 reference (tests/model_ref.py)."""
import math

import pytest
import torch

import bit_adamw_optimizer_amd as M
from tests import model_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SHAPES = [(1, 1, 0), (3, 2, 0), (5, 7, 1), (2, 64, 0), (3, 513, 0), (2, 1000, 8), (3, 2049, 0), (2, 4103, 3), (2, 8192, 0),
          (2, 16391, 0), (3, 32000, 0), (2, 50257, 0), (1, 70001, 5), (2, 140003, 0), (1, 300000, 0)]
INF = math.inf


def matrix(rows, cols, dtype, pad, seed, size=2.5):
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = (torch.randn(rows, cols, generator=g) * size).to(dtype)
    return buf[:, :cols]


def out_like(z):
    rows, vocab = z.shape
    buf = torch.full((rows + 1, vocab + 1), 7.0, dtype=z.dtype, device="cuda")
    return buf, buf[:rows, :vocab]


def near(val, err, got):
    for name, g in got.items():
        v, far = val[name], torch.isinf(val[name])  # the largest logit of a row that has none: -Inf itself
        assert torch.equal(g.cpu().double()[far], v[far]), name
        R.assert_near(g.cpu().masked_fill(far, 0.0), v.masked_fill(far, 0.0), err[name], name)


def cpu(t):
    return None if t is None else t.cpu()


def check_distill(z, ids, t, tau, dloss=None):
    """Loss alone with stats, the gradient from them, and both in one pass, over logits of their own."""
    rows, vocab = z.shape
    loss, stats = torch.full((rows,), 7.0, device="cuda"), torch.full((rows, 2), 7.0, device="cuda")
    M.distill_loss_forward(z, ids, t, loss, temperature=tau, stats=stats)
    buf, dz = out_like(z)
    M.distill_loss_backward(dloss, z, ids, t, stats, dz, temperature=tau)
    assert (buf[rows:] == 7).all() and (buf[:, vocab:] == 7).all()
    both, buf2, dz2 = torch.full((rows,), 7.0, device="cuda"), *out_like(z)
    M.distill_loss_forward(z, ids, t, both, temperature=tau, dlogits=dz2, dloss=dloss)
    assert (buf2[rows:] == 7).all() and (buf2[:, vocab:] == 7).all()
    val, err = R.distill(z.cpu(), ids.cpu(), t.cpu(), tau, cpu(dloss))
    near(val, err, {"loss": loss, "stats": stats, "dlogits": dz})
    near(val, err, {"loss": both, "dlogits": dz2})
    inplace = z.clone()
    M.distill_loss_forward(inplace, ids, t, both, temperature=tau, dlogits=inplace, dloss=dloss)
    near(val, err, {"loss": both, "dlogits": inplace})
    inplace = z.clone()
    M.distill_loss_backward(dloss, inplace, ids, t, stats, inplace, temperature=tau)
    near(val, err, {"dlogits": inplace})
    return loss, stats, dz


def classes(rows, vocab, top, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, vocab, (rows, top), generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,vocab,pad", SHAPES)
def test_distillation(rows, vocab, pad, dtype):
    z = matrix(rows, vocab, DT[dtype], pad, vocab)
    for top, tau, tt in ((1, 1.0, torch.float32), (5, 2.0, DT[dtype])):
        ids = classes(rows, vocab, top, top)
        t = matrix(rows, top, tt, 1, 3)
        g = torch.linspace(0.5, 300.0, rows).cuda()
        check_distill(z, ids, t, tau, g)
    check_distill(z, classes(rows, vocab, 3, 9, torch.int32), matrix(rows, 3, torch.bfloat16, 0, 3), 0.5)


@pytest.mark.parametrize("top", [20, 64, 65, 257, 512, 513, 1000, 1024])
def test_many_classes_some_twice_some_absent(top):
    rows, vocab = 4, 700  # more classes than that come more than once
    z, t = matrix(rows, vocab, torch.float32, 0, 1), matrix(rows, top, torch.float32, 0, 2)
    ids = classes(rows, vocab, top, top)
    ids[0, ::3] = -1
    ids[1, 1::2] = ids[1, :1]
    ids[2, 3] = vocab
    t[3, ::2] = -INF
    check_distill(z, ids, t, 1.3, torch.full((rows,), 100.0, device="cuda"))


def test_the_same_class_in_every_entry():
    z = matrix(3, 50, torch.float32, 0, 1)
    ids = torch.full((3, 17), 49, device="cuda")
    t = torch.zeros(3, 17, device="cuda")
    loss, _, dz = check_distill(z, ids, t, 1.0)
    hard = torch.nn.functional.cross_entropy(z.double().cpu(), torch.full((3,), 49), reduction="none")
    # 17 entries of p = 1/17 (entropy log 17), whose classes' q is counted for each
    assert torch.allclose(loss.cpu().double(), hard - math.log(17), atol=1e-5)


@pytest.mark.parametrize("dtype", list(DT))
def test_rows_that_are_left_out_and_masked_vocabularies(dtype):
    dt = DT[dtype]
    low = torch.finfo(dt).min
    rows, vocab = 9, 900
    z, t = matrix(rows, vocab, dt, 0, 1), matrix(rows, 4, torch.float32, 0, 2)
    ids = classes(rows, vocab, 4, 3)
    for r in range(rows):
        ids[r] = torch.arange(4) + 10 * r
    ids[0] = -1                      # no entry
    t[1] = -INF                      # none above -Inf
    z[2] = -INF                      # no logit
    z[3, 100:] = -INF                # a masked vocabulary
    z[4, 100:] = low                 # the same by the type's lowest value
    z[5] = low                       # every logit there: a uniform softmax
    ids[6] = torch.tensor([vocab, -5, 1 << 40, 61])
    z[7, 500:] = -INF
    z[8, :] = -INF
    z[8, 81] = 1.0                   # one class left
    ids[8] = torch.tensor([81, 81, -1, 81])
    g = torch.full((rows,), 64.0, device="cuda")
    loss, stats, dz = check_distill(z, ids, t, 1.0, g)
    for r in (0, 1, 2):
        assert loss[r] == 0 and not dz[r].any()
    assert (stats[0] == 0).all() and stats[2, 0] == -INF and stats[2, 1] == 0
    assert not dz[3, 100:].any() and not dz[4, 100:].any() and (dz[5, :10] > 0).all()

    act = torch.tensor([-1, vocab, 5, 50, 50, 50, 3, 4, 81], device="cuda")
    old = torch.full((rows,), -6.0, device="cuda")
    adv = torch.linspace(-1, 1, rows).cuda()
    check_policy(z, act, old, adv, 1.0, dloss=g)


def test_a_class_that_the_mask_leaves_out_is_infinitely_far():
    z = matrix(2, 40, torch.float32, 0, 1)
    z[0, 7] = -INF
    ids = torch.tensor([[7, 3], [7, 3]], device="cuda")
    t = torch.zeros(2, 2, device="cuda")
    loss, dz = torch.empty(2, device="cuda"), torch.empty_like(z)
    M.distill_loss_forward(z, ids, t, loss, dlogits=dz)
    assert loss[0] == INF and torch.isfinite(loss[1]) and torch.isfinite(dz).all() and dz[0, 7] == -0.5


def test_nan_and_infinite_logits_stay_in_their_rows():
    z, t = matrix(6, 1200, torch.float32, 0, 1), matrix(6, 3, torch.float32, 0, 2)
    ids = classes(6, 1200, 3, 3)
    z[1, 700], z[2, 5] = float("nan"), INF
    t[3, 1], t[4, 0] = float("nan"), INF
    loss, stats, dz = torch.empty(6, device="cuda"), torch.empty(6, 2, device="cuda"), torch.empty_like(z)
    M.distill_loss_forward(z, ids, t, loss, stats=stats, dlogits=dz)
    for r in range(6):
        assert torch.isnan(loss[r]) == (r in (1, 2, 3, 4)), r
        assert torch.isnan(dz[r]).any() == (r in (1, 2, 3, 4)), r
    assert torch.isnan(dz[1]).all()
    act, old, adv = ids[:, 0].contiguous(), torch.full((6,), -8.0, device="cuda"), torch.ones(6, device="cuda")
    M.policy_loss_forward(z, act, old, adv, loss, dlogits=dz)
    assert torch.isnan(loss).tolist() == [False, True, True, False, False, False]
    assert torch.isfinite(dz[[0, 3, 4, 5]]).all() and torch.isnan(dz[1]).any()


# ------------------------------------------------------------------ policy ---

def check_policy(z, act, old, adv, tau, ref=None, kl=0.0, low=0.2, high=0.2, dloss=None):
    rows, vocab = z.shape
    kw = dict(ref_logp=ref, kl=kl, clip_low=low, clip_high=high, temperature=tau)
    loss, logp, stats = (torch.full(s, 7.0, device="cuda") for s in ((rows,), (rows,), (rows, 2)))
    M.policy_loss_forward(z, act, old, adv, loss, logp=logp, stats=stats, **kw)
    buf, dz = out_like(z)
    M.policy_loss_backward(dloss, z, act, old, adv, stats, dz, **kw)
    assert (buf[rows:] == 7).all() and (buf[:, vocab:] == 7).all()
    both, buf2, dz2 = torch.full((rows,), 7.0, device="cuda"), *out_like(z)
    M.policy_loss_forward(z, act, old, adv, both, dlogits=dz2, dloss=dloss, **kw)
    assert (buf2[rows:] == 7).all() and (buf2[:, vocab:] == 7).all()
    val, err, clear = R.policy(z.cpu(), act.cpu(), old.cpu(), adv.cpu(), tau, cpu(ref), kl, low, high, cpu(dloss))
    assert clear.min() > 1e-5  # no ratio on a bound of the clip, where a rounding would decide
    near(val, err, {"loss": loss, "logp": logp, "stats": stats, "dlogits": dz})
    near(val, err, {"loss": both, "dlogits": dz2})
    inplace = z.clone()
    M.policy_loss_forward(inplace, act, old, adv, both, dlogits=inplace, dloss=dloss, **kw)
    near(val, err, {"loss": both, "dlogits": inplace})
    inplace = z.clone()
    M.policy_loss_backward(dloss, inplace, act, old, adv, stats, inplace, **kw)
    near(val, err, {"dlogits": inplace})
    return loss, logp, stats, dz


def rollout(z, tau, seed):
    """Actions, and old and reference log-probabilities around the present ones, on both sides of the clip."""
    rows, vocab = z.shape
    g = torch.Generator().manual_seed(seed)
    act = torch.randint(0, vocab, (rows,), generator=g)
    lp = torch.log_softmax(z.cpu().double() / tau, 1).gather(1, act[:, None])[:, 0]
    shift = torch.tensor([0.0, 0.5, -0.5, 0.1, -0.1])[torch.arange(rows) % 5]
    adv = torch.randn(rows, generator=g)
    return act.cuda(), (lp - shift).float().cuda(), (lp + 0.3 * torch.randn(rows, generator=g)).float().cuda(), adv.cuda()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,vocab,pad", SHAPES)
def test_policy(rows, vocab, pad, dtype):
    z = matrix(rows, vocab, DT[dtype], pad, vocab)
    g = torch.linspace(0.5, 300.0, rows).cuda()
    for tau, kl in ((1.0, 0.05), (0.7, 0.0)):
        act, old, ref, adv = rollout(z, tau, rows)
        check_policy(z, act, old, adv, tau, ref if kl else None, kl, dloss=g)
    check_policy(z, act.int(), old, adv, 0.7, ref, 0.0, 0.1, 0.3)


def test_every_side_of_the_clip():
    """Both signs of the advantage, and none, inside and beyond both bounds; no upper bound, a lower one of 0."""
    z = matrix(15, 333, torch.float32, 0, 1)
    act = torch.arange(15, device="cuda") * 7
    lp = torch.log_softmax(z.double(), 1).gather(1, act[:, None])[:, 0]
    shift = torch.tensor([0.0, 0.4, -0.4, 0.17, -0.2]).repeat(3).cuda()
    old, adv = (lp - shift).float(), torch.tensor([1.5, -2.0, 0.0]).repeat_interleave(5).cuda()
    ref = (lp + 0.5).float()
    loss, _, _, dz = check_policy(z, act, old, adv, 1.0, ref, 0.0)
    still = [not dz[i].any().item() for i in range(15)]
    # A > 0: beyond the upper bound only; A < 0: beyond the lower one only; A = 0: always
    assert still == [False, True, False, False, False] + [False, False, True, False, False] + [True] * 5
    check_policy(z, act, old, adv, 1.0, ref, 0.3)
    check_policy(z, act, old, adv, 1.0, ref, -0.3, 1.0, INF)
    check_policy(z, act, old, adv, 1.0, None, 0.0, 0.001, 1e9)


def test_left_out_rows_are_not_read():
    z = matrix(4, 600, torch.float16, 0, 1)
    z[1], z[3] = float("nan"), float("nan")
    act = torch.tensor([5, -1, 6, 600], device="cuda")
    v = torch.full((4,), -6.0, device="cuda")
    old, adv = v.clone(), torch.ones(4, device="cuda")
    old[1] = adv[3] = float("nan")
    loss, logp, dz = torch.full((4,), 7.0, device="cuda"), torch.full((4,), 7.0, device="cuda"), torch.full_like(z, 7.0)
    M.policy_loss_forward(z, act, old, adv, loss, logp=logp, dlogits=dz, ref_logp=v, kl=0.1)
    for r in (1, 3):
        assert loss[r] == 0 and logp[r] == 0 and not dz[r].any()
    assert torch.isfinite(loss).all() and torch.isfinite(dz).all()
    ids, t = act[:, None].repeat(1, 2), torch.zeros(4, 2, device="cuda")
    M.distill_loss_forward(z, ids, t, loss, dlogits=dz)
    assert loss[1] == 0 and not dz[3].any() and torch.isfinite(dz).all()


def test_ratios_next_to_a_bound_fall_on_their_side():
    """A relative 2e-6 from the bounds: far beyond what a sum of 32,000 terms may be off, and close to it in binary32."""
    rows, vocab = 64, 32000
    z = matrix(rows, vocab, torch.float32, 0, 1)
    act = torch.arange(rows, device="cuda") * 91
    lp = torch.log_softmax(z.double(), 1).gather(1, act[:, None])[:, 0]
    side = torch.where(torch.arange(rows) % 2 == 0, 1.0, -1.0).double().cuda()
    old = (lp - math.log(1.2) - 4e-6 * side).float()
    ratio = torch.exp(lp - old.double())
    beyond = ratio > 1.2
    assert ((ratio / 1.2 - 1).abs() > 2e-6).all() and beyond.sum() > 10 and (~beyond).sum() > 10
    loss, dz = torch.empty(rows, device="cuda"), torch.empty_like(z)
    M.policy_loss_forward(z, act, old, torch.ones(rows, device="cuda"), loss, dlogits=dz)
    assert torch.equal(dz.any(1), ~beyond)


def test_offsets_beyond_32_bits_and_empty_calls():
    rows, vocab = 9, 1 << 28
    z = torch.zeros(rows, vocab, dtype=torch.float16, device="cuda")
    z[8, -1] = 8.0
    act = torch.full((rows,), vocab - 1, device="cuda")
    v, adv, loss = torch.full((rows,), -19.0, device="cuda"), torch.ones(rows, device="cuda"), torch.empty(rows, device="cuda")
    logp = torch.empty(rows, device="cuda")
    M.policy_loss_forward(z, act, v, adv, loss, logp=logp, dlogits=z, clip_high=INF,
                          dloss=torch.full((rows,), 1024.0, device="cuda"))
    want = torch.tensor([-math.log(vocab)] * 8 + [8 - math.log(vocab - 1 + math.exp(8))], dtype=torch.float64)
    R.assert_near(logp, want, 1e-4 * torch.ones(9, dtype=torch.float64), "logp")  # sums of 2^28 equal terms
    assert (z[:, -1] != 0).all()
    del z
    for shape in ((0, 5), (3, 0)):
        e, f = torch.empty(shape, device="cuda"), torch.full((shape[0],), 7.0, device="cuda")
        i = torch.zeros(shape[0], dtype=torch.int64, device="cuda")
        M.policy_loss_forward(e, i, f, f.clone(), f.clone(), dlogits=torch.empty_like(e))
        M.distill_loss_forward(e, i[:, None], f[:, None], f.clone(), dlogits=torch.empty_like(e))
    f = torch.full((3,), 7.0, device="cuda")
    M.distill_loss_forward(torch.zeros(3, 5, device="cuda"), torch.zeros(3, 0, dtype=torch.int64, device="cuda"),
                           torch.zeros(3, 0, device="cuda"), f)
    assert not f.any()


def test_another_stream_and_replays():
    rows, vocab = 5, 40001
    z, t, ids = matrix(rows, vocab, torch.bfloat16, 0, 1), matrix(rows, 9, torch.float32, 0, 2), classes(rows, vocab, 9, 3)
    act, old, ref, adv = rollout(z, 1.0, 4)

    def outputs():
        return [torch.zeros(rows, device="cuda") for _ in range(2)] + [torch.zeros(rows, 2, device="cuda")] + [
            torch.zeros(rows, vocab, dtype=z.dtype, device="cuda") for _ in range(4)]

    def go(o):
        M.distill_loss_forward(z, ids, t, o[0], stats=o[2], dlogits=o[3])
        M.distill_loss_backward(None, z, ids, t, o[2], o[4])
        M.policy_loss_forward(z, act, old, adv, o[1], ref_logp=ref, kl=0.1, stats=o[2], dlogits=o[5])
        M.policy_loss_backward(None, z, act, old, adv, o[2], o[6], ref_logp=ref, kl=0.1)

    want, other = outputs(), outputs()
    go(want)
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
@pytest.mark.parametrize("vocab", [512, 1 << 15, 1 << 17])
def test_the_kl_term_next_to_the_reference_policy(vocab, dtype):
    """e^d - d - 1 is about d^2 / 2: every digit of it, where lp is exact (equal logits, a power of two of them: sums
    of ones, and a logarithm in binary64, off by less than 2^-49). One rounding, the binary64 logarithm's 2^-49 as
    a part of d, expm1's last place as a part of d / 2; the gradient's exact q leaves the factor and two products."""
    d = torch.tensor([0.3, -0.3, 1e-2, -1e-2, 1e-3, -1e-3, 1e-4, -1e-4, 1e-5, -1e-5, 1e-6, 0.0], dtype=torch.float64)
    rows, lp = len(d), -math.log(vocab)
    z = torch.full((rows, vocab), 1.5, dtype=DT[dtype], device="cuda")
    ref = (lp + d).float()
    d = ref.double() - lp
    act, old, adv = torch.arange(rows, device="cuda"), torch.full((rows,), lp, device="cuda"), torch.zeros(rows, device="cuda")
    for tau in (1.0, 2.0):
        loss, dz = torch.empty(rows, device="cuda"), torch.empty_like(z)
        M.policy_loss_forward(z, act, old, adv, loss, ref_logp=ref.cuda(), kl=0.5, dlogits=dz, temperature=tau)
        want = 0.5 * (torch.expm1(d) - d)
        R.assert_near(loss, want, 2 ** -47 * d.abs() + 2 ** -96, "loss")
        q = torch.full((rows, vocab), -1.0 / vocab, dtype=torch.float64)
        q[torch.arange(rows), torch.arange(rows)] += 1
        want = (-0.5 * torch.expm1(d) / tau)[:, None] * q
        R.assert_near(dz, want, 4 * R.U * want.abs() + 2 ** -48, "dlogits")


def test_a_masked_action_is_infinitely_far_from_a_reference_that_allows_it():
    z = matrix(3, 700, torch.float32, 0, 1)
    z[1, 5] = -INF
    act, v, adv = torch.full((3,), 5, device="cuda"), torch.full((3,), -6.0, device="cuda"), torch.ones(3, device="cuda")
    loss, logp = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    for kl, want in ((0.1, INF), (-0.1, -INF), (0.0, 0.0)):
        M.policy_loss_forward(z, act, v, adv, loss, logp=logp, ref_logp=v, kl=kl)
        assert loss[1] == want and logp[1] == -INF and torch.isfinite(loss[[0, 2]]).all()


@pytest.mark.parametrize("tau", [1e-25, 1e-12, 0.01, 20.0])
def test_temperatures_far_from_one(tau):
    """temperature^2 leaves binary32 before temperature times a logit does."""
    rows, vocab = 3, 900
    z, t = matrix(rows, vocab, torch.float32, 0, 1), matrix(rows, 5, torch.float32, 0, 2)
    loss, _, _ = check_distill(z, classes(rows, vocab, 5, 3), t, tau, torch.full((rows,), 8.0, device="cuda"))
    assert (loss > 0).all()


def test_more_rows_than_a_launch_has():
    """Rows in slices of 2^20."""
    rows, vocab = (1 << 20) + 3, 5
    z = matrix(rows, vocab, torch.float32, 0, 1)
    act, old, ref, adv = rollout(z, 1.0, 2)
    act[7::11] = -1
    lp = torch.log_softmax(z.double(), 1).gather(1, act.clamp_min(0)[:, None])[:, 0]
    near_bound = torch.minimum(((lp - old).exp() / 1.2 - 1).abs(), ((lp - old).exp() - 0.8).abs()) < 1e-4
    act[near_bound] = -1
    check_policy(z, act, old, adv, 1.0, ref, 0.1, dloss=torch.full((rows,), 64.0, device="cuda"))
    check_distill(z, torch.stack([act, act + 1], 1), z[:, :2].contiguous(), 2.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_longest_row(dtype):
    """2^29 logits, all but two equal: sums of a power of two and exact exponentials."""
    vocab = 1 << 29
    z = torch.zeros(1, vocab, dtype=DT[dtype], device="cuda")
    act = torch.tensor([vocab - 1], device="cuda")
    old, adv = torch.full((1,), -20.0, device="cuda"), torch.ones(1, device="cuda")
    loss, logp, stats = torch.empty(1, device="cuda"), torch.empty(1, device="cuda"), torch.empty(1, 2, device="cuda")
    want = -math.log(vocab)
    M.policy_loss_forward(z, act, old, adv, loss, logp=logp, stats=stats, clip_high=INF, dlogits=z,
                          dloss=torch.full((1,), float(vocab), device="cuda"))
    assert stats.tolist() == [[0.0, float(vocab)]] and abs(logp.item() - want) <= R.U * abs(want)
    r = math.exp(want + 20.0)
    # dlogits = -dloss r (onehot - q): r elsewhere, within the roundings of r, the factor, the product and the type
    tol = (8 * R.U + R.half(DT[dtype])) * r
    assert ((z[0, :-1].float() - r).abs().amax() <= tol) and abs(z[0, -1].double().item() / (-r * (vocab - 1)) - 1) <= tol / r
