"""The gated feed-forward block in every cut that its planner chooses from (tiles of 64, 128 and 256 rows, sums in one
part and in several), and on matrices of more than 2^31 elements, against the binary64 reference (tests/train_ref.py),
whose products run on the GPU here."""
import ctypes

import pytest
import torch

import bit_adamw_optimizer_amd as M
from tests import train_ref as R

DT = {"f16": torch.float16, "bf16": torch.bfloat16}

# (tokens, hidden, inner units) -> tile rows and parts (whole: 1) of the projections, dx, the weights' gradients.
# Hidden sizes that are multiples of 8 are read where they lie, the others are laid out first.
CUTS = {
    (1610, 3208, 1222): (256, 3, 256, 1, 256, 1),
    (1610, 3215, 1222): (256, 3, 256, 1, 256, 1),
    (3534, 200, 1665): (256, 1, 128, 4, 128, 4),
    (1609, 2356, 520): (128, 3, 128, 1, 128, 1),
    (2789, 401, 647): (128, 1, 64, 1, 64, 2),
    (1450, 1032, 1007): (64, 1, 256, 4, 256, 3),
    (1450, 1029, 1007): (64, 1, 256, 4, 256, 3),
    (653, 2097, 1315): (64, 2, 256, 4, 256, 1),
    (2165, 2904, 197): (64, 3, 256, 1, 256, 4),
    (803, 5459, 469): (64, 4, 256, 1, 256, 1),
    (4609, 9, 852): (64, 1, 128, 3, 128, 8),
    (327, 1081, 1423): (64, 3, 128, 8, 128, 1),
    (1359, 2534, 68): (64, 8, 128, 1, 128, 6),
    (477, 4904, 193): (64, 16, 128, 1, 128, 1),
    (130, 9, 194): (64, 1, 64, 4, 64, 2),
    (478, 8, 16): (64, 1, 64, 1, 64, 4),
    (1, 8, 194): (0, 0, 64, 4, 64, 1),
    (66, 8, 17): (64, 1, 64, 1, 64, 1),
}


def plan(t, k, f, backward):
    a = M._GatedFfn(t, k, f, 1, 0, 1 << 44, k, None, 2 << 44, k, 3 << 44, k, 4 << 44, f, 5 << 44, f, 6 << 44, k,
                    7 << 44, k, 8 << 44, k, 1, 0)
    out = (ctypes.c_int32 * 6)()
    assert M.lib().msamp_gated_ffn_plan(ctypes.byref(a), int(backward), out) == 0, M.lib().msamp_last_error()
    return tuple(out)


def test_the_sizes_reach_every_cut():
    """Each tile height whole and split: the projections, and dx beside the weights' gradients in all four pairs.
    (A new cost model may move the sizes: then others are looked for, and none of the cuts is left out.)"""
    for size, want in CUTS.items():
        assert plan(*size, True) == want, size
        assert plan(*size, False) == want[:2] + (0, 0, 0, 0), size
    p = set(CUTS.values())
    assert {(c[0], c[1] > 1) for c in p} == {(r, s) for r in (64, 128, 256) for s in (False, True)} | {(0, False)}
    assert {(c[2], c[3] > 1, c[5] > 1) for c in p} == {(r, x, w) for r in (64, 128, 256) for x in (False, True)
                                                         for w in (False, True)}
    assert plan(0, 8, 16, True) == plan(4, 0, 16, True) == plan(4, 8, 0, True) == (0,) * 6
    bad = M._GatedFfn(-1)
    assert M.lib().msamp_gated_ffn_plan(ctypes.byref(bad), 1, (ctypes.c_int32 * 6)()) == 1
    assert M.lib().msamp_gated_ffn_plan(None, 1, (ctypes.c_int32 * 6)()) == 1


def rand(rows, cols, dt, seed, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(rows, cols, dtype=dt, device="cuda")
    for i in range(0, rows, 1 << 16):  # no binary32 copy of a large matrix
        n = min(rows - i, 1 << 16)
        out[i:i + n] = torch.randn(n, cols, generator=g, device="cuda") * size
    return out


def problem(t, k, f, dt, seed):
    return (rand(t, k, dt, seed), rand(f, k, dt, seed + 1, 1.3 * k ** -0.5), rand(f, k, dt, seed + 2, 1.3 * k ** -0.5),
            rand(t, f, dt, seed + 3, 0.1))


def padded(rows, cols, dt, value=7.0):
    """A matrix inside a larger buffer, whose rest has to stay."""
    buf = torch.full((rows + 1, cols + 2), value, dtype=dt, device="cuda")
    return buf, buf[:rows, :cols]


def near(name, got, val, err, dt):
    got, val, err = got.cpu(), val.cpu(), err.cpu()
    R.assert_near(got, val, err, name)
    # in the 2-norm the roundings are as good as independent, as in test_gpu_ffn.check
    rel = ((got.double() - val).norm() / val.norm().clamp_min(1e-300)).item()
    assert rel <= 3 * R.half(dt) + (err.norm() / val.norm().clamp_min(1e-300)).item() * 0.25, (name, rel)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("t,k,f", list(CUTS))
def test_cut(t, k, f, dtype):
    dt = DT[dtype]
    assert plan(t, k, f, True) == CUTS[t, k, f]
    act = sorted(M.ACTIVATIONS)[(t + k + f + (dtype == "f16")) % 3]
    x, wg, wu, dh = problem(t, k, f, dt, t + k)
    val, err = R.ffn(x, wg, wu, act, dh, dt)
    buf, h = padded(t, f, dt)
    M.gated_ffn_forward(x, wg, wu, h, act=act)
    near("h", h, val["h"], err["h"], dt)
    assert (buf[t:] == 7).all() and (buf[:, f:] == 7).all()
    wide = None
    for wdt in (dt, torch.float32):
        bufs = {"h": padded(t, f, dt), "dx": padded(t, k, dt), "dw_gate": padded(f, k, wdt), "dw_up": padded(f, k, wdt)}
        got = {n: v[1] for n, v in bufs.items()}
        for again in (False, True):  # twice: the parts are joined in one order
            M.gated_ffn_backward(dh, x, wg, wu, got["dx"], got["dw_gate"], got["dw_up"], act=act, h=got["h"])
            if again:
                assert all(torch.equal(got[n], first[n]) for n in got)
            first = {n: v.clone() for n, v in got.items()}
        for n, (b, v) in bufs.items():
            assert (b[v.shape[0]:] == 7).all() and (b[:, v.shape[1]:] == 7).all(), n
            near(n, v, val[n], err[n], dt)
        wide = got
    a, b = torch.full((f, k), 0.5, device="cuda"), torch.full((f, k), -2.0, device="cuda")
    M.gated_ffn_backward(dh, x, wg, wu, wide["dx"], a, b, act=act, accumulate=True)
    assert torch.equal(a, 0.5 + wide["dw_gate"]) and torch.equal(b, -2.0 + wide["dw_up"])
    del x, wg, wu, dh, val, err


# x, h or a weight of more than 2^31 elements. dh is zero outside some tokens and inner units, so that the values there
# are sums of few terms, with bounds to match, and all other gradients are zero.
@pytest.mark.gpu
@pytest.mark.parametrize("t,k,f", [(70001, 72, 32776), (1048700, 2056, 40), (70, 1032, 2090003), (540000001, 8, 8)])
def test_more_than_2_to_the_31_elements(t, k, f):
    dt = torch.bfloat16
    assert max(t * k, t * f, f * k) > 1 << 31
    torch.cuda.empty_cache()
    need = 2 * (2 * t * k + 3 * t * f + 4 * f * k + 2 * t * (-(-f // 64) * 64)) * 1.1
    if torch.cuda.mem_get_info()[0] < need:  # the last: tiles of 64 rows would be more than a launch has
        pytest.skip("needs %d GB of GPU memory" % (need / 1e9))

    def some(n, *widths):
        """The rows around the element 2^31, 2^30 and 2^29 of matrices so wide, the first, the last, and others."""
        at = [e // w for e in (1 << 31, 1 << 30, 1 << 29) for w in widths] + [0, n - 1, n // 3, n // 2]
        return sorted({min(max(i + d, 0), n - 1) for i in at for d in range(-9, 10)})

    tokens, units = some(t, k, f), some(f, k)
    x, wg, wu = rand(t, k, dt, 1), rand(f, k, dt, 2, 1.3 * k ** -0.5), rand(f, k, dt, 3, 1.3 * k ** -0.5)
    dh = torch.zeros(t, f, dtype=dt, device="cuda")
    ti, ui = torch.tensor(tokens, device="cuda"), torch.tensor(units, device="cuda")
    dh[ti[:, None], ui] = rand(len(tokens), len(units), dt, 4, 0.1)
    val, err = R.ffn(x[ti], wg[ui], wu[ui], "silu", dh[ti[:, None], ui], dt)
    h, dx = torch.full_like(dh, 7.0), torch.full_like(x, 7.0)
    a, b = torch.full_like(wg, 7.0), torch.full_like(wu, 7.0)
    M.gated_ffn_forward(x, wg, wu, h)
    near("h", h[ti[:, None], ui], val["h"], err["h"], dt)
    first = h.clone()
    h.fill_(7.0)
    M.gated_ffn_backward(dh, x, wg, wu, dx, a, b, h=h)
    assert torch.equal(h, first)
    near("dx", dx[ti], val["dx"], err["dx"], dt)
    near("dw_gate", a[ui], val["dw_gate"], err["dw_gate"], dt)
    near("dw_up", b[ui], val["dw_up"], err["dw_up"], dt)
    for grad, rows in ((dx, ti), (a, ui), (b, ui)):
        grad[rows] = 0
        assert not grad.any()
    del x, dh, h, first, dx
    torch.cuda.empty_cache()
