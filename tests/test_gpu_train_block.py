"""The training operators together, as a step uses them: a normed gated
feed-forward block that keeps one 8-bit checkpoint, its backward pass from
that checkpoint, and the optimizer step on the gradients it produces."""
import numpy as np
import pytest
import torch

import bit_adamw_optimizer_amd as M
import oracle as O
from tests import train_ref as R

pytestmark = pytest.mark.gpu

T, K, F = 190, 144, 328


def test_block_from_one_checkpoint_into_the_optimizer_step():
    f16 = torch.float16
    g = torch.Generator().manual_seed(11)
    x = (torch.randn(T, K, generator=g) * 2).to(f16).cuda()
    # parameters of the O2 layout: FP16, flat, viewed as matrices by the block
    weights = [(torch.randn(n, generator=g) * s + m).to(f16).cuda() for n, s, m in
               ((K, 0.1, 1.0), (K, 0.1, 0.0), (F * K, 1.3 * K ** -0.5, 0.0), (F * K, 1.3 * K ** -0.5, 0.0))]
    gamma, beta, wg, wu = weights[0], weights[1], weights[2].view(F, K), weights[3].view(F, K)
    dh = (torch.randn(T, F, generator=g) * 0.05).to(f16).cuda()
    st = M.allocate_state(weights, "O2")
    grads = [torch.empty(w.numel(), device="cuda") for w in weights]
    codes = [torch.empty(w.numel(), dtype=torch.uint8, device="cuda") for w in weights]
    gmeta = M.new_meta(4, "cuda")
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    y, h = torch.empty_like(x), torch.empty(T, F, dtype=f16, device="cuda")

    # forward: one checkpoint is all that stays
    ck = M.new_checkpoint(T, K)
    M.layernorm_forward(x, gamma, beta, y, mean, rstd, save=ck)
    M.gated_ffn_forward(y, wg, wu, h)

    # backward: the norm's output again from the checkpoint, then both gradients
    y2, m2, r2 = torch.empty_like(x), torch.empty_like(mean), torch.empty_like(rstd)
    M.layernorm_forward(ck, gamma, beta, y2, m2, r2)
    dy, dx, h2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(h)
    M.gated_ffn_backward(dh, y2, wg, wu, dy, grads[2].view(F, K), grads[3].view(F, K), h=h2)
    M.layernorm_backward(dy, ck, gamma, m2, r2, dx, grads[0], grads[1])
    M.amax(grads, gmeta)
    before = [w.clone() for w in weights]
    M.quantize_adamw_o2_step(grads, M.E4M3, gmeta, codes, st["exp_avg"], st["exp_avg_meta"], st["exp_avg_sq"],
                             weights, lr=1e-3, step=1)
    torch.cuda.synchronize()

    # each stage against its reference, on the stage's own inputs
    gd, bd = before[0].cpu().double(), before[1].cpu().double()
    ry, _, _, bound = R.norm_forward(x.cpu(), gd, bd, 1e-5, True)
    R.assert_near(y, ry, bound, "y")
    val, err = R.ffn(y.cpu(), before[2].view(F, K).cpu(), before[3].view(F, K).cpu(), "silu", dtype=f16)
    R.assert_near(h, val["h"], err["h"], "h")
    rc, rs = R.checkpoint_save(x.float().cpu().numpy(), M.E4M3)
    xv = torch.from_numpy(R.checkpoint_values(rc, rs, M.E4M3))
    ry2, _, _, bound = R.norm_forward(xv, gd, bd, 1e-5, True)
    R.assert_near(y2, ry2, bound, "y from the checkpoint")
    val, err = R.ffn(y2.cpu(), before[2].view(F, K).cpu(), before[3].view(F, K).cpu(), "silu", dh.cpu(), f16)
    for name, got in (("h", h2), ("dx", dy), ("dw_gate", grads[2].view(F, K)), ("dw_up", grads[3].view(F, K))):
        R.assert_near(got, val[name], err[name], name)
    ref = R.norm_backward(dy.cpu(), xv, gd, m2.cpu(), r2.cpu(), True)
    for name, got, r, e in zip(("dx", "dweight", "dbias"), (dx, grads[0], grads[1]), ref[:3], ref[3:]):
        R.assert_near(got, r, e, name)
    # and the step on these gradients against the oracle
    for i, w in enumerate(weights):
        s = O.TensorState(before[i].view(torch.int16).cpu().numpy().view(np.uint16).copy(), "O2")
        O.step_tensor(s, grads[i].cpu().numpy(), O.E4M3, 1, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)
        assert np.array_equal(w.view(torch.int16).cpu().numpy().view(np.uint16), s.w)
