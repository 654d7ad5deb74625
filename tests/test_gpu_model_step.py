"""A whole training step from the library's operators: tokens through the
embedding, a norm, the recurrence, the gated block and the tied output
projection to a loss, all gradients back, and the optimizer step on them. Each
stage is compared with its binary64 reference on the stage's own inputs."""
import numpy as np
import pytest
import torch

import bit_adamw_optimizer_amd as M
import oracle as O
from tests import model_ref as R
from tests import train_ref as T

pytestmark = pytest.mark.gpu

B, S, K, F, V, TOP = 2, 75, 48, 96, 211, 6
N = B * S


def near(val, err, got):
    for name, g in got.items():
        R.assert_near(g, val[name], err[name], name)


@pytest.mark.parametrize("loss_of", ["distill", "policy"])
def test_tokens_to_the_optimizer_step(loss_of):
    f16 = torch.float16
    g = torch.Generator().manual_seed(5)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    ids = torch.randint(0, V, (N,), generator=g)
    ids[-9:] = -1  # the second sequence is shorter
    ids = ids.cuda()
    lengths = torch.tensor([S, S - 9], device="cuda")
    sizes = [("embedding", (V, K), 0.5, 0.0), ("gamma", (K,), 0.1, 1.0), ("mix", (2 * K, K), K ** -0.5, 0.0),
             ("gate", (F, K), K ** -0.5, 0.0), ("up", (F, K), K ** -0.5, 0.0), ("down", (K, F), F ** -0.5, 0.0)]
    weights = [(randn(int(np.prod(s))) * size + mean).to(f16).cuda() for _, s, size, mean in sizes]
    w = {name: v.view(s) for (name, s, _, _), v in zip(sizes, weights)}
    grads = [torch.zeros(v.numel(), device="cuda") for v in weights]
    d = {name: v.view(s) for (name, s, _, _), v in zip(sizes, grads)}
    st = M.allocate_state(weights, "O2")
    codes, gmeta = [torch.empty(v.numel(), dtype=torch.uint8, device="cuda") for v in weights], M.new_meta(len(weights), "cuda")
    new = lambda *s: torch.zeros(*s, dtype=f16, device="cuda")  # noqa: E731

    # forward
    x, xn, rstd = new(N, K), new(N, K), torch.empty(N, device="cuda")
    M.embedding_forward(ids, w["embedding"], x, scale=2.0)
    M.layernorm_forward(x, w["gamma"], None, xn, None, rstd)
    p = (xn.float() @ w["mix"].float().t()).to(f16).view(B, S, 2 * K)  # inputs and gates in one projection
    y, states = new(B, S, K), M.new_recurrence_states(B, S, K)
    M.recurrence_forward(p[..., :K], p[..., K:], y, states=states, lengths=lengths)
    h = new(N, F)
    M.gated_ffn_forward(y.view(N, K), w["gate"], w["up"], h)
    o = (h.float() @ w["down"].float().t()).to(f16)
    z = (o.float() @ w["embedding"].float().t()).to(f16)

    # loss and its gradient in one pass
    loss, dz, dloss = torch.empty(N, device="cuda"), new(N, V), torch.full((N,), 256.0 / N, device="cuda")
    t, cls = (randn(N, V) * 2).topk(TOP, 1)
    cls[torch.arange(N) >= N - 9] = -1
    t, cls = t.cuda(), cls.cuda()
    act, lp = cls[:, 0].contiguous(), torch.log_softmax(z.double(), 1)
    old = (lp.gather(1, act.clamp_min(0)[:, None])[:, 0] + 0.05).float()
    adv = randn(N).cuda()
    if loss_of == "distill":
        M.distill_loss_forward(z, cls, t, loss, temperature=1.5, dlogits=dz, dloss=dloss)
        val, err = R.distill(z.cpu(), cls.cpu(), t.cpu(), 1.5, dloss.cpu())
    else:
        M.policy_loss_forward(z, act, old, adv, loss, dlogits=dz, dloss=dloss, ref_logp=old, kl=0.1)
        val, err, clear = R.policy(z.cpu(), act.cpu(), old.cpu(), adv.cpu(), 1.0, old.cpu(), 0.1, dloss=dloss.cpu())
        assert clear.min() > 1e-5
    near(val, err, {"loss": loss, "dlogits": dz})
    assert (loss[-9:] == 0).all() and not dz[-9:].any()

    # backward
    do = (dz.float() @ w["embedding"].float()).to(f16)
    d["embedding"].copy_(dz.float().t() @ o.float())
    tied = d["embedding"].clone()
    dh = (do.float() @ w["down"].float()).to(f16)
    d["down"].copy_(do.float().t() @ h.float())
    dy, dp, dxn, dx = new(N, K), new(B, S, 2 * K), new(N, K), new(N, K)
    M.gated_ffn_backward(dh, y.view(N, K), w["gate"], w["up"], dy, d["gate"], d["up"])
    M.recurrence_backward(dy.view(B, S, K), p[..., :K], p[..., K:], states, dp[..., :K], dp[..., K:], lengths=lengths)
    dxn.copy_(dp.view(N, 2 * K).float() @ w["mix"].float())
    d["mix"].copy_(dp.view(N, 2 * K).float().t() @ xn.float())
    M.layernorm_backward(dxn, x, w["gamma"], None, rstd, dx, d["gamma"], None)
    M.embedding_backward(dx, ids, d["embedding"], scale=2.0, accumulate=True)
    before = [v.clone() for v in weights]
    M.amax(grads, gmeta)
    M.quantize_adamw_o2_step(grads, M.E4M3, gmeta, codes, st["exp_avg"], st["exp_avg_meta"], st["exp_avg_sq"], weights,
                             lr=1e-3, step=1)
    torch.cuda.synchronize()
    c = {name: v.view(s).cpu() for (name, s, _, _), v in zip(sizes, before)}

    # every new stage against its reference
    ref, bound = R.embedding_forward(ids.cpu(), c["embedding"], 2.0)
    R.assert_near(x, ref, bound, "x")
    n, pc = lengths.cpu(), p.cpu()
    hs, errs = R.recurrence_forward(pc[..., :K], pc[..., K:], lengths=n)
    live = (torch.arange(S)[None] < n[:, None])[..., None].expand(B, S, K)
    R.assert_near(y.cpu()[live], hs[:, 1:][live], errs[:, 1:][live], "y")
    assert not y.cpu()[~live].any()
    val, err = R.recurrence_backward(dy.view(B, S, K).cpu(), pc[..., :K], pc[..., K:], states.cpu(), lengths=n)
    R.assert_near(dp[..., :K].cpu()[live], val["dx"][live], err["dx"][live], "dx of the recurrence")
    R.assert_near(dp[..., K:].cpu()[live], val["dgate"][live], err["dgate"][live], "dgate")
    assert not dp.cpu()[1, S - 9:].any()
    ref, bound = R.embedding_backward(dx.cpu(), ids.cpu(), V, 2.0, tied.cpu())
    R.assert_near(d["embedding"], ref, bound, "dweight of the embedding")
    ref = T.norm_backward(dxn.cpu(), x.cpu(), c["gamma"].double(), None, rstd.cpu(), False)
    R.assert_near(dx, ref[0], ref[3], "dx of the norm")
    # and the step on these gradients against the oracle
    for i, v in enumerate(weights):
        s = O.TensorState(before[i].view(torch.int16).cpu().numpy().view(np.uint16).copy(), "O2")
        O.step_tensor(s, grads[i].cpu().numpy(), O.E4M3, 1, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)
        assert np.array_equal(v.view(torch.int16).cpu().numpy().view(np.uint16), s.w)
