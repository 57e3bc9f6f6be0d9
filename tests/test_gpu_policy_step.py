"""The example that uses the lookup, norm, scores and their backwards together:
its gradients against fp64 autograd of the same step, and what it learns."""
import os
import sys

import numpy as np
import pytest
import torch

import vce_run as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,H", [(200, 700, 64), (517, 3000, 128)])
def test_gradients_of_a_step(T, V, H):
    """Against autograd in fp64 on the bf16 weights. Five values are rounded to
    bf16 on the way (x, h, G, dx and de), each by at most 2^-8 of itself, and the
    gradients are linear in the last three: 6 * 2^-8 of the largest entry bounds
    them, the independent roundings of a sum's terms adding up to less."""
    import policy_step as E
    m = E.TiedPolicy(T, H, V, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    adv = torch.randn(T, generator=g, device="cuda")
    old = m.scores(ids, y).clone() + 0.05 * torch.randn(T, generator=g, device="cuda")
    m.gradient(ids, y, old, adv)
    torch.cuda.synchronize()
    assert int(m.status.item()) == 0
    W = m.W[:V].double().cpu().requires_grad_()
    w = torch.ones(H, dtype=torch.float64, requires_grad=True)
    b = torch.zeros(H, dtype=torch.float64, requires_grad=True)
    M = m.M.double().cpu().requires_grad_()
    x = W[ids.cpu()] @ M
    h = torch.nn.functional.layer_norm(x, (H,), w, b, 1e-5)
    lp = torch.log_softmax(h @ W.T, 1)
    logp = lp[torch.arange(T), y.cpu()]
    assert (logp.detach() - m.logp.cpu()).abs().max() < 0.02
    ent = -(lp.exp() * lp).sum(1)
    r = torch.exp(logp - old.double().cpu())
    a = adv.double().cpu()
    obj = torch.minimum(r * a, r.clamp(0.8, 1.2) * a).mean() + 0.01 * ent.mean()
    (-obj).backward()
    for got, want in ((m.dW[:V], W.grad), (m.dM, M.grad), (m.dnw, w.grad), (m.dnb, b.grad)):
        err = (got.double().cpu() - want).abs().max() / want.abs().max()
        assert err <= 6 * 2.0 ** -8, float(err)
    assert not m.dW[V:].any().item()


def test_learns_and_decodes():
    import policy_step as E
    m = E.train()
    first = torch.arange(32, device="cuda")
    ids, top, top_logp, entropy = m.decode(first, 3)
    assert int(m.status.item()) == 0
    ok = ((7 * ids[:, :-1] + 3) % 1000 == ids[:, 1:]).float().mean().item()
    assert ok > 0.9, ok
    assert torch.equal(top[:, 0], ids[:, -1])
    assert bool((top_logp[:, :-1] >= top_logp[:, 1:]).all()) and bool((entropy >= 0).all())
    assert np.isfinite(top_logp.cpu().numpy()).all()
