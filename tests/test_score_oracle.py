"""The token-score and norm oracle against differences, autograd and brute force (CPU)."""
import numpy as np
import pytest
import torch

from oracle import score_oracle as S


def _case(seed, T=5, H=6, V=11, Vp=64):
    rng = np.random.default_rng(seed)
    h, W = rng.standard_normal((T, H)), rng.standard_normal((Vp, H))
    W[V:] = np.nan                                   # padding rows hold anything
    y = rng.integers(0, V, T)
    y[1] = -100
    return rng, h, W, y


@pytest.mark.parametrize("scale", [1.0, 0.5, 1.7])
def test_scores_against_torch(scale):
    _, h, W, y = _case(1)
    V = 11
    r = S.token_scores(h, W, y, V, scale, 4)
    lp = torch.log_softmax(scale * torch.from_numpy(h) @ torch.from_numpy(W[:V]).T, dim=1)
    ent = torch.distributions.Categorical(logits=lp).entropy().numpy()
    ok = y >= 0
    assert np.allclose(r["logp"][ok], lp.numpy()[np.nonzero(ok)[0], y[ok]], atol=1e-13) and r["logp"][1] == 0
    assert np.allclose(r["entropy"][ok], ent[ok], atol=1e-13) and r["entropy"][1] == 0
    top = torch.topk(lp, 4, dim=1)
    assert np.array_equal(r["top_ids"], top.indices.numpy())
    assert np.allclose(r["top_logp"], top.values.numpy(), atol=1e-13)


def test_ties_go_to_the_lower_class():
    W = np.zeros((64, 2))
    W[[3, 7, 9], 0] = 1.0
    r = S.token_scores(np.ones((1, 2)), W, None, 12, 1.0, 5)
    assert r["top_ids"].tolist() == [[3, 7, 9, 0, 1]]


@pytest.mark.parametrize("terms", ["logp", "entropy", "both"])
def test_gradient_against_differences(terms):
    rng, h, W, y = _case(2)
    V, s = 11, 1.3
    gl = rng.standard_normal(5) if terms != "entropy" else None
    ge = rng.standard_normal(5) if terms != "logp" else None
    dH, dW = S.score_backward(h, W, y, V, gl, ge, s)

    def f(h, W):
        r = S.token_scores(h, W, y, V, s)
        return (0 if gl is None else gl @ r["logp"]) + (0 if ge is None else ge @ r["entropy"])

    e = 1e-6
    for M, g, rows in ((h, dH, 5), (W, dW, V)):
        for i in range(rows):
            for j in range(6):
                keep = M[i, j]
                M[i, j] = keep + e
                up = f(h, W)
                M[i, j] = keep - e
                down = f(h, W)
                M[i, j] = keep
                assert abs((up - down) / (2 * e) - g[i, j]) < 1e-7
    assert not dW[V:].any() and not dH[1].any()


def test_targetless_gradient_is_the_entropy_of_every_token():
    rng, h, W, _ = _case(3)
    hh = torch.from_numpy(h).requires_grad_()
    lp = torch.log_softmax(hh @ torch.from_numpy(W[:11]).T, dim=1)
    ge = torch.from_numpy(rng.standard_normal(5))
    (-(lp.exp() * lp).sum(1) * ge).sum().backward()
    dH, _ = S.score_backward(h, W, None, 11, None, ge.numpy())
    assert np.allclose(dH, hh.grad.numpy(), atol=1e-13)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_against_autograd(rms):
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((4, 9)) + 0.5).requires_grad_()
    w = torch.from_numpy(rng.standard_normal(9)).requires_grad_()
    b = torch.from_numpy(rng.standard_normal(9)).requires_grad_()
    dy = rng.standard_normal((4, 9))
    if rms:
        y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5) * w + b
    else:
        y = torch.nn.functional.layer_norm(x, (9,), w, b, 1e-5)
    y.backward(torch.from_numpy(dy))
    xn, wn, bn = (t.detach().numpy() for t in (x, w, b))
    yo, mean, rstd = S.norm_forward(xn, wn, bn, 1e-5, rms)
    assert np.allclose(yo, y.detach().numpy(), atol=1e-13)
    dx, dw, db = S.norm_backward(xn, wn, dy, mean, rstd, rms)
    for got, want in ((dx, x), (dw, w), (db, b)):
        assert np.allclose(got, want.grad.numpy(), atol=1e-13)
