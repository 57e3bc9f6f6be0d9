"""Oracle for the token scores (log probabilities, entropy, top alternatives),
their gradient, and the normalisation in front of the head: plain fp64 CPU
definitions.

TEST INFRASTRUCTURE, as vce_oracle.py: it never imports the CUDA path and is
never imported by it. Arrays of uint16 are read as bf16 bit patterns.
"""
from __future__ import annotations

import numpy as np


def as_f64(x) -> np.ndarray:
    x = np.asarray(x)
    if x.dtype == np.uint16:
        return (x.astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)
    return x.astype(np.float64)


def valid_targets(targets, V_real: int) -> np.ndarray:
    y = np.asarray(targets)
    return (y >= 0) & (y < V_real)


def token_scores(h, W, targets, V_real: int, scale: float = 1.0, n_top: int = 0):
    """Per token: lse, logp of the target and entropy (both 0 without a real
    target; entropy of every token when targets is None), and the n_top classes
    of the largest logits, the lower class first between equal ones."""
    z = as_f64(h) @ as_f64(W)[:V_real].T
    lz = scale * z
    m = lz.max(axis=1, keepdims=True)
    lse = (m + np.log(np.exp(lz - m).sum(axis=1, keepdims=True)))[:, 0]
    logprob = lz - lse[:, None]
    p = np.exp(logprob)
    ent = -np.where(p > 0, p * logprob, 0.0).sum(axis=1)
    out = dict(z=z, lse=lse, logprob=logprob)
    if targets is None:
        out.update(logp=None, entropy=ent)
    else:
        ok = valid_targets(targets, V_real)
        y = np.where(ok, targets, 0)
        out["logp"] = np.where(ok, logprob[np.arange(len(y)), y], 0.0)
        out["entropy"] = np.where(ok, ent, 0.0)
    # a stable sort of the negated logits keeps the lower class first
    out["top_ids"] = np.argsort(-z, axis=1, kind="stable")[:, :n_top].astype(np.int64)
    out["top_logp"] = np.take_along_axis(logprob, out["top_ids"], axis=1)
    return out


def score_logit_gradient(h, W, targets, V_real: int, g_logp=None, g_entropy=None, scale: float = 1.0, lse=None,
                         entropy=None) -> np.ndarray:
    """d/dz of sum_t g_logp logp + g_entropy entropy, z the unscaled logits; lse
    and entropy as given, or of these inputs."""
    s = token_scores(h, W, None, V_real, scale)
    lp = s["logprob"] if lse is None else scale * s["z"] - as_f64(lse)[:, None]
    if entropy is not None:
        s["entropy"] = as_f64(entropy)
    p = np.exp(lp)
    T = lp.shape[0]
    ok = np.ones(T, bool) if targets is None else valid_targets(targets, V_real)
    ge = np.zeros(T) if g_entropy is None else np.where(ok, g_entropy, 0.0)
    G = -ge[:, None] * p * (lp + s["entropy"][:, None])
    if g_logp is not None:
        gl = np.where(ok, g_logp, 0.0)
        G -= gl[:, None] * p
        G[np.arange(T), np.where(ok, targets, 0)] += gl
    return scale * G


def score_backward(h, W, targets, V_real: int, g_logp=None, g_entropy=None, scale: float = 1.0, lse=None,
                   entropy=None):
    """(dH [T,H], dW [Vp,H]); rows of h without a real target take no part."""
    hf, Wf = as_f64(h), as_f64(W)
    G = score_logit_gradient(h, W, targets, V_real, g_logp, g_entropy, scale, lse, entropy)
    dW = np.zeros_like(Wf)
    dW[:V_real] = G.T @ hf
    return G @ Wf[:V_real], dW


def norm_forward(x, weight=None, bias=None, eps: float = 1e-5, rms: bool = False):
    xf = as_f64(x)
    mean = np.zeros(xf.shape[0]) if rms else xf.mean(axis=1)
    d = xf - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * as_f64(weight)
    if bias is not None:
        y = y + as_f64(bias)
    return y, mean, rstd


def norm_backward(x, weight, dy, mean, rstd, rms: bool = False):
    """(dx, dweight, dbias) from the forward's statistics."""
    xhat = (as_f64(x) - (0.0 if rms else np.asarray(mean, np.float64)[:, None])) * np.asarray(rstd, np.float64)[:, None]
    d = as_f64(dy)
    g = d if weight is None else d * as_f64(weight)
    dx = g - xhat * (g * xhat).mean(axis=1, keepdims=True)
    if not rms:
        dx = dx - g.mean(axis=1, keepdims=True)
    return dx * np.asarray(rstd, np.float64)[:, None], (d * xhat).sum(axis=0), d.sum(axis=0)
