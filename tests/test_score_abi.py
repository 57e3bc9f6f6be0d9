"""Refusals of the token-score and norm entry points, on the host (no GPU):
every call below fails validation before anything is enqueued."""
import ctypes
import os

import pytest
import torch

from vocab_embedding_cross_gb300 import _lib as vce

FAKE = 1 << 20   # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(vce.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return vce.lib()


def P(**kw):
    base = dict(T=64, H=64, Vp=1024, V_real=1000, S=4, dtype=vce.VCE_BF16)
    base.update(kw)
    return vce.problem(**base)


def fwd(L, p, h=FAKE, W=FAKE, y=FAKE, scale=1.0, K=4, logp=FAKE, ent=FAKE, lse=FAKE, ids=FAKE, tlp=FAKE, ws=FAKE,
        nb=1 << 40):
    return L.vce_logprob_fwd(ctypes.byref(p), h, W, y, scale, K, logp, ent, lse, ids, tlp, ws, nb, None, None)


def bwd(L, p, h=FAKE, W=FAKE, y=FAKE, lse=FAKE, ent=FAKE, gl=FAKE, ge=FAKE, scale=1.0, dH=FAKE, dW=FAKE, dwt=None,
        ws=FAKE, nb=1 << 40):
    return L.vce_logprob_bwd(ctypes.byref(p), h, W, y, lse, ent, gl, ge, scale, dH, dW,
                             vce.VCE_F32 if dwt is None else dwt, ws, nb, None, None)


def nfwd(L, p, kind=0, x=FAKE, w=FAKE, b=FAKE, eps=1e-5, y=FAKE, mean=FAKE, rstd=FAKE):
    return L.vce_norm_fwd(ctypes.byref(p), kind, x, w, b, eps, y, mean, rstd, None, None)


def nbwd(L, p, kind=0, x=FAKE, w=FAKE, dy=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, db=FAKE, acc=0, ws=FAKE,
         nb=1 << 40):
    return L.vce_norm_bwd(ctypes.byref(p), kind, x, w, dy, mean, rstd, dx, dw, db, acc, ws, nb, None, None)


@pytest.mark.parametrize("call", [fwd, bwd, nfwd, nbwd])
@pytest.mark.parametrize("kw,code", [(dict(Vp=1000), vce.VCE_ERR_ARG), (dict(H=4), vce.VCE_ERR_UNSUPPORTED),
                                     (dict(T=-1), vce.VCE_ERR_ARG), (dict(dtype=7), vce.VCE_ERR_UNSUPPORTED),
                                     (dict(flags=4), vce.VCE_ERR_ARG), (dict(ignore_index=3), vce.VCE_ERR_ARG)])
def test_bad_problem(L, call, kw, code):
    assert call(L, P(**kw)) == code
    assert vce.vce_logprob_workspace_size(P(**kw), 4) == vce.SIZE_MAX
    for op in (vce.VCE_OP_LOGPROB_BWD, vce.VCE_OP_NORM_BWD):
        assert vce.vce_workspace_size(P(**kw), op) == vce.SIZE_MAX
        assert vce.vce_workspace_size_min(P(**kw), op) == vce.SIZE_MAX


def test_forward_refusals(L):
    p, A, U, WS = P(), vce.VCE_ERR_ARG, vce.VCE_ERR_UNSUPPORTED, vce.VCE_ERR_WORKSPACE
    for K in (-1, 33, 1001):
        assert fwd(L, p, K=K) == A
        assert vce.vce_logprob_workspace_size(p, K) == vce.SIZE_MAX
    small = P(Vp=64, V_real=7)
    assert fwd(L, small, K=8) == A and vce.vce_logprob_workspace_size(small, 8) == vce.SIZE_MAX
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(L, p, scale=s) == A
    assert fwd(L, p, h=None) == A and fwd(L, p, W=None) == A
    assert fwd(L, p, y=None) == A                                # a log probability of no target
    assert fwd(L, p, ids=None) == A and fwd(L, p, tlp=None) == A
    assert fwd(L, p, h=FAKE + 8) == U and fwd(L, p, y=FAKE + 4) == U and fwd(L, p, ids=FAKE + 4) == U
    assert fwd(L, p, lse=FAKE + 2) == U
    need = vce.vce_logprob_workspace_size(p, 4)
    assert fwd(L, p, ws=None) == WS and fwd(L, p, nb=need - 1) == WS and fwd(L, p, ws=FAKE + 16) == WS
    assert fwd(L, P(T=0), h=None, W=None, y=None, ws=None, nb=0) == vce.VCE_OK


def test_backward_refusals(L):
    p, A, U, WS = P(), vce.VCE_ERR_ARG, vce.VCE_ERR_UNSUPPORTED, vce.VCE_ERR_WORKSPACE
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert bwd(L, p, scale=s) == A
    for k in ("h", "W", "lse", "dH", "dW"):
        assert bwd(L, p, **{k: None}) == A
    assert bwd(L, p, gl=None, ge=None) == A                      # the gradient of nothing
    assert bwd(L, p, y=None) == A                                # g_logp without targets
    assert bwd(L, p, ent=None) == A                              # g_entropy without the entropy
    assert bwd(L, p, dwt=5) == U
    assert bwd(L, P(tied=True), dwt=vce.VCE_BF16) == U           # added into: fp32 only
    assert bwd(L, P(dtype=vce.VCE_F32), dwt=vce.VCE_BF16) == U
    assert bwd(L, p, dH=FAKE + 8) == U and bwd(L, p, dW=FAKE + 8) == U and bwd(L, p, gl=FAKE + 2) == U
    for q in (p, P(flags=vce.VCE_FLAG_DH_BF16)):
        mn = vce.vce_workspace_size_min(q, vce.VCE_OP_LOGPROB_BWD)
        assert vce.vce_workspace_size(q, vce.VCE_OP_LOGPROB_BWD) > mn
        assert bwd(L, q, nb=mn - 256) == WS and bwd(L, q, nb=0) == WS
        assert bwd(L, q, ws=None) == WS and bwd(L, q, ws=FAKE + 16) == WS
    assert bwd(L, P(T=0, tied=True), h=None, W=None, ws=None, nb=0) == vce.VCE_OK


def test_norm_refusals(L):
    p, A, U, WS = P(), vce.VCE_ERR_ARG, vce.VCE_ERR_UNSUPPORTED, vce.VCE_ERR_WORKSPACE
    assert nfwd(L, p, kind=2) == A and nbwd(L, p, kind=-1) == A
    for e in (-1e-9, float("nan"), float("inf")):
        assert nfwd(L, p, eps=e) == A
    assert nfwd(L, p, x=None) == A and nfwd(L, p, y=None) == A
    assert nfwd(L, p, x=FAKE + 8) == U and nfwd(L, p, w=FAKE + 8) == U and nfwd(L, p, mean=FAKE + 2) == U
    assert nbwd(L, p, acc=2) == A and nbwd(L, p, dx=None, dw=None, db=None) == A
    assert nbwd(L, p, x=None) == A and nbwd(L, p, dy=None) == A and nbwd(L, p, rstd=None) == A
    assert nbwd(L, p, mean=None) == A                            # layer norm needs it
    assert nbwd(L, p, dy=FAKE + 8) == U and nbwd(L, p, dw=FAKE + 4) == U
    need = vce.vce_workspace_size(p, vce.VCE_OP_NORM_BWD)
    assert nbwd(L, p, nb=need - 1) == WS and nbwd(L, p, ws=None) == WS and nbwd(L, p, ws=FAKE + 16) == WS
    assert nfwd(L, P(T=0), x=None, y=None) == vce.VCE_OK
    assert nbwd(L, P(T=0), x=None, dw=None, db=None) == vce.VCE_OK


def test_binding_checks_tensors():
    """Wrong element types, shapes, orders and devices are refused by name before the call."""
    p = P(T=4, H=64, Vp=64, V_real=50)
    ok = dict(dtype=torch.float32)
    with pytest.raises(ValueError, match="h: expected a contiguous CUDA tensor"):
        vce.vce_logprob_fwd(p, torch.zeros(4, 64, dtype=torch.bfloat16), None, None, ws=None)
    with pytest.raises(ValueError, match="h is required"):
        vce.vce_logprob_fwd(p, None, None, None, ws=None)
    with pytest.raises(ValueError, match="x: expected"):
        vce.vce_norm_fwd(p, torch.zeros(4, 64, **ok), None, None, None)
