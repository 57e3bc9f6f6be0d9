"""Token scores (vce_logprob_fwd) and their gradient (vce_logprob_bwd) against the fp64 oracle.

Most inputs lie on a coarse grid (steps of 1/4 and 1/128, at most eight bits):
every logit is then exact in fp32 whatever the order of summation, so the ids
of the alternatives must equal the oracle's and errors come from the
exponentials, the sums and the stated roundings alone.

Tolerances. u = 2^-24. With A the largest |scaled logit| of the case, exp(l - m)
is off by at most e = (4 A + 8) u relatively (rounding of the scaled logit and
of the exponent's argument, and the exponential itself). A sum of one sign
over chains of at most 2048 terms adds 2048 u. So S and U are off by
r = e + 2200 u relatively, lse and logp by r + 4 A u absolutely, and entropy =
log S - U/S by 2 r (1 + |U/S|).
Gradient: with Gabs the sum of the magnitudes of G's terms, G is off by
(2 e + 2 A u + 64 u) Gabs plus, in bf16, 2^-8 |G|; a product over n terms adds
n u. The result's own rounding adds 2^-8 of it in bf16.
"""
import numpy as np
import pytest
import torch

import vce_run as R
from oracle import score_oracle as S
from vocab_embedding_cross_gb300 import device as D
from vocab_embedding_cross_gb300 import inputs as I

pytestmark = pytest.mark.gpu
vce = R.vce
U24 = 2.0 ** -24


def store(x, dtype):
    return I.bf16_bits(x.astype(np.float32)) if dtype == "bf16" else np.ascontiguousarray(x, np.float32)


def grid_case(T, H, V, dtype, seed=0, pad=np.nan, ignore=0.1, lean=None):
    rng = np.random.default_rng([seed, T, H, V])
    Vp = -(-V // 64) * 64
    w = np.clip(np.round(rng.standard_normal((Vp, H)) * 8), -127, 127)
    y = np.minimum((V ** rng.random(T)).astype(np.int64) - 1, V - 1).clip(0)
    a = rng.random((T, 1)) * (min(0.5, 120.0 / H) if lean is None else lean)
    h = np.clip(np.round(rng.standard_normal((T, H)) * 4 + a * w[y]), -127, 127)
    w /= 128
    w[V:] = pad                                   # rows that are never read
    y[rng.random(T) < ignore] = -100
    return store(h / 4, dtype), store_nan(w, dtype), y, Vp


def store_nan(w, dtype):
    out = store(np.nan_to_num(w), dtype)
    out[np.isnan(w)] = 0x7FC0 if dtype == "bf16" else np.nan
    return out


def problem(dtype, T, H, Vp, V, S_=4, **kw):
    return vce.problem(T, H, Vp, V, S_, vce.VCE_BF16 if dtype == "bf16" else vce.VCE_F32, **kw)


def run_fwd(dtype, h, W, y, V, Vp, K, scale, S_=4, status=0):
    T, H = h.shape
    p = problem(dtype, T, H, Vp, V, S_)
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    out = dict(logp=nan(T) if y is not None else None, entropy=nan(T), lse=nan(T))
    out["top_ids"] = torch.full((T, K), -7, dtype=torch.int64, device="cuda") if K else None
    out["top_logp"] = nan(T, K) if K else None
    st = R.status_word()
    ws = D.workspace(vce.vce_logprob_workspace_size(p, K))
    ws.fill_(0xFF)                                # scratch holds anything before the call
    yd = None if y is None else torch.from_numpy(y).cuda()
    vce.vce_logprob_fwd(p, D.to_device(h), D.to_device(W), yd, **out, logit_scale=scale, ws=ws, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return {k: (None if v is None else v.cpu().numpy()) for k, v in out.items()}


def check_fwd(got, ref, scale, K, rows=None, ids=True):
    A = np.abs(scale * ref["z"]).max()
    e = (4 * A + 8) * U24
    r = e + 2200 * U24
    ratio = np.abs(ref["entropy"]) + 40           # |U/S| = log S - entropy < log V + entropy
    sl = slice(None) if rows is None else rows
    assert np.all(np.abs(got["lse"] - ref["lse"])[sl] <= r + 4 * A * U24)
    if ref["logp"] is not None:
        assert np.all(np.abs(got["logp"] - ref["logp"])[sl] <= r + 8 * A * U24)
    assert np.all((np.abs(got["entropy"] - ref["entropy"]) <= 2 * r * (1 + ratio))[sl])
    if K:
        if ids:
            assert np.array_equal(got["top_ids"][sl], ref["top_ids"][sl])
        assert np.all(np.abs(got["top_logp"] - ref["top_logp"])[sl] <= r + 8 * A * U24)


SIZES = [  # T, H, V, S, K, scale
    (1, 64, 1, 1, 1, 1.0), (1, 8, 40, 1, 32, 1.0), (1, 2048, 1000, 8, 20, 1.0), (2, 72, 33, 2, 32, 0.5),
    (3, 64, 4001, 4, 20, 1.7), (15, 128, 257, 3, 5, 1.0), (16, 256, 5000, 8, 8, 1.0), (17, 200, 2049, 7, 20, 1.25),
    (33, 64, 20000, 8, 32, 1.0), (48, 1024, 3000, 8, 5, 1.0), (64, 64, 1000, 4, 10, 1.0), (65, 136, 6500, 5, 1, 1.0),
    (127, 64, 4100, 2, 0, 1.0), (128, 64, 4096, 1, 17, 1.0), (129, 256, 9999, 8, 20, 1 / 0.7),
    (200, 64, 50001, 8, 32, 1.0), (255, 128, 7000, 8, 2, 0.5), (257, 320, 12000, 8, 20, 1.0),
    (520, 64, 30011, 8, 24, 1.0), (1030, 128, 8200, 8, 20, 1.0),
]


@pytest.mark.parametrize("T,H,V,S_,K,scale", SIZES)
def test_scores_bf16(T, H, V, S_, K, scale):
    h, W, y, Vp = grid_case(T, H, V, "bf16", seed=1)
    ref = S.token_scores(h, W, y, V, scale, K)
    check_fwd(run_fwd("bf16", h, W, y, V, Vp, K, scale, S_), ref, scale, K)


@pytest.mark.parametrize("T,H,V,S_,K,scale", [(1, 4, 1, 1, 1, 1.0), (1, 64, 1000, 4, 20, 1.0), (64, 64, 1000, 4, 10, 1.0),
                                              (70, 100, 65, 2, 32, 0.5), (130, 36, 5003, 7, 20, 1 / 0.7),
                                              (257, 64, 2000, 8, 0, 1.0)])
def test_scores_f32(T, H, V, S_, K, scale):
    h, W, y, Vp = grid_case(T, H, V, "f32", seed=2)
    ref = S.token_scores(h, W, y, V, scale, K)
    check_fwd(run_fwd("f32", h, W, y, V, Vp, K, scale, S_), ref, scale, K)


@pytest.mark.parametrize("dtype,T", [("bf16", 5), ("bf16", 300), ("f32", 70)])
def test_scores_off_the_grid(dtype, T):
    """Ordinary values: a logit is off by at most H u sum |h||w| besides, and an
    alternative's logit by as much (the ids of close ones may change places)."""
    H, V, Vp, K = 256, 3000, 3008, 12
    rng = np.random.default_rng(9)
    h, W = store(rng.standard_normal((T, H)), dtype), store(rng.standard_normal((Vp, H)) * 0.1, dtype)
    y = rng.integers(0, V, T)
    ref = S.token_scores(h, W, y, V, 1.0, K)
    got = run_fwd(dtype, h, W, y, V, Vp, K, 1.0)
    dz = 2 * H * U24 * (np.abs(S.as_f64(h)) @ np.abs(S.as_f64(W))[:V].T).max()
    r = (4 * np.abs(ref["z"]).max() + 2300) * U24 + 2 * dz
    for k in ("lse", "logp", "top_logp"):
        assert np.all(np.abs(got[k] - ref[k]) <= r), k
    assert np.all(np.abs(got["entropy"] - ref["entropy"]) <= 80 * r)
    # what is listed has the logits of the alternatives, each class once
    at = np.take_along_axis(ref["z"], got["top_ids"], axis=1)
    assert np.all(np.abs(at - np.take_along_axis(ref["z"], ref["top_ids"], axis=1)) <= 2 * dz)
    assert all(len(set(row)) == K for row in got["top_ids"].tolist())


@pytest.mark.parametrize("dtype,T", [("bf16", 4), ("bf16", 70), ("bf16", 300), ("f32", 66)])
def test_without_targets(dtype, T):
    h, W, _, Vp = grid_case(T, 64, 3000, dtype, seed=3)
    ref = S.token_scores(h, W, None, 3000, 1.0, 7)
    check_fwd(run_fwd(dtype, h, W, None, 3000, Vp, 7, 1.0), ref, 1.0, 7)


@pytest.mark.parametrize("dtype,T", [("bf16", 40), ("bf16", 300), ("f32", 66)])
def test_only_what_is_asked_for(dtype, T):
    """Each optional output alone, and the status word left out."""
    h, W, y, Vp = grid_case(T, 64, 2000, dtype, seed=4)
    ref = S.token_scores(h, W, y, 2000, 1.0, 6)
    p = problem(dtype, T, 64, Vp, 2000)
    hd, Wd, yd = D.to_device(h), D.to_device(W), torch.from_numpy(y).cuda()
    for name in ("logp", "entropy", "lse", "top"):
        K = 6 if name == "top" else 0
        ws = D.workspace(vce.vce_logprob_workspace_size(p, K))
        out = {name: torch.empty(T, device="cuda")} if K == 0 else dict(
            top_ids=torch.empty((T, K), dtype=torch.int64, device="cuda"), top_logp=torch.empty((T, K), device="cuda"))
        vce.vce_logprob_fwd(p, hd, Wd, yd, **out, ws=ws)
        torch.cuda.synchronize()
        if K:
            assert np.array_equal(out["top_ids"].cpu().numpy(), ref["top_ids"])
        else:
            assert np.abs(out[name].cpu().numpy() - ref[name]).max() < 1e-3


@pytest.mark.parametrize("dtype,T", [("bf16", 6), ("bf16", 66), ("bf16", 300), ("f32", 66)])
@pytest.mark.parametrize("order", ["equal", "ascending", "descending", "one_block", "duplicates"])
def test_orders_of_the_logits(dtype, T, order):
    """Rows whose logits are all equal (h = 0 for every third token), ascend or
    descend with the class, sit in one run of 40 classes, or come in equal
    groups across the vocabulary: alternatives in the stated order always."""
    H, V, K = 64, 9000, 20
    Vp = 9024
    w = np.zeros((Vp, H))
    v = np.arange(V)
    # two digits of the class in two columns, so that the logit 2^-3 (hi * 64 + lo) is exact
    val = {"equal": 0 * v, "ascending": v, "descending": V - v, "one_block": np.where((v >= 5000) & (v < 5040), 8000 + v % 7, v % 50),
           "duplicates": v % 1000}[order]
    w[:V, 0], w[:V, 1] = val // 64, val % 64
    h = np.zeros((T, H))
    h[:, 0], h[:, 1] = 1.0, 2.0 ** -6
    h[::3] = 0.0
    y = v[np.arange(T) * 37 % V]
    hb, Wb = store(h, dtype), store(w, dtype)
    ref = S.token_scores(hb, Wb, y, V, 0.5, K)
    check_fwd(run_fwd(dtype, hb, Wb, y, V, Vp, K, 0.5), ref, 0.5, K)


@pytest.mark.parametrize("dtype,T", [("bf16", 20), ("bf16", 280), ("f32", 70)])
def test_ignored_rows_may_hold_anything(dtype, T):
    """Infinite and NaN rows of ignored tokens, and bad targets: reported, the
    others as ever, the ignored ones' logp and entropy 0."""
    h, W, y, Vp = grid_case(T, 64, 1500, dtype, seed=5, ignore=0.0)
    bad = [1, T // 2, T - 1]
    clean = h.copy()
    h[bad] = np.uint16(0x7F80) if dtype == "bf16" else np.inf
    h[bad[1]] = np.uint16(0x7FC0) if dtype == "bf16" else np.nan
    y[bad[0]], y[bad[1]], y[bad[2]] = -100, 1500, -3
    ref = S.token_scores(clean, W, y, 1500, 1.0, 5)
    got = run_fwd(dtype, h, W, y, 1500, Vp, 5, 1.0, status=vce.VCE_ERR_BAD_INDEX)
    ok = np.ones(T, bool)
    ok[bad] = False
    check_fwd(got, ref, 1.0, 5, rows=ok)
    assert not got["logp"][bad].any() and not got["entropy"][bad].any()


@pytest.mark.parametrize("dtype,T", [("bf16", 7), ("bf16", 300), ("f32", 65)])
def test_nan_row_lists_nothing_and_classes_of_minus_infinity(dtype, T):
    H, V, Vp, K = 64, 100, 128, 32
    h, W, y, _ = grid_case(T, H, V, dtype, seed=6, ignore=0.0)
    Wf = S.as_f64(W)
    W[3:90] = 0
    W[3:90, 0] = np.uint16(0xFF80) if dtype == "bf16" else -np.inf    # -inf times a positive h
    Wf[3:90] = 0
    Wf[3:90, 0] = -np.inf
    hf = S.as_f64(h)
    hf[:, 0] = 1.0
    h = store(hf, dtype)
    h[0] = np.uint16(0x7FC0) if dtype == "bf16" else np.nan
    y[:] = 95
    got = run_fwd(dtype, h, W, y, V, Vp, K, 1.0)
    assert np.isnan(got["lse"][0]) and np.isnan(got["entropy"][0]) and np.isnan(got["logp"][0])
    assert np.all(got["top_ids"][0] == -1) and np.all(np.isnan(got["top_logp"][0]))
    with np.errstate(all="ignore"):
        z = hf[1:] @ np.where(np.isinf(Wf), 0, Wf)[:V].T
    z[:, 3:90] = -np.inf
    lse = np.log(np.exp(z).sum(1))
    lp = z - lse[:, None]
    ent = -np.where(np.isinf(lp), 0, np.exp(lp) * np.where(np.isinf(lp), 0, lp)).sum(1)
    assert np.abs(got["lse"][1:] - lse).max() < 1e-3 and np.abs(got["entropy"][1:] - ent).max() < 1e-3
    ids = np.argsort(-z, axis=1, kind="stable")[:, :K]
    assert np.array_equal(got["top_ids"][1:], ids)                    # 13 finite classes, then the lowest at -inf
    assert np.all(np.isneginf(got["top_logp"][1:, 13:]))


def test_large_logits_and_peaked_rows():
    """Scaled logits of over a thousand: probabilities of one class alone."""
    h, W, y, Vp = grid_case(150, 256, 3000, "bf16", seed=7, lean=0.5)
    ref = S.token_scores(h, W, y, 3000, 60.0, 3)
    assert np.abs(ref["z"]).max() * 60 > 1000
    check_fwd(run_fwd("bf16", h, W, y, 3000, Vp, 3, 60.0), ref, 60.0, 3)


@pytest.mark.parametrize("dtype,T", [("bf16", 9), ("bf16", 700)])
def test_same_bits_each_time_and_on_a_side_stream(dtype, T):
    h, W, y, Vp = grid_case(T, 128, 12000, dtype, seed=8)
    a = run_fwd(dtype, h, W, y, 12000, Vp, 20, 1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run_fwd(dtype, h, W, y, 12000, Vp, 20, 1.0)
    for k in a:
        assert np.array_equal(a[k], b[k]), k


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def run_bwd(dtype, h, W, y, V, Vp, ref, gl, ge, scale, flags=0, tied=False, dH=None, dW=None, dw_bf16=False,
            minimal=False, status=0, S_=4):
    T, H = h.shape
    p = problem(dtype, T, H, Vp, V, S_, flags=flags, tied=tied)
    if dH is None:
        dH = torch.full((T, H), float("nan"), device="cuda",
                        dtype=torch.bfloat16 if flags & vce.VCE_FLAG_DH_BF16 else torch.float32)
    if dW is None:
        dW = torch.full((Vp, H), float("nan"), device="cuda", dtype=torch.bfloat16 if dw_bf16 else torch.float32)
    size = vce.vce_workspace_size_min if minimal else vce.vce_workspace_size
    ws = D.workspace(size(p, vce.VCE_OP_LOGPROB_BWD))
    ws.fill_(0xFF)
    st = R.status_word()
    dev = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
    vce.vce_logprob_bwd(p, D.to_device(h), D.to_device(W), None if y is None else torch.from_numpy(y).cuda(),
                        dev(ref["lse"]), dev(ref["entropy"]), dev(gl), dev(ge), dH, dW, ws, logit_scale=scale,
                        dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return dH, dW


def check_bwd(dtype, got, h, W, y, V, ref, gl, ge, scale, dh_bf16=False, dw_bf16=False, base=(0.0, 0.0),
              g_round=2.0 ** -8):
    hf, Wf = S.as_f64(h), S.as_f64(W)
    T = hf.shape[0]
    ok = np.ones(T, bool) if y is None else S.valid_targets(y, V)
    hf = np.where(ok[:, None], hf, 0.0)
    # the formula at what the call is given: fp32 scale, lse and entropy
    scale = float(np.float32(scale))
    lse, ent = (np.where(ok, ref[k], 0).astype(np.float32).astype(np.float64) for k in ("lse", "entropy"))
    G = S.score_logit_gradient(hf, np.where(np.isnan(Wf), 0, Wf), y, V, gl, ge, scale, lse, ent)
    lp = scale * (hf @ np.where(np.isnan(Wf), 0, Wf)[:V].T) - lse[:, None]
    p_ = np.exp(lp)
    glv = np.zeros(T) if gl is None else np.where(ok, np.abs(gl), 0)
    gev = np.zeros(T) if ge is None else np.where(ok, np.abs(ge), 0)
    Gabs = gev[:, None] * p_ * (np.abs(lp) + np.abs(ent)[:, None]) + glv[:, None] * p_
    if gl is not None:
        Gabs[np.arange(T), np.where(ok, y, 0)] += glv
    Gabs *= scale
    A = np.abs(scale * ref["z"][ok]).max() if ok.any() else 0.0
    dG = ((8 * A + 80) + 2 * A) * U24 * Gabs + (g_round * np.abs(G) if dtype == "bf16" else 0)
    for name, x, g, b, n, wide, pre in (("dH", got[0], G @ Wf[:V], dG @ np.abs(Wf[:V]) , V, dh_bf16, base[0]),
                                        ("dW", got[1][:V], G.T @ hf, dG.T @ np.abs(hf), T, dw_bf16, base[1])):
        mag = np.abs(G) @ np.abs(Wf[:V]) if name == "dH" else np.abs(G).T @ np.abs(hf)
        want = g + pre
        tol = b + (n + 8) * U24 * mag + 2 * U24 * np.abs(want) + (2.0 ** -8 * (np.abs(want) + b) if wide else 0) + 1e-30
        x = x.float().cpu().numpy().astype(np.float64)
        worst = (np.abs(x - want) / tol).max()
        assert worst <= 1.0, (name, worst)


BWD = [(1, 64, 1, 1, 1.0), (1, 64, 1000, 4, 1.0), (2, 8, 70, 1, 0.5), (40, 72, 300, 3, 1.7), (64, 64, 1000, 4, 1.0),
       (130, 256, 4001, 8, 1 / 0.7), (257, 200, 5000, 7, 1.0), (517, 128, 3000, 8, 1.0)]


@pytest.mark.parametrize("T,H,V,S_,scale", BWD)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("terms", ["logp", "entropy", "both"])
def test_gradient(dtype, T, H, V, S_, scale, terms):
    h, W, y, Vp = grid_case(T, H, V, dtype, seed=11)
    rng = np.random.default_rng([12, T])
    gl = rng.standard_normal(T) if terms != "entropy" else None
    ge = rng.standard_normal(T) * 0.3 if terms != "logp" else None
    gl, ge = (None if g is None else g.astype(np.float32).astype(np.float64) for g in (gl, ge))
    ref = S.token_scores(h, W, y, V, scale)
    got = run_bwd(dtype, h, W, y, V, Vp, ref, gl, ge, scale, S_=S_)
    check_bwd(dtype, got, h, W, y, V, ref, gl, ge, scale)
    assert not got[1][V:].any().item()                    # padding rows of an untied dW are zero
    assert not got[0][torch.from_numpy(y < 0).cuda()].any().item()


@pytest.mark.parametrize("T", [1, 9, 31, 32, 33, 64, 100, 128])
@pytest.mark.parametrize("how", ["stored", "added", "chunks", "no targets"])
def test_gradient_of_few_tokens_keeps_what_rounding_left(T, how):
    """Up to 128 tokens G is the sum of two bf16 values: half a step of half a step, 2^-16, is lost."""
    H, V = 200, 4001
    h, W, y, Vp = grid_case(T, H, V, "bf16", seed=17)
    rng = np.random.default_rng([18, T])
    gl, ge = (rng.standard_normal(T).astype(np.float32).astype(np.float64) * s for s in (1.0, 0.25))
    if how == "no targets":
        y = gl = None
    ref = S.token_scores(h, W, y, V, 1.25)
    added = how == "added"
    dH, dW = torch.full((T, H), 2.0, device="cuda"), torch.full((Vp, H), -1.5, device="cuda")
    got = run_bwd("bf16", h, W, y, V, Vp, ref, gl, ge, 1.25, flags=vce.VCE_FLAG_ACCUMULATE_DH if added else 0,
                  tied=added, dH=dH if added else None, dW=dW if added else None, minimal=how == "chunks")
    check_bwd("bf16", got, h, W, y, V, ref, gl, ge, 1.25, base=(2.0, -1.5) if added else (0.0, 0.0),
              g_round=2.0 ** -16)


@pytest.mark.parametrize("dtype,T", [("bf16", 7), ("bf16", 300), ("f32", 65)])
@pytest.mark.parametrize("terms", ["logp", "entropy", "both"])
def test_gradient_with_classes_of_minus_infinity(dtype, T, terms):
    """Classes of logit -inf have no probability: no gradient of theirs, and none lost to the others."""
    H, V, Vp = 64, 100, 128
    h, W, y, _ = grid_case(T, H, V, dtype, seed=15, ignore=0.0)
    W[3:90] = 0
    W[3:90, 0] = np.uint16(0xFF80) if dtype == "bf16" else -np.inf
    hf = S.as_f64(h)
    hf[:, 0] = 1.0
    h = store(hf, dtype)
    y[:] = 95
    real = np.r_[0:3, 90:V]
    W13, y13 = W[real], np.full(T, 8)                     # the finite classes alone
    rng = np.random.default_rng(16)
    gl = rng.standard_normal(T).astype(np.float32).astype(np.float64) if terms != "entropy" else None
    ge = rng.standard_normal(T).astype(np.float32).astype(np.float64) if terms != "logp" else None
    ref = S.token_scores(h, W13, y13, 13, 1.0)
    dH, dW = run_bwd(dtype, h, W, y, V, Vp, ref, gl, ge, 1.0)
    assert not dW[3:90].any().item()
    # column 0 of dH multiplies a zero of G by -inf, as the formula does
    dH[:, 0] = torch.from_numpy(S.score_backward(h, W13, y13, 13, gl, ge, 1.0)[0][:, 0]).cuda()
    check_bwd(dtype, (dH, dW[torch.from_numpy(real).cuda()]), h, W13, y13, 13, ref, gl, ge, 1.0)


@pytest.mark.parametrize("minimal", [False, True])
@pytest.mark.parametrize("T", [100, 600])
def test_gradient_in_bf16(T, minimal):
    """dH and dW rounded once, also when the smallest workspace cuts the vocabulary into many chunks."""
    h, W, y, Vp = grid_case(T, 136, 2100, "bf16", seed=13)
    rng = np.random.default_rng(14)
    gl, ge = (rng.standard_normal(T).astype(np.float32).astype(np.float64) * s for s in (1.0, 0.25))
    ref = S.token_scores(h, W, y, 2100, 1.0)
    got = run_bwd("bf16", h, W, y, 2100, Vp, ref, gl, ge, 1.0, flags=vce.VCE_FLAG_DH_BF16, dw_bf16=True,
                  minimal=minimal)
    check_bwd("bf16", got, h, W, y, 2100, ref, gl, ge, 1.0, dh_bf16=True, dw_bf16=True)
    assert not got[1][2100:].any().item()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_adds_into_tied_weights_and_dH(dtype):
    T, H, V = 200, 64, 900
    h, W, y, Vp = grid_case(T, H, V, dtype, seed=15)
    rng = np.random.default_rng(16)
    gl = rng.standard_normal(T).astype(np.float32).astype(np.float64)
    ref = S.token_scores(h, W, y, V, 1.0)
    dH0, dW0 = rng.standard_normal((T, H)).astype(np.float32), rng.standard_normal((Vp, H)).astype(np.float32)
    dH, dW = torch.from_numpy(dH0).cuda(), torch.from_numpy(dW0).cuda()
    run_bwd(dtype, h, W, y, V, Vp, ref, gl, None, 1.0, flags=vce.VCE_FLAG_ACCUMULATE_DH, tied=True, dH=dH, dW=dW)
    check_bwd(dtype, (dH, dW), h, W, y, V, ref, gl, None, 1.0, base=(dH0.astype(np.float64), dW0[:V].astype(np.float64)))
    assert np.array_equal(dW[V:].cpu().numpy(), dW0[V:])


@pytest.mark.parametrize("dtype,T", [("bf16", 30), ("bf16", 300), ("f32", 70)])
def test_gradient_ignores_what_ignored_rows_hold(dtype, T):
    h, W, y, Vp = grid_case(T, 64, 800, dtype, seed=17, ignore=0.3)
    y[0], y[1] = -100, 800                                 # the second is reported
    clean = h.copy()
    clean[y < 0] = 0
    h[y < 0] = np.uint16(0x7F80) if dtype == "bf16" else np.inf
    h[1] = np.uint16(0x7FC0) if dtype == "bf16" else np.nan
    clean[1] = 0
    gl = np.random.default_rng(18).standard_normal(T).astype(np.float32).astype(np.float64)
    ref = S.token_scores(clean, W, y, 800, 1.0)
    bad = ~S.valid_targets(y, 800)
    lse = ref["lse"].copy()
    lse[bad] = np.nan                                      # as the forward leaves it for such rows
    got = run_bwd(dtype, h, W, y, 800, Vp, dict(ref, lse=lse), gl, gl, 1.0, status=vce.VCE_ERR_BAD_INDEX)
    check_bwd(dtype, got, clean, W, y, 800, ref, gl, gl, 1.0)
    assert not got[0][torch.from_numpy(bad).cuda()].any().item()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_entropy_gradient_without_targets_and_all_ignored(dtype):
    T, H, V = 90, 64, 700
    h, W, y, Vp = grid_case(T, H, V, dtype, seed=19)
    ge = np.random.default_rng(20).standard_normal(T).astype(np.float32).astype(np.float64)
    ref = S.token_scores(h, W, None, V, 1.0)
    check_bwd(dtype, run_bwd(dtype, h, W, None, V, Vp, ref, None, ge, 1.0), h, W, None, V, ref, None, ge, 1.0)
    y[:] = -100
    dH, dW = run_bwd(dtype, h, W, y, V, Vp, ref, ge, ge, 1.0)
    assert not dH.any().item() and not dW.any().item()


def test_gradient_against_differences_of_the_forward():
    """fp32: the change of sum g logp + e entropy along a direction of h and of
    W, by central differences of the library's own forward. A step of 2^-6 leaves
    a truncation error of step^2 / 6 times the third derivative and a rounding
    error of about 1e-5 / step; 2% of the largest slope covers both."""
    T, H, V = 24, 32, 150
    h, W, y, Vp = grid_case(T, H, V, "f32", seed=21, pad=0.0)
    rng = np.random.default_rng(22)
    gl, ge = rng.standard_normal(T).astype(np.float32), rng.standard_normal(T).astype(np.float32)
    f0 = run_fwd("f32", h, W, y, V, Vp, 0, 1.0)
    dH, dW = run_bwd("f32", h, W, y, V, Vp, f0, gl, ge, 1.0)
    f = lambda a, b: (lambda r: float((gl * r["logp"] + ge * r["entropy"]).astype(np.float64).sum()))(  # noqa: E731
        run_fwd("f32", a.astype(np.float32), b.astype(np.float32), y, V, Vp, 0, 1.0))
    s = 2.0 ** -6
    for _ in range(4):
        a, b = rng.standard_normal(h.shape).astype(np.float32), rng.standard_normal(W.shape).astype(np.float32)
        a, b = a / np.linalg.norm(a), b / np.linalg.norm(b)
        b[V:] = 0
        for da, db in ((a, 0 * b), (0 * a, b)):
            slope = (f(h + s * da, W + s * db) - f(h - s * da, W - s * db)) / (2 * s)
            want = float((dH.cpu().numpy().astype(np.float64) * da).sum() + (dW.cpu().numpy().astype(np.float64) * db).sum())
            scale = np.linalg.norm((dH if da.any() else dW).cpu().numpy())
            assert abs(slope - want) <= 0.02 * scale, (slope, want)


def test_forward_and_gradient_in_a_cuda_graph():
    T, H, V, K = 300, 128, 5000, 8
    h, W, y, Vp = grid_case(T, H, V, "bf16", seed=23)
    p = problem("bf16", T, H, Vp, V, flags=vce.VCE_FLAG_DH_BF16)
    hd, Wd, yd = D.to_device(h), D.to_device(W), torch.from_numpy(y).cuda()
    g = torch.randn(T, device="cuda")
    out = [torch.empty(T, device="cuda") for _ in range(3)]
    ids, tl = torch.empty((T, K), dtype=torch.int64, device="cuda"), torch.empty((T, K), device="cuda")
    dH, dW = torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), torch.empty((Vp, H), dtype=torch.bfloat16, device="cuda")
    wf, wb = D.workspace(vce.vce_logprob_workspace_size(p, K)), D.workspace(vce.vce_workspace_size(p, vce.VCE_OP_LOGPROB_BWD))

    def step():
        vce.vce_logprob_fwd(p, hd, Wd, yd, *out, ids, tl, ws=wf)
        vce.vce_logprob_bwd(p, hd, Wd, yd, out[2], out[1], g, g, dH, dW, wb)

    step()
    torch.cuda.synchronize()
    every = [*out, tl, dH, dW, ids]
    want = [x.clone() for x in every]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        for x in every:
            x.fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(every, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_empty_batch():
    p = problem("bf16", 0, 64, 128, 100)
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((128, 64), dtype=torch.bfloat16, device="cuda")
    z, i = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    vce.vce_logprob_fwd(p, e, W, i, z, z, z, torch.empty((0, 3), dtype=torch.int64, device="cuda"),
                        torch.empty((0, 3), device="cuda"), ws=D.workspace(256))
    dW = torch.ones((128, 64), device="cuda")
    vce.vce_logprob_bwd(p, e, W, i, z, z, z, z, torch.empty((0, 64), device="cuda"), dW, D.workspace(256))
    torch.cuda.synchronize()
    assert not dW.any().item()


@pytest.mark.parametrize("T", [1100])
def test_gradient_with_parts_added_in_turn(T):
    """Enough tiles of dH that its K parts are added one after the other."""
    H, V = 1024, 4100
    h, W, y, Vp = grid_case(T, H, V, "bf16", seed=24)
    rng = np.random.default_rng(25)
    gl, ge = (rng.standard_normal(T).astype(np.float32).astype(np.float64) * s for s in (1.0, 0.25))
    ref = S.token_scores(h, W, y, V, 1.0)
    got = run_bwd("bf16", h, W, y, V, Vp, ref, gl, ge, 1.0, flags=vce.VCE_FLAG_DH_BF16, dw_bf16=True)
    check_bwd("bf16", got, h, W, y, V, ref, gl, ge, 1.0, dh_bf16=True, dw_bf16=True)
    again = run_bwd("bf16", h, W, y, V, Vp, ref, gl, ge, 1.0, flags=vce.VCE_FLAG_DH_BF16, dw_bf16=True)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_tokens_in_several_passes():
    """More tokens than one pass of the workspace takes, the last pass a short one."""
    T, H, V, K = 50100, 64, 20000, 32
    h, W, y, Vp = grid_case(T, H, V, "bf16", seed=26)
    assert vce.vce_logprob_workspace_size(problem("bf16", T, H, Vp, V), K) < 600 << 20
    got = run_fwd("bf16", h, W, y, V, Vp, K, 1.0)
    rng = np.random.default_rng(27)
    rows = np.unique(np.concatenate([rng.integers(0, T, 200), np.arange(T - 150, T), np.arange(0, T, 2048)]))
    ref = S.token_scores(h[rows], W, y[rows], V, 1.0, K)
    check_fwd({k: v[rows] for k, v in got.items()}, ref, 1.0, K)
    assert np.all(np.isfinite(got["lse"])) and np.all((got["top_ids"] >= 0) & (got["top_ids"] < V))


def test_classes_past_32_bit_offsets():
    """W of more than 2^31 elements: the classes that matter lie at its end."""
    H, V = 2048, 1100032
    W = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
    last = torch.arange(V - 40, V, device="cuda")
    W[last, 0] = (torch.arange(40, device="cuda") + 1).bfloat16()
    for T in (3, 200):
        h = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
        h[:, 0] = 0.5
        y = torch.full((T,), V - 1, dtype=torch.int64, device="cuda")
        p = vce.problem(T, H, V, V, 8, vce.VCE_BF16)
        logp, ent, lse = (torch.empty(T, device="cuda") for _ in range(3))
        ids, tl = torch.empty((T, 20), dtype=torch.int64, device="cuda"), torch.empty((T, 20), device="cuda")
        vce.vce_logprob_fwd(p, h, W, y, logp, ent, lse, ids, tl, ws=D.workspace(vce.vce_logprob_workspace_size(p, 20)))
        torch.cuda.synchronize()
        z = 0.5 * (np.arange(40) + 1)
        want = np.log(np.exp(z).sum() + V - 40)
        assert np.abs(lse.cpu().numpy() - want).max() < 1e-3
        assert np.abs(logp.cpu().numpy() - (z[-1] - want)).max() < 1e-3
        assert torch.equal(ids, torch.arange(V - 1, V - 21, -1, device="cuda").expand(T, 20))
