"""vce_norm_fwd and vce_norm_bwd against the fp64 oracle.

Tolerances, u = 2^-24: a sum of H terms in chains of at most c = H/32 + 64 and
a tree adds c u of the sum of magnitudes. mean: c u mean|x|. rstd: c u and the
mean's error over the deviation, (c + 16) u (1 + max|x| rstd)^2 relatively.
y: the same relative error on xhat's and the mean's part, plus 2^-8 |y| in
bf16. dx: (2 c + 32) u of the sum of its terms' magnitudes, plus 2^-8 |dx|.
dweight, dbias: (T + 32) u of the sum of their terms' magnitudes.
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
KIND = {"layer": vce.VCE_NORM_LAYER, "rms": vce.VCE_NORM_RMS}


def store(x, dtype):
    return I.bf16_bits(x.astype(np.float32)) if dtype == "bf16" else np.ascontiguousarray(x, np.float32)


def case(T, H, dtype, seed=0, dy="f32"):
    rng = np.random.default_rng([seed, T, H])
    size = np.exp(0.5 * rng.standard_normal(H)) * np.where(rng.random(H) < 0.02, 20.0, 1.0)
    x = store(rng.standard_normal((T, H)) * size + 0.3, dtype)
    w, b = store(1 + 0.2 * rng.standard_normal(H), dtype), store(0.1 * rng.standard_normal(H), dtype)
    return x, w, b, store(rng.standard_normal((T, H)), dy)


def problem(dtype, T, H, dy="f32"):
    return vce.problem(T, H, 64, 64, 1, vce.VCE_BF16 if dtype == "bf16" else vce.VCE_F32,
                       flags=vce.VCE_FLAG_DH_BF16 if dy == "bf16" else 0)


def tdt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def run_fwd(dtype, x, w, b, kind, eps=1e-5, stats=True):
    T, H = x.shape
    y = torch.full((T, H), float("nan"), dtype=tdt(dtype), device="cuda")
    mean, rstd = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    dev = lambda a: None if a is None else D.to_device(a)  # noqa: E731
    vce.vce_norm_fwd(problem(dtype, T, H), dev(x), dev(w), dev(b), y, mean if stats else None, rstd if stats else None,
                     eps=eps, kind=KIND[kind])
    torch.cuda.synchronize()
    return y, mean, rstd


SIZES = [(1, 8), (1, 2048), (2, 16), (3, 64), (5, 72), (7, 1024), (33, 200), (48, 1024), (129, 520), (300, 2048), (40, 4096),
         (9, 8192), (4, 16384), (2, 65536), (1000, 256), (2500, 64)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_forward(T, H, dtype, kind):
    x, w, b, _ = case(T, H, dtype, 1)
    for wt, bs in ((w, b), (w, None), (None, None)):
        got, mean, rstd = run_fwd(dtype, x, wt, bs, kind)
        y, mu, r = S.norm_forward(x, wt, bs, 1e-5, kind == "rms")
        c = H / 32 + 64
        ax = np.abs(S.as_f64(x))
        assert np.all(np.abs(mean.cpu().numpy() - mu) <= c * U24 * ax.mean(1))
        rel = (c + 16) * U24 * (1 + np.abs(mu) * r) ** 2 * 4
        assert np.all(np.abs(rstd.cpu().numpy() - r) <= rel * r)
        wf = 1.0 if wt is None else np.abs(S.as_f64(wt))
        mag = (ax + np.abs(mu)[:, None]) * r[:, None] * wf + (0 if bs is None else np.abs(S.as_f64(bs)))
        tol = (rel[:, None] + (c + 16) * U24) * (mag + (ax.mean(1) * r)[:, None] * wf)
        tol = tol + (2.0 ** -8 * (np.abs(y) + tol) if dtype == "bf16" else 0)
        assert np.all(np.abs(got.float().cpu().numpy() - y) <= tol)
        if bs is None:
            y2, _, _ = run_fwd(dtype, x, wt, bs, kind, stats=False)   # statistics not asked for
            assert torch.equal(y2, got)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype,dy", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward(T, H, dtype, dy, kind):
    x, w, _, d = case(T, H, dtype, 2, dy)
    _, mu, r = S.norm_forward(x, w, None, 1e-5, kind == "rms")
    mu, r = mu.astype(np.float32), r.astype(np.float32)
    p = problem(dtype, T, H, dy)
    ws = D.workspace(vce.vce_workspace_size(p, vce.VCE_OP_NORM_BWD))
    md, rd = torch.from_numpy(mu).cuda(), torch.from_numpy(r).cuda()
    xd, wd, dd = D.to_device(x), D.to_device(w), D.to_device(d)
    for wt in (w, None):
        ws.fill_(0xFF)
        dx = torch.full((T, H), float("nan"), dtype=tdt(dtype), device="cuda")
        dw, db = (torch.full((H,), float("nan"), device="cuda") for _ in range(2))
        vce.vce_norm_bwd(p, xd, None if wt is None else wd, dd, md if kind == "layer" else None, rd, dx, dw, db, ws,
                         kind=KIND[kind])
        torch.cuda.synchronize()
        want = S.norm_backward(x, wt, d, mu, r, kind == "rms")
        c = H / 32 + 64
        mean = 0.0 if kind == "rms" else mu.astype(np.float64)[:, None]
        r64 = r.astype(np.float64)[:, None]
        xa = (np.abs(S.as_f64(x)) + np.abs(mean)) * r64                # terms of xhat
        g = np.abs(S.as_f64(d)) * (1.0 if wt is None else np.abs(S.as_f64(wt)))
        mag = r64 * (g + g.mean(1, keepdims=True) + xa * (g * xa).mean(1, keepdims=True))
        tol = (2 * c + 32) * U24 * mag
        tol = tol + (2.0 ** -8 * (np.abs(want[0]) + tol) if dtype == "bf16" else 0)
        assert np.all(np.abs(dx.float().cpu().numpy() - want[0]) <= tol)
        da = np.abs(S.as_f64(d))
        assert np.all(np.abs(dw.cpu().numpy() - want[1]) <= (T + 32) * U24 * (da * xa).sum(0))
        assert np.all(np.abs(db.cpu().numpy() - want[2]) <= (T + 32) * U24 * da.sum(0))


@pytest.mark.parametrize("T,H", [(1, 4), (37, 12), (300, 20), (200, 1028), (5, 8196)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward_of_bf16_rows_that_are_not_whole_16_byte_units(T, H, kind):
    test_backward(T, H, "f32", "bf16", kind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_accumulates_and_leaves_out_what_is_not_asked_for(dtype):
    T, H = 130, 264
    x, w, _, d = case(T, H, dtype, 3)
    _, mu, r = S.norm_forward(x, w, None)
    p = problem(dtype, T, H)
    ws = D.workspace(vce.vce_workspace_size(p, vce.VCE_OP_NORM_BWD))
    args = (D.to_device(x), D.to_device(w), D.to_device(d), torch.from_numpy(mu.astype(np.float32)).cuda(),
            torch.from_numpy(r.astype(np.float32)).cuda())
    full = [torch.empty((T, H), dtype=tdt(dtype), device="cuda"), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")]
    vce.vce_norm_bwd(p, *args, *full, ws)
    torch.cuda.synchronize()
    for keep in ((0,), (1,), (2,), (0, 2), (1, 2)):
        out = [torch.full_like(t, 3.0) if i in keep else None for i, t in enumerate(full)]
        vce.vce_norm_bwd(p, *args, *out, ws, accumulate=True)
        torch.cuda.synchronize()
        for i in keep:
            want = full[i] + 3.0 if i else full[i]                    # dx is written, the sums added into
            assert torch.equal(out[i], want), (keep, i)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_constant_and_huge_rows(kind):
    """A row of one value (deviation zero), one of zeros, one near the largest
    value whose squares fit: finite results of the formula."""
    H = 512
    x = np.zeros((4, H), np.float32)
    x[0] = 2.5
    x[2] = np.where(np.arange(H) % 2, 1e17, -1e17)
    x[3, 5] = 1e-18
    y, mean, rstd = run_fwd("f32", x, None, None, kind)
    yo, mu, r = S.norm_forward(x, None, None, 1e-5, kind == "rms")
    assert np.all(np.abs(y.cpu().numpy() - yo) <= 1e-4 * (1 + np.abs(yo)))
    assert np.all(np.abs(rstd.cpu().numpy() - r) <= 1e-5 * r)


def test_same_bits_each_time_and_in_a_graph():
    T, H = 1111, 1024
    x, w, b, d = case(T, H, "bf16", 4)
    p = problem("bf16", T, H)
    dev = [D.to_device(a) for a in (x, w, b, d)]
    y, dx = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ws = D.workspace(vce.vce_workspace_size(p, vce.VCE_OP_NORM_BWD))

    def step():
        vce.vce_norm_fwd(p, dev[0], dev[1], dev[2], y, mean, rstd)
        vce.vce_norm_bwd(p, dev[0], dev[1], dev[3], mean, rstd, dx, dw, db, ws)

    step()
    torch.cuda.synchronize()
    every = [y, dx, mean, rstd, dw, db]
    want = [t.clone() for t in every]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        for t in every:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b_ in zip(every, want):
            assert torch.equal(a.view(torch.uint8), b_.view(torch.uint8))


def test_rows_past_32_bit_offsets():
    """x of more than 2^31 elements: the last rows, and the sums over all of them."""
    T, H = 1050001, 2048
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    base = torch.randn((1, H), generator=g, device="cuda").bfloat16()
    x.copy_(base.expand(T, H))
    x[-3:] = torch.randn((3, H), generator=g, device="cuda").bfloat16()
    p = problem("bf16", T, H, "bf16")
    y = torch.empty_like(x)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    vce.vce_norm_fwd(p, x, None, None, y, mean, rstd)
    torch.cuda.synchronize()
    for rows in (slice(0, 2), slice(T - 3, T)):
        xs = D.to_host_bits(x[rows])
        yo, mu, r = S.norm_forward(xs)
        assert np.all(np.abs(y[rows].float().cpu().numpy() - yo) <= 2.0 ** -8 * np.abs(yo) + 1e-4)
        assert np.all(np.abs(rstd[rows].cpu().numpy() - r) <= 1e-4 * r)
    assert bool((rstd[:-3] == rstd[0]).all())
    dy = x                                        # any bf16 gradient
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    vce.vce_norm_bwd(p, x, None, dy, mean, rstd, y, dw, db, D.workspace(vce.vce_workspace_size(p, vce.VCE_OP_NORM_BWD)))
    torch.cuda.synchronize()
    _, dw1, db1 = S.norm_backward(D.to_host_bits(x[:1]), None, D.to_host_bits(x[:1]), mean[:1].cpu().numpy(),
                                  rstd[:1].cpu().numpy())
    _, dw3, db3 = S.norm_backward(D.to_host_bits(x[-3:]), None, D.to_host_bits(x[-3:]), mean[-3:].cpu().numpy(),
                                  rstd[-3:].cpu().numpy())
    n = T - 3
    # equal terms added one by one in chains of at most T / 152 rows: n u of the sum, u = 2^-24
    for got, one, three in ((dw, dw1, dw3), (db, db1, db3)):
        want = n * one + three
        assert np.all(np.abs(got.cpu().numpy() - want) <= (T / 152 + 200) * U24 * n * (np.abs(one) + 0.01))
