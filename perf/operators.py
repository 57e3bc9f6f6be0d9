"""The token-score and normalisation operators: what is measured, on which sizes.

Each case is one call of an operator as a program makes it. ``run`` computes it
either in plain torch operations (``own`` false) or through the library
(``own`` true); ``exact`` computes it in 64 bits from the definition.

The head's inputs lie on a coarse grid (hidden states in steps of 1/4, weights
in steps of 1/128, eight bits each): every logit is then exact in fp32 in any
order of summation, so that the order of the top alternatives, and which of two
equal logits comes first, is decided by the inputs and not by rounding.
"""
import math

import torch

own = False

IGNORE = -100
STEP_H, STEP_W = 2.0 ** -2, 2.0 ** -7


def listed():
    return [
        # One new token of one sequence: serving with the top alternatives shown.
        dict(name="score_one_token", op="score", dtype="bf16", T=1, H=2048, V=151936, S=8, K=20, scale=1.0),
        # One step of a decoding batch, on a head whose vocabulary is padded.
        dict(name="score_decode_batch", op="score", dtype="bf16", T=48, H=1024, V=50000, S=8, K=5, scale=1.25),
        # A prompt of odd length scored with a few alternatives a position.
        dict(name="score_prompt", op="score", dtype="bf16", T=1311, H=2048, V=151936, S=8, K=8, scale=1.0),
        # A training batch scored under the sampling temperature, with 20 alternatives.
        dict(name="score_rollout", op="score", dtype="bf16", T=8192, H=2048, V=151936, S=8, K=20, scale=1.0 / 0.7),
        # The smallest fp32 head.
        dict(name="score_f32", op="score", dtype="f32", T=64, H=64, V=1000, S=4, K=10, scale=1.0),
        # Policy-gradient step with an entropy term over the whole batch.
        dict(name="grad_rollout", op="grad", dtype="bf16", T=8192, H=2048, V=151936, S=8, scale=1.0 / 0.7),
        # A ragged micro-batch on the smaller head.
        dict(name="grad_ragged", op="grad", dtype="bf16", T=517, H=1024, V=50000, S=8, scale=1.0),
        # The smallest fp32 head, its gradients in fp32.
        dict(name="grad_f32", op="grad", dtype="f32", T=64, H=64, V=1000, S=4, scale=1.0),
        # The final norm of a decoding batch.
        dict(name="norm_decode", op="norm", dtype="bf16", T=48, H=1024, kind="layer", bias=True),
        # The final norm of a training batch (no mean taken, no bias).
        dict(name="norm_batch", op="norm", dtype="bf16", T=16384, H=2048, kind="rms", bias=False),
        # Its backward pass; the head's gradient arrives in fp32.
        dict(name="norm_grad_batch", op="norm_grad", dtype="bf16", T=8192, H=2048, kind="layer", bias=True, dy="f32"),
        # A ragged micro-batch, the head's gradient in bf16.
        dict(name="norm_grad_ragged", op="norm_grad", dtype="bf16", T=517, H=1024, kind="rms", bias=False, dy="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score", "grad", "norm", "norm_grad"])
    if op in ("score", "grad"):
        if rng.random() < 0.2:   # fp32 heads are small
            c = dict(op=op, dtype="f32", T=_log_int(rng, 1, 300), H=4 * _log_int(rng, 8, 128), V=_log_int(rng, 40, 8000))
        else:
            c = dict(op=op, dtype="bf16", T=_log_int(rng, 1, 8192), H=8 * _log_int(rng, 8, 256), V=_log_int(rng, 500, 151936))
        c["S"] = rng.randint(1, 8)
        c["scale"] = rng.choice([1.0, 1.0, 1.0 / 0.7, 0.5, 1.25])
        if op == "score":
            c["K"] = rng.choice([0, 1, rng.randint(2, 8), rng.randint(9, 20), 20, rng.randint(21, 32)])
        return c
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, dtype=dtype, T=_log_int(rng, 1, 16384), H=8 * _log_int(rng, 8, 512), kind=rng.choice(["layer", "rms"]))
    while c["T"] * c["H"] > 16384 * 2048:
        c["T"] = max(1, c["T"] // 2)
    c["bias"] = rng.random() < 0.5
    if op == "norm_grad":
        c["dy"] = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
    return c


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, H, dt = case["T"], case["H"], _dt(case["dtype"])

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case=case)
    if case["op"] in ("score", "grad"):
        V = case["V"]
        Vp = -(-V // 64) * 64
        w = torch.round(randn(Vp, H) * 8).clamp_(-127, 127)
        # Zipf-like targets, one in twenty ignored
        y = (V ** rand(T) - 1).long().clamp_(0, V - 1)
        # hidden states: noise, and a part along the target's row, from none to
        # enough to lift its logit by about 15
        lean = rand(T, 1) * min(0.5, 120.0 / H)
        h = torch.round(randn(T, H) * 4 + lean * w[y]).clamp_(-127, 127)
        s["W"] = (w * STEP_W).to(dt)
        s["W"][V:] = 8.0                       # padding rows hold anything
        s["h"] = (h * STEP_H).to(dt)
        s["targets"] = torch.where(rand(T) < 0.05, IGNORE, y)
        del w
        new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        if case["op"] == "score":
            s["logp"], s["entropy"], s["lse"] = new(T), new(T), new(T)
            if case["K"]:
                s["top_ids"], s["top_logp"] = new(T, case["K"], dtype=torch.int64), new(T, case["K"])
        else:
            # what the forward pass left, and the step's weights of each token
            _, s["lse"], s["entropy"] = _plain_stats(s)
            s["g_logp"] = randn(T) / T
            s["g_entropy"] = -0.01 * (0.5 + rand(T)) / T
            s["dH"], s["dW"] = new(T, H, dtype=dt), new(Vp, H, dtype=dt)
        return s
    # residual stream: channels of different size and offset, a few large ones
    size = torch.exp(0.5 * randn(H)) * torch.where(rand(H) < 0.01, 20.0, 1.0)
    s["x"] = (randn(T, H) * size + 0.3 * randn(H) + 0.2).to(dt)
    s["weight"] = (1.0 + 0.2 * randn(H)).to(dt)
    s["bias"] = (0.1 * randn(H)).to(dt) if case["bias"] else None
    s["eps"] = 1e-5
    stat = lambda: torch.empty(T, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        s["y"], s["rstd"] = torch.empty_like(s["x"]), stat()
        s["mean"] = stat() if case["kind"] == "layer" else None
    else:
        x = s["x"].float()
        s["mean"] = x.mean(1) if case["kind"] == "layer" else None
        if s["mean"] is not None:
            x = x - s["mean"][:, None]
        s["rstd"] = 1.0 / torch.sqrt((x * x).mean(1) + s["eps"])
        s["dy"] = (randn(T, H) * 1e-3).to(_dt(case["dy"]))
        s["dx"] = torch.empty_like(s["x"])
        s["dweight"] = torch.empty(H, device="cuda")
        s["dbias"] = torch.empty(H, device="cuda") if case["bias"] else None
    return s


def work(case):
    T, H = case["T"], case["H"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "score":
        out = T * (3 * 4 + case["K"] * 12)
        return {"bytes": (T + case["V"]) * H * e + T * 8 + out, "flops": 2 * T * H * case["V"]}
    if case["op"] == "grad":
        # h and W in, dH and dW out; the logits once more and the two products of their gradient
        return {"bytes": 2 * (T + case["V"]) * H * e + T * 24, "flops": 6 * T * H * case["V"]}
    stats = 8 if case["kind"] == "layer" else 4
    if case["op"] == "norm":
        return {"bytes": 2 * T * H * e + (2 if case["bias"] else 1) * H * e + T * stats, "flops": 6 * T * H}
    d = 2 if case["dy"] == "bf16" else 4
    return {"bytes": T * H * (2 * e + d) + H * e + (2 if case["bias"] else 1) * H * 4 + T * stats, "flops": 12 * T * H}


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------

def _plain_stats(s):
    """Unscaled logits, and lse and entropy of the scaled ones (0 entropy where ignored)."""
    c = s["case"]
    z0 = s["h"].float() @ s["W"][:c["V"]].float().T
    d = z0 * c["scale"]
    m = d.amax(1, keepdim=True)
    d -= m
    e = torch.exp(d)
    tot = e.sum(1)
    ent = torch.log(tot) - (e * d).sum(1) / tot
    valid = s["targets"] >= 0
    return z0, m[:, 0] + torch.log(tot), torch.where(valid, ent, 0.0)


def _plain_score(s):
    c = s["case"]
    z0, lse, ent = _plain_stats(s)
    valid = s["targets"] >= 0
    zy = torch.gather(z0, 1, s["targets"].clamp(min=0)[:, None])[:, 0]
    out = dict(logp=torch.where(valid, zy * c["scale"] - lse, 0.0), entropy=ent, lse=lse)
    if c["K"]:
        # one key a logit: its value's order above, the lower class first below
        b = (z0 + 0.0).view(torch.int32)
        key = torch.where(b >= 0, b, b ^ 0x7FFFFFFF).long()
        key = (key << 32) + (0xFFFFFFFF - torch.arange(c["V"], device=b.device))
        top = torch.topk(key, c["K"], dim=1).values
        out["top_ids"] = 0xFFFFFFFF - (top & 0xFFFFFFFF)
        out["top_logp"] = torch.gather(z0, 1, out["top_ids"]) * c["scale"] - lse[:, None]
    return out


def _plain_grad(s):
    c = s["case"]
    V, scale = c["V"], c["scale"]
    h, W = s["h"].float(), s["W"][:V].float()
    lp = (h @ W.T) * scale - s["lse"][:, None]
    valid = s["targets"] >= 0
    gl = torch.where(valid, s["g_logp"], 0.0)[:, None]
    ge = torch.where(valid, s["g_entropy"], 0.0)[:, None]
    G = -torch.exp(lp) * (gl + ge * (lp + s["entropy"][:, None]))
    G.scatter_add_(1, s["targets"].clamp(min=0)[:, None], gl)
    G *= scale
    dW = torch.zeros_like(s["W"])
    dW[:V] = (G.T @ h).to(dW.dtype)
    return dict(dH=(G @ W).to(s["h"].dtype), dW=dW)


def _plain_norm(s):
    x = s["x"].float()
    out = {}
    if s["case"]["kind"] == "layer":
        out["mean"] = x.mean(1)
        x = x - out["mean"][:, None]
    out["rstd"] = 1.0 / torch.sqrt((x * x).mean(1) + s["eps"])
    y = x * out["rstd"][:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out["y"] = y.to(s["x"].dtype)
    return out


def _plain_norm_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    if s["mean"] is not None:
        x = x - s["mean"][:, None]
    xh = x * s["rstd"][:, None]
    gy = dy * s["weight"].float()
    dx = gy - xh * (gy * xh).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - gy.mean(1, keepdim=True)
    out = dict(dx=(dx * s["rstd"][:, None]).to(s["x"].dtype), dweight=(dy * xh).sum(0))
    if s["dbias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


# ----------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------

def _problem(vce, s, flags=0):
    c = s["case"]
    V = c.get("V", 64)
    return vce.problem(c["T"], c["H"], -(-V // 64) * 64, V, c.get("S", 1),
                       vce.VCE_BF16 if c["dtype"] == "bf16" else vce.VCE_F32, ignore_index=IGNORE, flags=flags)


def _workspace(s, nbytes):
    """The state's workspace, laid out at its first pass and kept by the program."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(int(nbytes()), 1), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_score(s):
    from vocab_embedding_cross_gb300 import _lib as vce
    c = s["case"]
    p = _problem(vce, s)
    ws = _workspace(s, lambda: vce.vce_logprob_workspace_size(p, c["K"]))
    vce.vce_logprob_fwd(p, s["h"], s["W"], s["targets"], s["logp"], s["entropy"], s["lse"], s.get("top_ids"),
                        s.get("top_logp"), logit_scale=c["scale"], ws=ws)
    return {k: s[k] for k in ("logp", "entropy", "lse", "top_ids", "top_logp") if k in s}


def _own_grad(s):
    from vocab_embedding_cross_gb300 import _lib as vce
    c = s["case"]
    p = _problem(vce, s, flags=vce.VCE_FLAG_DH_BF16 if c["dtype"] == "bf16" else 0)
    ws = _workspace(s, lambda: vce.vce_workspace_size(p, vce.VCE_OP_LOGPROB_BWD))
    vce.vce_logprob_bwd(p, s["h"], s["W"], s["targets"], s["lse"], s["entropy"], s["g_logp"], s["g_entropy"], s["dH"],
                        s["dW"], ws, logit_scale=c["scale"])
    return dict(dH=s["dH"], dW=s["dW"])


def _own_norm(s):
    from vocab_embedding_cross_gb300 import _lib as vce
    kind = vce.VCE_NORM_LAYER if s["case"]["kind"] == "layer" else vce.VCE_NORM_RMS
    vce.vce_norm_fwd(_problem(vce, s), s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], eps=s["eps"],
                     kind=kind)
    return {k: s[k] for k in ("y", "mean", "rstd") if s[k] is not None}


def _own_norm_grad(s):
    from vocab_embedding_cross_gb300 import _lib as vce
    kind = vce.VCE_NORM_LAYER if s["case"]["kind"] == "layer" else vce.VCE_NORM_RMS
    p = _problem(vce, s, flags=vce.VCE_FLAG_DH_BF16 if s["case"]["dy"] == "bf16" else 0)
    ws = _workspace(s, lambda: vce.vce_workspace_size(p, vce.VCE_OP_NORM_BWD))
    vce.vce_norm_bwd(p, s["x"], s["weight"], s["dy"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"], ws,
                     kind=kind)
    return {k: s[k] for k in ("dx", "dweight", "dbias") if s[k] is not None}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"score": _own_score, "grad": _own_grad, "norm": _own_norm, "norm_grad": _own_norm_grad}[op](state)
    return {"score": _plain_score, "grad": _plain_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad}[op](state)


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    T, H = case["T"], case["H"]
    if case["op"] in ("score", "grad") and work(case)["flops"] > 2e13:
        return None
    s = prepare(case, seed)
    f = lambda k: s[k].double()  # noqa: E731
    if case["op"] in ("score", "grad"):
        V = case["V"]
        logit = torch.matmul(f("h"), f("W")[:V].t())
        y = s["targets"].clamp(min=0)
        keep = (s["targets"] != IGNORE).double()
        rows = torch.arange(T, device="cuda")
    if case["op"] == "score":
        ids = None
        if case["K"]:
            # steps of 2^-9 between different logits; 2^-28 a class decides between equal ones
            ids = torch.topk(logit - torch.arange(V, device="cuda") * 2.0 ** -28, case["K"], dim=1, sorted=True).indices
        top = torch.gather(logit, 1, ids) * case["scale"] if case["K"] else None
        logit *= case["scale"]
        lse = torch.logsumexp(logit, 1)
        zy = logit[rows, y]
        logit -= lse[:, None]
        out = dict(logp=(zy - lse) * keep, entropy=-(torch.exp(logit) * logit).sum(1) * keep, lse=lse)
        if case["K"]:
            out["top_ids"], out["top_logp"] = ids, top - lse[:, None]
        return out
    if case["op"] == "grad":
        # L = sum_t g_logp logp + g_entropy H, by the chain rule through p = exp(logit - lse)
        logit *= case["scale"]
        logit -= f("lse")[:, None]
        p = torch.exp(logit)
        dz = -(logit + f("entropy")[:, None]) * p * (f("g_entropy") * keep)[:, None]
        gl = f("g_logp") * keep
        dz -= p * gl[:, None]
        dz[rows, y] += gl
        dz *= case["scale"]
        dW = torch.zeros(s["W"].shape, dtype=torch.float64, device="cuda")
        dW[:V] = torch.matmul(dz.t(), f("h"))
        return dict(dH=torch.matmul(dz, f("W")[:V]), dW=dW)
    x = f("x")
    if case["op"] == "norm":
        mean = x.sum(1) / H if case["kind"] == "layer" else torch.zeros(T, dtype=torch.float64, device="cuda")
        dev = x - mean[:, None]
        rstd = torch.rsqrt(dev.square().sum(1) / H + s["eps"])
        y = dev * rstd[:, None] * f("weight") + (f("bias") if case["bias"] else 0.0)
        out = dict(y=y, rstd=rstd)
        if case["kind"] == "layer":
            out["mean"] = mean
        return out
    rstd = f("rstd")[:, None]
    unit = (x - (f("mean")[:, None] if case["kind"] == "layer" else 0.0)) * rstd
    up = f("dy") * f("weight")
    back = up - unit * (up * unit).sum(1, keepdim=True) / H
    if case["kind"] == "layer":
        back -= up.sum(1, keepdim=True) / H
    out = dict(dx=back * rstd, dweight=torch.einsum("th,th->h", f("dy"), unit))
    if case["bias"]:
        out["dbias"] = f("dy").sum(0)
    return out
