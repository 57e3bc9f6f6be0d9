"""Policy-gradient training and decoding of a tied embedding and head.

    python examples/policy_step.py [--steps 60] [--tokens 512] [--vocab 1000] [--hidden 128]

The smallest model that uses the library's calls together: a token's embedding,
one matrix for a trunk, layer norm, and the head over the embedding's weights,
which learns to answer token v with (7 v + 3) mod V from scored rollouts. One
training step is

    vce_embed_fwd_plan   e = W[ids], with the embedding backward's plan beside it
    (torch)              x = e M
    vce_norm_fwd         h = norm(x)
    vce_logprob_fwd      logp, entropy and lse of the rollout's tokens
    (torch)              clipped ratio objective: its slope per token
    vce_logprob_bwd      dh, and dW of the head
    vce_norm_bwd         dx, and the norm's weight and bias gradients
    (torch)              de = dx M^T, dM = e^T dx
    vce_embed_bwd_apply  dW += the embedding's gradient
    (torch)              Adam on the fp32 weights

and decoding a batch takes the first of vce_logprob_fwd's alternatives of each
token. Nothing is read back inside a step. Workspaces and outputs are allocated
once and kept.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from vocab_embedding_cross_gb300 import _lib as vce  # noqa: E402
from vocab_embedding_cross_gb300 import device as D  # noqa: E402


class TiedPolicy:
    def __init__(self, T: int, H: int, V: int, seed: int = 0):
        Vp = -(-V // 64) * 64
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.H, self.V = T, H, V
        self.p = vce.problem(T, H, Vp, V, 1, vce.VCE_BF16, tied=True)
        self.master = torch.randn(Vp, H, generator=g, device="cuda") * 0.02
        self.trunk = torch.randn(H, H, generator=g, device="cuda") / H ** 0.5
        self.norm_w, self.norm_b = torch.ones(H, device="cuda"), torch.zeros(H, device="cuda")
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.e, self.h, self.dx = bf16(T, H), bf16(T, H), bf16(T, H)
        self.mean, self.rstd = f32(T), f32(T)
        self.logp, self.entropy, self.lse = f32(T), f32(T), f32(T)
        self.dh, self.dW, self.dnw, self.dnb = f32(T, H), f32(Vp, H), f32(H), f32(H)
        self.round()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        size = lambda op: vce.vce_workspace_size(self.p, op)  # noqa: E731
        self.ws_embed = D.workspace(size(vce.VCE_OP_EMBED_BWD))
        self.ws_norm = D.workspace(size(vce.VCE_OP_NORM_BWD))
        self.ws_bwd = D.workspace(size(vce.VCE_OP_LOGPROB_BWD))
        self.ws_fwd = D.workspace(vce.vce_logprob_workspace_size(self.p, 0))

    def round(self):
        """The bf16 weights that the calls take, from the fp32 ones."""
        self.W, self.M = self.master.bfloat16(), self.trunk.bfloat16()
        self.nw, self.nb = self.norm_w.bfloat16(), self.norm_b.bfloat16()

    def scores(self, ids, targets):
        """logp, entropy and lse of `targets` after `ids`; keeps what the backward needs."""
        st = self.status
        vce.vce_embed_fwd_plan(self.p, ids, self.W, self.e, self.ws_embed, dev_status=st)
        self.x = self.e @ self.M
        vce.vce_norm_fwd(self.p, self.x, self.nw, self.nb, self.h, self.mean, self.rstd, dev_status=st)
        vce.vce_logprob_fwd(self.p, self.h, self.W, targets, self.logp, self.entropy, self.lse, ws=self.ws_fwd,
                            dev_status=st)
        return self.logp

    def gradient(self, ids, targets, old_logp, advantage, beta=0.01, clip=0.2):
        """Gradient of -mean(min(r A, clip(r) A)) - beta mean(entropy), r = exp(logp - old_logp)."""
        logp = self.scores(ids, targets)
        r = torch.exp(logp - old_logp)
        passes = torch.where(advantage >= 0, r < 1 + clip, r > 1 - clip)   # the clipped side has no slope
        g_logp = torch.where(passes, -r * advantage, 0.0) / self.T
        g_entropy = torch.full_like(logp, -beta / self.T)
        self.dW.zero_()
        st = self.status
        vce.vce_logprob_bwd(self.p, self.h, self.W, targets, self.lse, self.entropy, g_logp, g_entropy, self.dh,
                            self.dW, self.ws_bwd, dev_status=st)
        vce.vce_norm_bwd(self.p, self.x, self.nw, self.dh, self.mean, self.rstd, self.dx, self.dnw, self.dnb,
                         self.ws_norm, dev_status=st)
        self.dM = (self.e.T @ self.dx).float()
        vce.vce_embed_bwd_apply(self.p, self.dx @ self.M.T, self.dW, self.ws_embed, dev_status=st)

    def update(self, optimiser):
        for weight, grad in ((self.master, self.dW), (self.trunk, self.dM), (self.norm_w, self.dnw),
                             (self.norm_b, self.dnb)):
            weight.grad = grad
        optimiser.step()
        self.round()

    def decode(self, ids, n, alternatives=4):
        """n greedy steps for a batch of tokens: [B, n + 1] ids and the last step's alternatives."""
        B = ids.numel()
        p = vce.problem(B, self.H, self.p.Vp, self.V, 1, vce.VCE_BF16)
        e, h = (torch.empty((B, self.H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        top = torch.empty((B, alternatives), dtype=torch.int64, device="cuda")
        top_logp, entropy = torch.empty((B, alternatives), device="cuda"), torch.empty(B, device="cuda")
        ws = D.workspace(vce.vce_logprob_workspace_size(p, alternatives))
        out = [ids]
        for _ in range(n):
            vce.vce_embed_fwd(p, out[-1], self.W, e)
            vce.vce_norm_fwd(p, e @ self.M, self.nw, self.nb, h)
            vce.vce_logprob_fwd(p, h, self.W, None, None, entropy, None, top, top_logp, ws=ws, dev_status=self.status)
            out.append(top[:, 0].contiguous())
        return torch.stack(out, 1), top, top_logp, entropy


def train(steps=60, T=512, V=1000, H=128, lr=0.01, seed=0, log=None):
    m = TiedPolicy(T, H, V, seed)
    optimiser = torch.optim.Adam([m.master, m.trunk, m.norm_w, m.norm_b], lr=lr)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    for step in range(steps):
        ids = torch.randint(0, V, (T,), generator=g, device="cuda")
        right = (7 * ids + 3) % V
        # a scored rollout: three in four answers are right, the others random and marked down
        good = torch.rand(T, generator=g, device="cuda") < 0.75
        answer = torch.where(good, right, torch.randint(0, V, (T,), generator=g, device="cuda"))
        advantage = torch.where(good, 1.0, -0.25)
        old = m.scores(ids, answer).clone()
        for _ in range(2):   # two passes over the rollout
            m.gradient(ids, answer, old, advantage)
            m.update(optimiser)
        if log and (step % 10 == 9 or step == 0):
            lp = m.scores(ids, right)
            log(f"step {step + 1}: mean logp of the right answer {lp.mean().item():.3f}, entropy "
                f"{m.entropy.mean().item():.3f}")
    return m


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--hidden", type=int, default=128)
    ap.add_argument("--lr", type=float, default=0.01)
    a = ap.parse_args(argv)
    m = train(a.steps, a.tokens, a.vocab, a.hidden, a.lr, log=print)
    ids, top, top_logp, entropy = m.decode(torch.arange(8, device="cuda"), 5)
    print("decoded:", ids.tolist())
    right = ((7 * ids[:, :-1] + 3) % a.vocab == ids[:, 1:]).float().mean().item()
    print(f"right answers {right:.2f}; last alternatives {top[0].tolist()} at "
          f"{[round(v, 2) for v in top_logp[0].tolist()]}, entropy {entropy[0].item():.2f}")
    status = int(m.status.item())
    if status:
        print(vce.status_str(status))
    return 1 if status else 0


if __name__ == "__main__":
    sys.exit(main())
