"""One layer around the MoE block, trained to follow a teacher:  python -m top_softmax_router_gb300.example_layer

    h    = embedding[tokens]
    n1   = layer_norm(h);  idx, gates = expert scores of n1 Wr^T (sigmoid, balance bias, groups)
    h2   = h + experts(n1, idx, gates)
    loss = distillation of the head  layer_norm(h2) W^T  from the teacher's top logits

Every operator is the library's; the router's product and the sums are torch's.  After each step the bias of experts
that took more tokens than the average is lowered, and that of the others raised.
"""
from __future__ import annotations

import argparse
import dataclasses

import torch

import top_softmax_router_gb300 as M


@dataclasses.dataclass(frozen=True)
class Sizes:
    N: int = 1024      # tokens
    V: int = 8000      # vocabulary
    H: int = 512
    E: int = 16
    k: int = 4
    I: int = 256
    K: int = 16        # teacher logits a token
    groups: int = 4
    topk_groups: int = 2
    P: int = 2         # vocabulary strips of the head's backward


class Layer:
    """The layer's parameters (bf16, router and norms fp32) and the library's units for one shape."""

    def __init__(self, s: Sizes, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def param(*shape, std, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g) * std).to(device=device, dtype=dtype).requires_grad_()

        def ones():
            return torch.ones(s.H, device=device).requires_grad_(), torch.zeros(s.H, device=device).requires_grad_()

        self.s = s
        self.table = param(s.V, s.H, std=1.0)
        self.w1, self.b1 = ones()
        self.Wr = param(s.E, s.H, std=s.H ** -0.5, dtype=torch.float32)
        self.Wg, self.Wu = param(s.E, s.I, s.H, std=s.H ** -0.5), param(s.E, s.I, s.H, std=s.H ** -0.5)
        self.Wd = param(s.E, s.H, s.I, std=s.I ** -0.5)
        self.w2, self.b2 = ones()
        self.head = param(s.V, s.H, std=s.H ** -0.5)
        self.balance = torch.zeros(s.E, device=device)
        self.embed = M.TokenEmbedding(M.EmbeddingConfig(N=s.N, V=s.V, H=s.H), device)
        self.norm = M.LayerNorm(M.LayerNormConfig(N=s.N, H=s.H), device)
        self.router = M.ScoreRouter(M.ScoreRouterConfig(N=s.N, E=s.E, k=s.k, groups=s.groups, topk_groups=s.topk_groups,
                                                        score="sigmoid"), device)
        self.block = M.MoEBlock(M.Config(N=s.N, H=s.H, E=s.E, k=s.k, I=s.I, c=s.N, K_max=1), device)
        self.distill = M.VocabDistill(M.DistillConfig(N=s.N, H=s.H, V=s.V, K=s.K, P=s.P, temperature=2.0), device)

    def parameters(self):
        return [self.table, self.w1, self.b1, self.Wr, self.Wg, self.Wu, self.Wd, self.w2, self.b2, self.head]

    def loss(self, tokens, t_ids, t_logits):
        """(loss, counts): the mean distillation loss, and how many tokens each expert took."""
        h = M.token_embedding(tokens, self.table, self.embed)
        n1 = M.layer_norm(h, self.w1, self.b1, self.norm)
        idx, gates, counts = M.expert_scores(n1.float() @ self.Wr.t(), self.router, self.balance)
        h2 = h + M.moe_experts(n1, idx, gates, self.Wg, self.Wu, self.Wd, self.block)
        n2 = M.layer_norm(h2, self.w2, self.b2, self.norm)
        return M.vocab_distill(n2, self.head, t_ids, t_logits, self.distill), counts

    def step(self, tokens, t_ids, t_logits, rate: float = 0.02, balance_rate: float = 1e-3):
        """One step of gradient descent in which each parameter moves by `rate` of its own size (a vector near zero: of
        one); returns the loss before it."""
        loss, counts = self.loss(tokens, t_ids, t_logits)
        loss.backward()
        with torch.no_grad():
            for p in self.parameters():
                size = p.float().norm().clamp(min=1.0 if p.dim() == 1 else 0.0)
                p -= (rate * size / p.grad.float().norm().clamp(min=1e-20) * p.grad.float()).to(p.dtype)
                p.grad = None
            mean = self.s.N * self.s.k / self.s.E
            self.balance -= balance_rate * torch.sign(counts.float() - mean)
        return loss.detach()

    def check(self):
        for unit in (self.embed, self.norm, self.router, self.block, self.distill):
            unit.check()


def batch(s: Sizes, seed: int = 1, device="cuda"):
    """Tokens whose frequency falls as 1 / rank, and a teacher that knows each token's K classes."""
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(s.N, generator=g, dtype=torch.float64)
    tokens = ((torch.tensor(s.V + 1.0, dtype=torch.float64) ** u) - 1).long().clamp_(0, s.V - 1)
    near = torch.arange(s.K) * (s.V // s.K)
    t_ids = ((tokens[:, None] * 7 + near) % s.V).int()
    t_logits = torch.randn(s.N, s.K, generator=g) + 4.0 * torch.linspace(1, 0, s.K)
    return tokens.to(device), t_ids.to(device), t_logits.to(device)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=0.02)
    a = ap.parse_args()
    s = Sizes()
    layer, data = Layer(s), batch(s)
    for i in range(a.steps):
        loss = layer.step(*data, rate=a.rate)
        if i % 5 == 0 or i + 1 == a.steps:
            print(f"step {i}: loss {loss.item():.4f}", flush=True)
    layer.check()


if __name__ == "__main__":
    main()
