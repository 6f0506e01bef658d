"""The layer of example_layer.py: its operators together against the same layer in torch, fp64, and the autograd
wrappers one by one where they differ from the direct calls.

Tolerance of a gradient: the activations between the operators are bf16 (2^-8 each), about a dozen of them in a row:
a relative 2-norm error of 12 x 2^-8 = 0.05 at most; the loss, a mean over tokens of values with independent errors of
2^-8 of their size: 2^-6.
"""
import pytest
import torch

from gpu_util import lib_api, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    need_gpu()
    return lib_api()


def reference(layer, tokens, t_ids, t_logits, idx):
    """The layer in fp64 by torch's autograd, for the experts that the library chose."""
    s = layer.s
    P = [p.detach().double().requires_grad_() for p in layer.parameters()]
    table, w1, b1, Wr, Wg, Wu, Wd, w2, b2, head = P

    def norm(x, w, b):
        return torch.nn.functional.layer_norm(x, (s.H,), w, b, 1e-5)

    h = table[tokens]
    n1 = norm(h, w1, b1)
    score = torch.sigmoid(n1 @ Wr.t()).gather(1, idx.long())
    gates = score / score.sum(dim=1, keepdim=True)
    out = torch.zeros_like(h)
    for e in range(s.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        x = n1[t]
        y = (torch.nn.functional.silu(x @ Wg[e].t()) * (x @ Wu[e].t())) @ Wd[e].t()
        out = out.index_add(0, t, y * gates[t, j][:, None])
    z = norm(h + out, w2, b2) @ head.t() / 2.0
    q = torch.softmax(t_logits.double() / 2.0, dim=1)
    logp = torch.log_softmax(z, dim=1).gather(1, t_ids.long())
    loss = 4.0 * (q * (q.log() - logp)).sum(dim=1).mean()
    loss.backward()
    return loss.detach(), [p.grad for p in P]


def test_the_layer_against_torch(M):
    from top_softmax_router_gb300.example_layer import Layer, Sizes, batch
    s = Sizes(N=384, V=1000, H=256, E=8, k=3, I=128, K=8)
    layer, data = Layer(s), batch(s)
    loss, counts = layer.loss(*data)
    loss.backward()
    layer.check()
    h = layer.embed.forward(data[0], layer.table.detach())
    n1 = layer.norm.forward(h, layer.w1.detach(), layer.b1.detach())[0]
    idx, _, again = layer.router.forward(n1.float() @ layer.Wr.detach().t(), layer.balance)
    assert torch.equal(counts, again) and counts.sum().item() == s.N * s.k
    ref, grads = reference(layer, *data, idx)
    assert abs(loss.item() - ref.item()) <= 2.0 ** -6 * abs(ref.item())
    for name, p, g in zip("table w1 b1 Wr Wg Wu Wd w2 b2 head".split(), layer.parameters(), grads):
        off = (p.grad.double() - g).norm() / g.norm()
        assert p.grad.dtype == p.dtype and off <= 0.05, (name, off.item())


def test_the_example_learns(M):
    from top_softmax_router_gb300.example_layer import Layer, Sizes, batch
    s = Sizes(N=512, V=2000, H=256, E=8, I=128)
    layer, data = Layer(s), batch(s)
    losses = [layer.step(*data).item() for _ in range(12)]
    layer.check()
    assert losses[-1] < 0.9 * losses[0]
    assert layer.balance.abs().sum() > 0


def test_experts_backward_is_the_block_without_its_router(M):
    """The same experts' gradients as moe_backward with a router of zeros (whose part of dX is then exactly 0)."""
    g = torch.Generator().manual_seed(0)
    N, H, E, k, I = 300, 128, 8, 2, 64
    for c, K_max in ((N, 1), (100, 3)):
        blk = M.MoEBlock(M.Config(N=N, H=H, E=E, k=k, I=I, c=c, K_max=K_max))
        X, dY = (torch.randn(N, H, generator=g).bfloat16().cuda() for _ in range(2))
        Wg, Wu = ((torch.randn(E, I, H, generator=g) * H ** -0.5).bfloat16().cuda() for _ in range(2))
        Wd = (torch.randn(E, H, I, generator=g) * I ** -0.5).bfloat16().cuda()
        idx = torch.rand(N, E, generator=g).argsort(dim=1)[:, :k].int().contiguous().cuda()
        idx[idx == 3] = 4                         # an expert without tokens (a token may take one twice)
        gates = torch.rand(N, k, generator=g).cuda()
        got = blk.experts_backward(X, idx, gates, Wg, Wu, Wd, dY)
        ref = blk.backward(X, torch.zeros(E, H, device="cuda"), idx, gates, Wg, Wu, Wd, dY)
        blk.check()
        assert not got["dWg"][3].any() and not got["dWd"][3].any()
        for n, t in got.items():
            assert torch.equal(t, ref[n]), n


def test_expanded_gradients_and_unwanted_ones(M):
    ln = M.LayerNorm(M.LayerNormConfig(N=6, H=40))
    x = torch.randn(6, 40, device="cuda", requires_grad=True)
    w = torch.ones(40, device="cuda", requires_grad=True)
    M.layer_norm(x, w, None, ln).sum().backward()          # the gradient of a sum is one value, expanded
    assert x.grad.abs().max() < 1e-4 and w.grad.shape == (40,)
    x2 = x.detach()
    b = torch.zeros(40, device="cuda", requires_grad=True)
    M.layer_norm(x2, w.detach(), b, ln).sum().backward()
    assert torch.equal(b.grad, torch.full((40,), 6.0, device="cuda"))
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=6, V=9, H=40))
    table = torch.randn(9, 40, device="cuda", dtype=torch.bfloat16).requires_grad_()
    ids = torch.tensor([1, 1, 8, 0, 1, 3], device="cuda")
    M.token_embedding(ids, table, emb).sum().backward()
    assert torch.equal(table.grad[:, 0].float().cpu(), torch.tensor([1.0, 3, 0, 1, 0, 0, 0, 0, 1]))
    assert table.grad.dtype == torch.bfloat16
