"""The autograd wrappers of the layer operators and of the older functions, with stand-in units on the host."""
import pytest
import torch


@pytest.fixture(scope="module")
def M():
    import top_softmax_router_gb300 as M
    return M


class Norm:
    def forward(self, x, weight, bias):
        return x * weight, x.mean(1), x.std(1)

    def backward(self, x, weight, mean, rstd, dy, want_dx, want_dweight, want_dbias):
        return dy * weight, (dy * x).sum(0), dy.sum(0)


class Embedding:
    def forward(self, ids, table):
        return table[ids] * table[ids]

    def backward(self, ids, dy):
        return torch.zeros(5, 4).index_add_(0, ids, dy)


class Router:
    def forward(self, logits, bias):
        idx = logits.argsort(dim=1, descending=True)[:, :2].int()
        return idx, torch.softmax(logits, dim=1).gather(1, idx.long()), torch.bincount(idx.flatten(), minlength=4)

    def backward(self, logits, idx, dweights):
        return torch.zeros_like(logits).scatter_(1, idx.long(), dweights)


class Block:
    def route(self, X, Wr, bias):
        return torch.zeros(X.shape[0], 1, dtype=torch.int32), torch.ones(X.shape[0], 1)

    def forward(self, X, idx, gates, Wg, Wu, Wd):
        return X * X * gates

    def experts_backward(self, X, idx, gates, Wg, Wu, Wd, dY):
        return dict(dX=2 * X * dY, dgates=(X * X * dY).sum(1, keepdim=True), dWg=Wg * 0, dWu=Wu * 0, dWd=Wd * 0)

    def backward(self, X, Wr, idx, gates, Wg, Wu, Wd, dY, want_dgates):
        return self.experts_backward(X, idx, gates, Wg, Wu, Wd, dY) | dict(dWr=Wr * 0)


class Head:
    def forward(self, X, W, *_):
        z = X @ W.t()
        return (z * z).sum(1), z.sum(1), (z * z).sum(1).mean().view(1)

    def backward(self, X, W, *_, dW_dtype=None):
        return X + 0, W + 0


def leaf(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(3)).requires_grad_()


def calls(M):
    x = leaf(3, 4)
    w = torch.randn(4, 4)
    ids, t = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    table = leaf(5, 4)
    return {
        "layer_norm": (x, lambda: M.layer_norm(x, torch.ones(4), torch.zeros(4), Norm())),
        "token_embedding": (table, lambda: M.token_embedding(torch.tensor([0, 3, 3]), table, Embedding())),
        "expert_scores": (x, lambda: M.expert_scores(x, Router())[1]),
        "moe_experts": (x, lambda: M.moe_experts(x, ids[:, :1], torch.ones(3, 1), w, w, w, Block())),
        "vocab_distill": (x, lambda: M.vocab_distill(x, w, ids, t, Head())),
        "moe_block": (x, lambda: M.moe_block(x, w, None, w, w, w, Block())),
        "vocab_cross_entropy": (x, lambda: M.vocab_cross_entropy(x, w, ids[:, 0], Head())),
    }


NAMES = ["layer_norm", "token_embedding", "expert_scores", "moe_experts", "vocab_distill", "moe_block", "vocab_cross_entropy"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("upstream", ["constant", "of the output"])
def test_a_second_derivative_is_refused(M, name, upstream):
    """The gradients are the library's kernels' and have no graph: differentiated again they would count as constants."""
    if name == "token_embedding" and upstream == "constant":
        pytest.skip("the lookup is linear in its table: its gradient is a constant there")
    x, f = calls(M)[name]
    y = f().sum() if upstream == "constant" else f().pow(2).sum()
    g, = torch.autograd.grad(y, x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated twice"):
        ((g * g).sum() + (x * x).sum()).backward()


@pytest.mark.parametrize("name", NAMES)
def test_a_first_derivative_is_the_unit_s(M, name):
    x, f = calls(M)[name]
    a, = torch.autograd.grad(f().sum(), x)
    b, = torch.autograd.grad(f().sum(), x, create_graph=True)
    assert torch.equal(a, b) and a.shape == x.shape and a.any() and not a.requires_grad
    x.grad = None
    f().sum().backward()
    assert torch.equal(x.grad, a)
