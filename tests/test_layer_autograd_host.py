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


class Linear:
    """Products by expert of a unit made without room for the backward pass of operands in 8 bits, or with it."""

    def __init__(self, M, blocks8=False):
        self.cfg = M.ExpertLinearConfig(N=8, K=16, O=32, blocks8=blocks8)
        self.calls = []

    def forward(self, x, w, offsets, x_scales=None, w_scales=None):
        self.calls.append("forward")
        return x @ w[0].t()

    def backward(self, x, w, dy, offsets, x_scales, w_scales, want_dx, want_dw, dw_dtype):
        self.calls.append(("x" if x is not None else "no x", "scales" if x_scales is not None else "no scales", want_dx, want_dw))
        return dy @ w[0] if want_dx else None, (dy.t() @ x)[None].to(dw_dtype) if want_dw else None


def linear_inputs(dtype=torch.bfloat16):
    return torch.randn(8, 16).bfloat16(), torch.randn(1, 32, 16).to(dtype)


def test_what_the_backward_pass_could_not_do_is_refused_before_the_forward(M):
    """Weights in fp16, in which no gradient is made, and units without room for operands in 8 bits."""
    x, w = linear_inputs(torch.float16)
    room, none = Linear(M, True), Linear(M)
    with pytest.raises(TypeError, match="w: expected bfloat16 or float32"):
        M.expert_linear(x, w.requires_grad_(), room, keep="blocks8")
    with pytest.raises(TypeError, match="w: expected bfloat16 or float32"):
        M.rms_norm_linear8(x, None, w, None, room)
    x, w = linear_inputs()
    for a, b, keep in ((x, w.clone().requires_grad_(), "checkpoint8"), (x, w.clone().requires_grad_(), "blocks8"),
                       (x.clone().requires_grad_(), w, "blocks8")):
        with pytest.raises(ValueError, match="blocks8"):
            M.expert_linear(a, b, none, keep=keep)
    with pytest.raises(ValueError, match="blocks8"):
        M.rms_norm_linear8(x, torch.ones(16, requires_grad=True), w, None, none)
    assert not room.calls and not none.calls


def test_a_checkpoint_is_only_made_for_the_weights_gradient(M):
    """Packing x takes a GPU: on the host it would raise."""
    x, w = linear_inputs()
    unit = Linear(M)
    y = M.expert_linear(x, w, unit, keep="checkpoint8")
    assert torch.equal(y, x @ w[0].t()) and unit.calls == ["forward"]
    with torch.no_grad():
        assert torch.equal(M.expert_linear(x, w.clone().requires_grad_(), unit, keep="checkpoint8"), y)
    a = x.clone().requires_grad_()
    dy = torch.randn(8, 32).bfloat16()
    dx, = torch.autograd.grad(M.expert_linear(a, w, unit, keep="checkpoint8"), a, dy)
    assert torch.equal(dx, dy @ w[0]) and unit.calls[-1] == ("no x", "no scales", True, False)
