"""The 8-bit path as a layer uses it: RMS norm with 8-bit output, products by expert, checkpoints, under autograd."""
import pytest
import torch

from gpu_util import lib_api, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    need_gpu()
    return lib_api()


N, H, I, E = 500, 384, 272, 5
ENDS = [0, 130, 130, 131, 400, 480]          # an expert without rows, one with a single row, 20 rows of nobody


def make(M, seed=0):
    g = torch.Generator().manual_seed(seed)

    def t(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).bfloat16().cuda()

    v = dict(x=t(N, H), r=t(N, H), weight=(torch.rand(H, generator=g) + 0.5).cuda(), w1=t(E, I, H, std=H ** -0.5),
             w2=t(E, H, I, std=I ** -0.5), g=t(N, H, std=0.1), gh=t(N, H, std=0.1))
    off = torch.tensor(ENDS, dtype=torch.int32, device="cuda")
    units = (M.RMSNorm(M.RMSNormConfig(N=N, H=H)), M.ExpertLinear(M.ExpertLinearConfig(N=N, K=H, O=I, E=E, blocks8=True)),
             M.ExpertLinear(M.ExpertLinearConfig(N=N, K=I, O=H, E=E, blocks8=True)))
    return v, off, units


def layer(M, v, off, units):
    a, h = M.rms_norm_linear8(v["x"], v["weight"], v["w1"], units[0], units[1], residual=v["r"], offsets=off)
    return h + M.expert_linear(torch.nn.functional.silu(a), v["w2"], units[2], off, keep="checkpoint8")


def grads(M, v, off, units):
    names = ("x", "r", "weight", "w1", "w2")
    leaves = {k: v[k].detach().requires_grad_() for k in names}
    out = layer(M, {**v, **leaves}, off, units)
    return (out, *torch.autograd.grad(out, [leaves[k] for k in names], v["g"]))


def test_against_float64(M):
    """The layer in fp64 with the same codes of weights and of the norm's output.  A bf16 rounding is off by at most 2^-8,
    three follow each other on the way to the output; dy's codes and the checkpoint are off by at most 2^-4 from the values
    they stand for, uniformly spread: 2^-4 / sqrt(3) of a gradient's 2-norm each, two of them meet on the way to x."""
    v, off, units = make(M)
    out, dx, dr, dweight, dw1, dw2 = grads(M, v, off, units)
    for u in units[1:]:
        u.check()
    d = {k: t.double().requires_grad_() for k, t in v.items()}
    _, h8, rstd, c, s = units[0].forward(v["x"], v["weight"], v["r"], want_codes=True)
    y8 = M.Checkpoint8(M.Checkpoint8Config(N=N, H=H)).unpack(c, s).double()
    wc, ws = M.pack_weight8(v["w1"])
    w8 = wc.double() * ws.double().repeat_interleave(128, 1)[:, :I].repeat_interleave(128, 2)[:, :, :H]
    h = d["x"] + d["r"]
    h = h + (h8.double() - h).detach()
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-6) * d["weight"]
    y = y + (y8 - y).detach()                      # gradients pass through the roundings
    w1 = d["w1"] + (w8 - d["w1"]).detach()
    parts = []
    for e in range(E):
        a = y[ENDS[e]:ENDS[e + 1]] @ w1[e].t()
        parts.append(torch.nn.functional.silu(a) @ d["w2"][e].t())
    ref = h + torch.cat(parts + [torch.zeros(N - ENDS[-1], H, dtype=torch.float64, device="cuda")])
    want = torch.autograd.grad(ref, [d[k] for k in ("x", "r", "weight", "w1", "w2")], v["g"].double())

    def off_by(got, ref):
        return ((got.double() - ref).norm() / ref.norm()).item()

    assert off_by(out, ref) < 3 * 2.0 ** -8
    one = 2.0 ** -4 / 3 ** 0.5 + 3 * 2.0 ** -8
    for got, r, bound in zip((dx, dr, dweight, dw1, dw2), want, (one, one, one, 4 * 2.0 ** -8, one)):
        assert got.dtype == (torch.float32 if got is dweight else torch.bfloat16)
        assert off_by(got, r) < bound
    assert torch.equal(dx, dr)
    assert torch.all(dw1[1] == 0) and torch.all(dw2[1] == 0)


def test_wrappers_give_the_units_bits(M):
    v, off, (norm, up, down) = make(M, 3)
    x, r, w = (v[k].detach().requires_grad_() for k in ("x", "r", "weight"))
    y, h = M.rms_norm(x, w, norm, residual=r)
    got = torch.autograd.grad((y, h), (x, r, w), (v["g"], v["gh"]))
    y2, h2, rstd, _, _ = norm.forward(v["x"], v["weight"], v["r"])
    dx, dw = norm.backward(h2, v["weight"], rstd, v["g"], v["gh"])
    assert torch.equal(y, y2) and torch.equal(h, h2)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dx) and torch.equal(got[2], dw)
    only_h = torch.autograd.grad(M.rms_norm(x, w, norm, residual=r)[1], x, v["gh"])[0]
    assert torch.equal(only_h, v["gh"])
    alone = torch.autograd.grad(M.rms_norm(x, w, norm), (x, w), v["g"])
    _, _, rstd, _, _ = norm.forward(v["x"], v["weight"])
    assert all(torch.equal(p, q) for p, q in zip(alone, norm.backward(v["x"], v["weight"], rstd, v["g"])))
    a = v["x"][:, :I].contiguous()
    ck = M.Checkpoint8(M.Checkpoint8Config(N=N, H=I))
    ac, asc = ck.pack(a)
    wc, ws = M.pack_weight8(v["w2"])
    forms = {"bf16": (a, None, v["w2"], None), "checkpoint8": (ac, asc, v["w2"], None), "blocks8": (ac, asc, wc, ws)}
    for keep, (xk, xs, wk, wks) in forms.items():
        al, wl = a.detach().requires_grad_(), v["w2"].detach().requires_grad_()
        y = M.expert_linear(al, wl, down, off, keep=keep)
        got = torch.autograd.grad(y, (al, wl), v["g"])
        assert torch.equal(y, down.forward(xk, wk, off, xs, wks) if keep == "blocks8" else down.forward(a, wk, off))
        want = down.backward(xk, wk, v["g"], off, xs, wks, dw_dtype=torch.bfloat16)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    with pytest.raises(ValueError, match="keep"):
        M.expert_linear(a, v["w2"], down, off, keep="fp8")
    with pytest.raises(RuntimeError, match="twice"):
        g, = torch.autograd.grad(M.rms_norm(x, w, norm).sum(), x, create_graph=True)
        g.sum().backward()


def test_the_layer_in_a_graph(M):
    """Forward and backward captured together: replays on new contents give the eager bits."""
    v, off, units = make(M)
    other = make(M, 9)[0]
    want = [tuple(t.clone() for t in grads(M, q, off, units)) for q in (other, v)]
    held = {k: t.clone() for k, t in v.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads(M, held, off, units)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = grads(M, held, off, units)
    for q, w in zip((other, v), want):
        for k in held:
            held[k].copy_(q[k])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_one_token_at_a_time(M):
    """A decode step: the rows of a batch one by one, each its expert's, as the batch gives them."""
    v, off, (norm, up, _) = make(M, 5)
    wc, ws = M.pack_weight8(v["w1"])
    _, _, _, c, s = norm.forward(v["x"], v["weight"], v["r"], want_y=False, want_codes=True)
    whole = up.forward(c, wc, off, s, ws)
    for n, e in ((0, 0), (130, 2), (300, 3)):
        _, _, _, c1, s1 = norm.forward(v["x"][n:n + 1], v["weight"], v["r"][n:n + 1], want_y=False, want_codes=True)
        assert torch.equal(c1.view(torch.uint8), c[n:n + 1].view(torch.uint8))
        at = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        at[e + 1:] = 1
        y = up.forward(c1, wc, at, s1, ws)
        # shares of K add in another order: 2^-23 (K / 16 + 32) of the terms' magnitudes, and a step of bf16
        size = c1.float().abs() * s1.float().repeat_interleave(128, 1) @ (wc[e].float().abs() * ws[e].float().repeat_interleave(128, 0)[:I].repeat_interleave(128, 1)[:, :H]).t()
        assert torch.all((y - whole[n]).float().abs() <= 2.0 ** -7 * whole[n].float().abs() + (H / 16 + 32) * 2.0 ** -22 * size)
    up.check()
