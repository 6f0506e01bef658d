"""Layer norm on the GPU against the float64 oracle, forward and backward.

Tolerances, from the arithmetic before any run (u = 2^-24, one fp32 rounding):
  mean   a tree over at most 16 values a thread and 1024 threads adds at most 16 + 15 roundings of values
         bounded by mean |x|, and one for the product: 32 u mean|x|
  rstd   the same for the variance, the square root and division, half of it by the square root: relative 24 u,
         and the mean's error d enters as d^2 / var: negligible for the inputs here (|mean| <= std)
  y      (x - mean) rstd weight + bias: 40 u (|xh weight| + |weight| rstd mean|x| + |bias|) + half a step of y
  dx     the same, of rstd |weight| terms: 64 u rstd (|t| + mean|t| + |xh| mean|t xh|) + half a step
  dweight, dbias   fp32 sums over n rows in up to 608 blocks: at most n + 8 + 608 / 8 roundings of the running
         sum in the worst case; the random walk of independent roundings is its square root, taken with
         factor 8: 8 sqrt(n + 90) u sqrt(sum terms^2) + 48 u sum|terms| / sqrt(n) (each term's own error)
"""
import numpy as np
import pytest
import torch

from gpu_util import lib_api, need_gpu
from oracle import layer_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def M():
    need_gpu()
    return lib_api()


def host(t):
    return t.detach().double().cpu().numpy()


def inputs(n, h, t, pt, seed=0, mean=0.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(n, h, generator=g) * 2 + mean).to(TYPES[t])
    w = (torch.randn(h, generator=g) * 0.3 + 1).to(TYPES[pt])
    b = (torch.randn(h, generator=g) * 0.3).to(TYPES[pt])
    dy = torch.randn(n, h, generator=g).to(TYPES[t])
    return x, w, b, dy


def check(M, x, w, b, dy, eps=1e-5, unit=None, place=lambda t: t.cuda()):
    n, h = x.shape
    ln = unit or M.LayerNorm(M.LayerNormConfig(N=n, H=h, eps=eps))
    xd, dyd = place(x), place(dy)
    wd, bd = (None if p is None else p.cuda() for p in (w, b))
    y, mean, rstd = ln.forward(xd, wd, bd)
    dx, dw, db = ln.backward(xd, wd, mean, rstd, dyd)
    X, DY = host(x), host(dy)
    Wf, Bf = np.ones(h) if w is None else host(w), np.zeros(h) if b is None else host(b)
    ry, rm, rr = R.norm_forward(X, Wf, Bf, eps)
    rdx, rdw, rdb = R.norm_backward(X, Wf, DY, eps)
    half = torch.finfo(x.dtype).eps / 2
    ax = np.abs(X).mean(axis=1)
    xh = np.abs((X - rm[:, None]) * rr[:, None])
    tiny = 1e-30 if x.dtype != torch.float16 else 2.0 ** -25
    assert np.all(np.abs(host(mean) - rm) <= 32 * U * ax + 1e-30)
    assert np.all(np.abs(host(rstd) - rr) <= 24 * U * rr + 16 * U * ax * rr * rr * (32 * U * ax * rr + U) + 1e-30)
    bound = 40 * U * (xh * np.abs(Wf) + np.abs(Wf) * (rr * ax)[:, None] + np.abs(Bf)) + half * np.abs(ry) + tiny
    assert np.all(np.abs(host(y) - ry) <= bound)
    t = np.abs(DY * Wf)
    bound = 64 * U * rr[:, None] * (t + t.mean(axis=1, keepdims=True) + (xh + (rr * ax)[:, None]) *
                                    (t * (xh + (rr * ax)[:, None])).mean(axis=1, keepdims=True))
    assert np.all(np.abs(host(dx) - rdx) <= bound + half * np.abs(rdx) + tiny)
    walk = 8 * np.sqrt(n + 90) * U
    for got, ref, terms in ((dw, rdw, DY * (xh + (rr * ax)[:, None])), (db, rdb, DY)):
        l2, l1 = np.sqrt((terms ** 2).sum(axis=0)), np.abs(terms).sum(axis=0)
        assert got.dtype == torch.float32
        assert np.all(np.abs(host(got) - ref) <= walk * l2 + 48 * U * l1 / np.sqrt(n) + 1e-30)
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("t,pt", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                  ("fp16", "fp32")])
@pytest.mark.parametrize("n,h", [(1, 1), (1, 8), (3, 7), (5, 64), (130, 256), (33, 512), (17, 1000), (9, 1001),
                                 (300, 1024), (40, 2048), (7, 4100), (11, 7168), (3, 8192), (2, 8200), (2, 16384),
                                 (2, 16383)])
def test_against_the_oracle(M, t, pt, n, h):
    check(M, *inputs(n, h, t, pt, seed=n * h))


@pytest.mark.parametrize("n", [1, 2, 607, 609, 5000])
def test_many_rows(M, n):
    check(M, *inputs(n, 72, "bf16", "fp32", seed=n))


def test_without_parameters(M):
    x, w, b, dy = inputs(20, 320, "bf16", "bf16")
    check(M, x, None, None, dy)
    check(M, x, w, None, dy)
    check(M, x, None, b, dy)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,first", [(8, 0), (3, 0), (16, 8), (5, 3)])
def test_strided_rows(M, t, pad, first):
    """Rows of a wider buffer, aligned and not."""
    def place(v):
        wide = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=v.dtype, device="cuda")
        view = wide[:, first:first + v.shape[1]]
        view.copy_(v)
        return view
    check(M, *inputs(19, 264, t, "fp32", seed=3), place=place)


def test_a_unit_serves_fewer_rows_and_repeats_its_bits(M):
    ln = M.LayerNorm(M.LayerNormConfig(N=900, H=520))
    for n in (900, 1, 77):
        a = inputs(n, 520, "bf16", "fp32", seed=n)
        first = check(M, *a, unit=ln)
        again = check(M, *a, unit=ln)
        for p, q in zip(first, again):
            assert torch.equal(p, q)


def test_no_rows_and_partial_wants(M):
    ln = M.LayerNorm(M.LayerNormConfig(N=4, H=32))
    x = torch.empty(0, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    y, mean, rstd = ln.forward(x, w, w)
    dx, dw, db = ln.backward(x, w, mean, rstd, x)
    assert y.shape == (0, 32) and dx.shape == (0, 32) and not dw.any() and not db.any()
    x, w, b, dy = (v.cuda() for v in inputs(4, 32, "fp32", "fp32"))
    y, mean, rstd = ln.forward(x, w, b)
    whole = ln.backward(x, w, mean, rstd, dy)
    for i in range(3):
        wants = [j == i for j in range(3)]
        got = ln.backward(x, w, mean, rstd, dy, *wants)
        assert [g is not None for g in got] == wants and torch.equal(got[i], whole[i])


def test_constant_and_bad_rows_keep_to_themselves(M):
    x, w, b, dy = inputs(6, 640, "fp32", "fp32", seed=9)
    clean = x.clone()
    x[1] = 3.0                      # variance 0: y = bias
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    ln = M.LayerNorm(M.LayerNormConfig(N=6, H=640))
    y, mean, rstd = ln.forward(x.cuda(), w.cuda(), b.cuda())
    assert torch.equal(y[1].cpu(), b)
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).any()
    z = ln.forward(clean.cuda(), w.cuda(), b.cuda())[0]
    for r in (0, 2, 5):
        assert torch.equal(y[r], z[r])


def test_gradient_against_differences(M):
    """Central differences of sum(y dy) in fp32: the step's error h^2 f''' and rounding u |f| / h, at h = 2^-6 and
    |f| of a few hundred, leave 2e-3 of the gradients' scale."""
    x, w, b, dy = (v.cuda() for v in inputs(3, 24, "fp32", "fp32", seed=4))
    ln = M.LayerNorm(M.LayerNormConfig(N=3, H=24))

    def f(x, w, b):
        return (ln.forward(x, w, b)[0].double() * dy.double()).sum().item()

    _, mean, rstd = ln.forward(x, w, b)
    got = ln.backward(x, w, mean, rstd, dy)
    h = 2.0 ** -6
    for which, g in zip((0, 1, 2), got):
        args = [x, w, b]
        for i in range(0, args[which].numel(), 5):
            e = torch.zeros_like(args[which])
            e.view(-1)[i] = h
            up, dn = list(args), list(args)
            up[which], dn[which] = args[which] + e, args[which] - e
            assert abs((f(*up) - f(*dn)) / (2 * h) - g.view(-1)[i].item()) <= 2e-3 * max(1.0, g.abs().max().item())


def test_other_stream_and_graph(M):
    x, w, b, dy = (v.cuda() for v in inputs(50, 1024, "bf16", "fp32", seed=5))
    ln = M.LayerNorm(M.LayerNormConfig(N=50, H=1024))
    y, mean, rstd = ln.forward(x, w, b)
    ref = (y, mean, rstd) + ln.backward(x, w, mean, rstd, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, m2, r2 = ln.forward(x, w, b, stream=s)
    got = (y2, m2, r2) + ln.backward(x, w, m2, r2, dy, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(ref, got):
        assert torch.equal(p, q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y3, m3, r3 = ln.forward(x, w, b)
        got = (y3, m3, r3) + ln.backward(x, w, m3, r3, dy)
    for t in got:
        t.zero_()
    g.replay()
    for p, q in zip(ref, got):
        assert torch.equal(p, q)


def test_a_wait_that_ran_out_is_raised_by_check(M):
    """The status that a timed-out wait leaves in the unit's workspace (here from the library's own diagnostic wait)."""
    from top_softmax_router_gb300._lib import MoeError
    ln = M.LayerNorm(M.LayerNormConfig(N=4, H=32))
    ln.check()
    M.diag_wait_timeout(1_000_000, ln.ws)
    with pytest.raises(MoeError) as e:
        ln.check()
    assert e.value.code == -5
    ln.check()


@pytest.mark.parametrize("t,pt,n,h", [("bf16", "fp32", 6000, 1032), ("fp32", "fp32", 6000, 1024), ("bf16", "bf16", 3000, 7168),
                                      ("fp16", "fp16", 2500, 4096), ("fp32", "fp32", 1300, 7680), ("bf16", "bf16", 1100, 14336),
                                      ("fp32", "fp32", 2500, 1001), ("bf16", "bf16", 1300, 8200), ("fp32", "fp32", 700, 8192),
                                      ("bf16", "fp32", 500, 16384), ("bf16", "fp32", 700, 4101), ("fp16", "fp16", 2600, 300),
                                      ("bf16", "bf16", 600, 2051), ("bf16", "fp32", 3000, 1000)])
def test_many_rows_of_each_form(M, t, pt, n, h):
    """Every form of the backward with more rows a block than it holds at a time (the ring: than it has places)."""
    a = inputs(n, h, t, pt, seed=n + h)
    unit = M.LayerNorm(M.LayerNormConfig(N=n, H=h))
    first = check(M, *a, unit=unit)
    again = check(M, *a, unit=unit)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
