"""RMS norm on the GPU against the float64 oracle, forward and backward.

Tolerances, from the arithmetic before any run (u = 2^-24, one fp32 rounding):
  rstd   a thread sums at most 32 squares, then 5 + 16 additions of a tree, the product, the square root and the division,
         half of it by the square root: relative 32 u
  y      h rstd weight: 36 u |y|, and half a step of y's type
  codes  of y before it is rounded: those of the oracle, unless y lies within 36 u of a border between two codes (or its
         block's largest value of a border between two scales): the restored value is then one step off.  Held to: off by
         at most half a step and 36 u of the value
  dx     rstd (t - xh c) + dh: 64 u rstd (|t| + |xh| mean|t xh|) + 2 u |dh| + half a step
  dweight  fp32 sums over n rows in at most 1216 blocks: the walk of independent roundings, factor 8:
         8 sqrt(n + 90) u sqrt(sum terms^2) + 48 u sum|terms| / sqrt(n) (each term's own error)
"""
import numpy as np
import pytest
import torch

from gpu_util import lib_api, need_gpu
from oracle import blocks8_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def M():
    need_gpu()
    return lib_api()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inputs(n, h, t, pt, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, r = (torch.randn(n, h, generator=g) * 2).to(TYPES[t]), torch.randn(n, h, generator=g).to(TYPES[t])
    w = (torch.randn(h, generator=g) * 0.3 + 1).to(TYPES[pt])
    dy, dh = torch.randn(n, h, generator=g).to(TYPES[t]), torch.randn(n, h, generator=g).to(TYPES[t])
    return x, r, w, dy, dh


def check(M, x, r, w, dy, dh, eps=1e-6, unit=None, place=lambda t: t.cuda()):
    n, H = x.shape
    put = lambda t: None if t is None else place(t)   # noqa: E731
    rms = unit or M.RMSNorm(M.RMSNormConfig(N=n, H=H, eps=eps))
    wd = None if w is None else w.cuda()
    y, h, rstd, codes, scales = rms.forward(put(x), wd, put(r), want_codes=True)
    dx, dw = rms.backward(put(h) if r is None else h, wd, rstd, put(dy), put(dh))
    want_h = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert torch.equal(h.cpu(), want_h)
    Hh = host(want_h)
    W = np.ones(H) if w is None else host(w)
    ry, rr = R.rms_forward(Hh, W, eps)
    half = torch.finfo(x.dtype).eps / 2
    tiny = 1e-30 if x.dtype != torch.float16 else 2.0 ** -25
    assert np.all(np.abs(host(rstd) - rr) <= 32 * U * rr)
    assert np.all(np.abs(host(y) - ry) <= (36 * U + half) * np.abs(ry) + tiny)
    v, s = R.unpack(host(codes), host(scales)), np.repeat(host(scales), 128, axis=1)[:, :H]
    assert np.all(np.abs(v - ry) <= np.maximum(2.0 ** -4 * np.abs(ry), 2.0 ** -10 * s) + 36 * U * np.abs(ry))
    rs = R.pack(ry)[1]
    assert np.all((host(scales) == rs) | (host(scales) == 2 * rs) | (2 * host(scales) == rs))
    assert np.mean(host(scales) != rs) <= 0.01 + 1 / rs.size
    rdx, rdw = R.rms_backward(Hh, W, host(dy), None if dh is None else host(dh), eps)
    xh, t = np.abs(Hh * rr[:, None]), np.abs(host(dy) * W)
    bound = 64 * U * rr[:, None] * (t + xh * (t * xh).mean(axis=1, keepdims=True)) + half * np.abs(rdx) + tiny
    if dh is not None:
        bound = bound + 2 * U * np.abs(host(dh))
    assert np.all(np.abs(host(dx) - rdx) <= bound)
    terms = host(dy) * xh
    walk = 8 * np.sqrt(n + 90) * U
    assert dw.dtype == torch.float32
    assert np.all(np.abs(host(dw) - rdw) <= walk * np.sqrt((terms ** 2).sum(axis=0)) + 48 * U * np.abs(terms).sum(axis=0) / np.sqrt(n) + 1e-30)
    return y, h, rstd, codes.view(torch.uint8), scales.view(torch.uint8), dx, dw


@pytest.mark.parametrize("t,pt", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")])
@pytest.mark.parametrize("n,h", [(1, 1), (1, 8), (3, 7), (5, 64), (130, 256), (33, 512), (17, 1000), (9, 1001), (300, 1024), (41, 2048),
                                 (7, 4100), (11, 7168), (3, 8200), (2, 16384), (2, 16383)])
def test_against_the_oracle(M, t, pt, n, h):
    check(M, *inputs(n, h, t, pt, seed=n * h))


@pytest.mark.parametrize("n", [1, 2, 607, 1217, 9800])
@pytest.mark.parametrize("h", [72, 384])
def test_many_rows(M, n, h):
    check(M, *inputs(n, h, "bf16", "fp32", seed=n))


def test_without_residual_weight_or_further_gradient(M):
    x, r, w, dy, dh = inputs(20, 320, "bf16", "bf16")
    check(M, x, None, w, dy, None)
    check(M, x, r, None, dy, dh)
    check(M, x, None, None, dy, dh)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,first", [(8, 0), (3, 0), (16, 8), (5, 3)])
def test_strided_rows(M, t, pad, first):
    def place(v):
        wide = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=v.dtype, device="cuda")
        view = wide[:, first:first + v.shape[1]]
        view.copy_(v)
        return view
    x, r, w, dy, dh = inputs(19, 264, t, "fp32", seed=3)
    check(M, x, r, w, dy, dh, place=place)
    check(M, x, None, w, dy, dh, place=place)


def test_codes_are_those_of_the_norms_output(M):
    """In fp32 the output is what is packed: Checkpoint8.pack of it gives the same codes."""
    x, r, w, _, _ = inputs(50, 1001, "fp32", "fp32", seed=5)
    rms = M.RMSNorm(M.RMSNormConfig(N=50, H=1001))
    y, _, _, c, s = rms.forward(x.cuda(), w.cuda(), r.cuda(), want_codes=True)
    c2, s2 = M.Checkpoint8(M.Checkpoint8Config(N=50, H=1001)).pack(y)
    assert torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s.view(torch.uint8), s2.view(torch.uint8))


def test_a_unit_serves_fewer_rows_and_repeats_its_bits(M):
    rms = M.RMSNorm(M.RMSNormConfig(N=900, H=520))
    for n in (900, 1, 77):
        a = inputs(n, 520, "bf16", "fp32", seed=n)
        for p, q in zip(check(M, *a, unit=rms), check(M, *a, unit=rms)):
            assert torch.equal(p, q)


def test_no_rows_and_partial_wants(M):
    rms = M.RMSNorm(M.RMSNormConfig(N=4, H=32))
    none = torch.empty(0, 32, device="cuda")
    y, h, rstd, c, s = rms.forward(none, None, none, want_codes=True)
    assert y.shape == h.shape == c.shape == (0, 32) and s.shape == (0, 1) and rstd.shape == (0,)
    dx, dw = rms.backward(none, None, rstd, none)
    assert dx.shape == (0, 32) and torch.equal(dw, torch.zeros(32, device="cuda"))
    x = torch.randn(4, 32, device="cuda")
    y, h, rstd, c, s = rms.forward(x, want_y=False)
    assert y is None and c is None and s is None and h is x
    whole = rms.backward(x, None, rstd, x)
    assert rms.backward(x, None, rstd, x, want_dx=False)[0] is None
    assert torch.equal(rms.backward(x, None, rstd, x, want_dx=False)[1], whole[1])
    assert torch.equal(rms.backward(x, None, rstd, x, want_dweight=False)[0], whole[0])


def test_rows_that_hold_no_numbers(M):
    """NaN and infinity stay in their rows; a row of zeros has y = 0 and a scale of 1."""
    x, r, w, _, _ = inputs(6, 300, "bf16", "fp32")
    rms = M.RMSNorm(M.RMSNormConfig(N=6, H=300))
    clean = rms.forward(x.cuda(), w.cuda(), r.cuda(), want_codes=True)
    x[1, 7], x[3, 200] = float("nan"), float("inf")
    x[5], r[5] = 0, 0
    got = rms.forward(x.cuda(), w.cuda(), r.cuda(), want_codes=True)
    keep = torch.tensor([0, 2, 4], device="cuda")
    for p, q in zip(clean, got):
        p, q = (t.view(torch.uint8) if t.element_size() == 1 else t for t in (p, q))
        assert torch.equal(p[keep], q[keep])
    y, _, _, c, s = got
    assert torch.all(torch.isnan(y[1])) and torch.isnan(y[3, 200])
    assert torch.all(y[5] == 0) and torch.all(c[5].float() == 0) and torch.all(s[5].float() == 1)
    assert torch.all(torch.isnan(c[1].float()))


def test_gradients_against_differences(M):
    """Central differences of the kernel's own fp32 forward, summed in fp64: y is smooth on the step 2^-8, the difference's
    own error about 2^-16 of the third derivative and 2^-24 / 2^-8 of |y| a term."""
    x, _, w, dy, _ = inputs(3, 40, "fp32", "fp32", seed=8)
    rms = M.RMSNorm(M.RMSNormConfig(N=3, H=40))
    _, _, rstd, _, _ = rms.forward(x.cuda(), w.cuda())
    dx, _ = rms.backward(x.cuda(), w.cuda(), rstd, dy.cuda())
    step = 2.0 ** -8
    for i in range(3):
        for j in range(0, 40, 7):
            d = torch.zeros_like(x)
            d[i, j] = step
            up, down = (host(rms.forward((x + k * d).cuda(), w.cuda())[0]) for k in (1, -1))
            assert abs(((up - down) * host(dy)).sum() / (2 * step) - host(dx)[i, j]) < 40 * 2.0 ** -15 + 1e-3


def test_rows_past_2_to_31_elements(M):
    """The last rows of an odd and of an aligned width, forward and backward."""
    for h in (7168, 7169):
        n = 300_000
        last = inputs(3, h, "bf16", "fp32", seed=h)
        x, r, dy, dh = (torch.zeros(n, h, dtype=torch.bfloat16, device="cuda") for _ in range(4))
        for t, v in zip((x, r, dy, dh), (last[0], last[1], last[3], last[4])):
            t[-3:] = v.cuda()
        w = last[2].cuda()
        rms = M.RMSNorm(M.RMSNormConfig(N=n, H=h))
        y, kept, rstd, codes, scales = rms.forward(x, w, r, want_codes=True)
        del x, r
        dx, dw = rms.backward(kept, w, rstd, dy, dh)
        few = M.RMSNorm(M.RMSNormConfig(N=3, H=h))
        want = few.forward(last[0].cuda(), w, last[1].cuda(), want_codes=True)
        for p, q in zip((y, kept, rstd, codes, scales), want):
            p, q = (t.view(torch.uint8) if t.element_size() == 1 else t for t in (p, q))
            assert torch.equal(p[-3:], q)
        want_dx, want_dw = few.backward(want[1], w, want[2], last[3].cuda(), last[4].cuda())
        assert torch.equal(dx[-3:], want_dx) and not dx[:-3].any()
        # three terms, each rounded once as a product and at most twice in a sum, in both orders
        terms = np.abs(host(last[3]) * host(want[1]) * host(want[2])[:, None]).sum(axis=0)
        assert np.all(np.abs(host(dw) - host(want_dw)) <= 6 * U * terms)


@pytest.mark.parametrize("t", list(TYPES))
def test_scales_are_the_oracles_but_at_borders(M, t):
    """A block's scale is the definition's for a largest value that is 36 u of itself off, which moves it only where that
    value lies at a border between two scales."""
    x, r, w, _, _ = inputs(700, 1024, t, "fp32", seed=11)
    _, h, rstd, _, scales = M.RMSNorm(M.RMSNormConfig(N=700, H=1024)).forward(x.cuda(), w.cuda(), r.cuda(), want_codes=True)
    ry, _ = R.rms_forward(host(h), host(w), 1e-6)
    top = np.abs(ry.reshape(700, 8, 128)).max(axis=2)
    low, high = R.scale_of(top * (1 - 36 * U)), R.scale_of(top * (1 + 36 * U))
    got = host(scales)
    assert np.all((got == low) | (got == high)) and np.mean(low != high) < 1e-3
