"""The distillation head on the GPU against the float64 oracle.

Tolerances (u = 2^-24; a rounding to bf16 is off by at most 2^-8 of the value):
  logits   fp32 sums of H products: at most H u sum|x w| / T =: dz (the tensor cores may truncate: twice that)
  lse      dz + (2^-22 of each exponential, 40 u of the sum) + 4 u |lse|
  loss     T^2 (2 dz + the lse's error + 64 u (|z| + |lse| + sum |q log q|)) at the row's largest |z|
  d        one bf16 rounding (2^-8) of each d, and its error exp(..) (dz + lse error + 2^-22)
  dX, dW   sums of d w and d x: 2^-8 + 4 dz of sum|d||w| worst case; roundings of d are independent, so the bound is
           6 sqrt(sum (2^-8 d w)^2) + (4 dz + 64 u) sum|d w| + half a step of the output
"""
import numpy as np
import pytest
import torch

from gpu_util import lib_api, need_gpu
from oracle import layer_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def M():
    need_gpu()
    return lib_api()


def make(N, H, V, K, seed=0, std=2.0):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(N, H, generator=g).bfloat16()
    W = (torch.randn(V, H, generator=g) * std / H ** 0.5).bfloat16()
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]) if K <= V and N else \
        torch.randint(0, V, (N, K), generator=g)
    t = torch.randn(N, K, generator=g) * 2
    dloss = torch.randn(N, generator=g) / max(N, 1)
    return X, W, ids.int(), t, dloss


def f64(t):
    return t.double().cpu().numpy()


def run(M, X, W, ids, t, dloss, P=1, T=1.0, unit=None, dt=torch.bfloat16):
    N, H = X.shape
    kd = unit or M.VocabDistill(M.DistillConfig(N=N, H=H, V=W.shape[0], K=ids.shape[1], P=P, temperature=T))
    X, W, ids, t, dloss = (v.cuda() for v in (X, W, ids, t, dloss))
    loss, lse, mean = kd.forward(X, W, ids, t)
    dX, dW = kd.backward(X, W, ids, t, lse, dloss, dW_dtype=dt)
    kd.check()
    return loss, lse, mean, dX, dW


def compare(out, X, W, ids, t, dloss, T):
    loss, lse, mean, dX, dW = out
    x, w, i, tl, g = f64(X), f64(W), ids.numpy(), f64(t), f64(dloss)
    N, H = x.shape
    V = w.shape[0]
    rl, rs, rdX, rdW = R.distill(x, w, i, tl, T, g)
    q, ent = R.teacher(i, tl, V, T)
    z = np.abs(x @ w.T).max(axis=1) / T
    dz = 2 * H * U * (np.abs(x) @ np.abs(w).T).max(axis=1) / T
    dl = dz + 2.0 ** -22 + 40 * U + 4 * U * np.abs(rs)
    assert np.all(np.abs(f64(lse) - rs) <= dl)
    bound = T * T * (2 * dz + dl + 64 * U * (z + np.abs(rs) + np.abs(ent)))
    assert np.all(np.abs(f64(loss) - rl) <= bound)
    assert abs(f64(mean)[0] - rl.mean()) <= bound.mean() + 64 * U * np.abs(rl).mean()
    p = np.exp(x @ w.T / T - rs[:, None]) * q.sum(axis=1, keepdims=True)
    c = (T * np.abs(g))[:, None]
    d, mass = np.abs(p - q) * c, (p + q) * c
    err = mass * (4 * dz + 4 * dl + 64 * U)[:, None]
    r = 2.0 ** -8
    aw, ax = np.abs(w), np.abs(x)
    bX = 6 * r * np.sqrt((d ** 2) @ (aw ** 2)) + err @ aw + 64 * U * (mass @ aw) + r * np.abs(rdX) + 1e-30
    assert np.all(np.abs(f64(dX) - rdX) <= bX)
    bW = 6 * r * np.sqrt((d ** 2).T @ (ax ** 2)) + err.T @ ax + 64 * U * (mass.T @ ax) + 1e-30
    bW += r * np.abs(rdW) if dW.dtype == torch.bfloat16 else 0
    assert np.all(np.abs(f64(dW) - rdW) <= bW)


@pytest.mark.parametrize("N,H,V,K,P,T", [
    (1, 64, 1, 1, 1, 1.0), (1, 64, 300, 5, 1, 2.0), (2, 64, 257, 3, 2, 1.0), (31, 128, 255, 8, 1, 4.0),
    (33, 64, 513, 64, 3, 1.0), (128, 192, 1000, 10, 1, 2.0), (129, 64, 256, 256, 1, 1.0), (257, 320, 777, 17, 2, 0.5),
    (300, 128, 1000, 8, 3, 1.0), (511, 64, 2049, 33, 8, 2.0), (600, 512, 1300, 100, 1, 8.0), (65, 1024, 3001, 4, 4, 1.0)])
def test_against_the_oracle(M, N, H, V, K, P, T):
    a = make(N, H, V, K, seed=N + V)
    compare(run(M, *a, P=P, T=T), *a, T)


@pytest.mark.parametrize("N,H,V,K,P,T", [(511, 64, 9001, 8, 8, 1.0), (1030, 128, 4500, 33, 3, 2.0), (2100, 64, 2049, 5, 2, 1.0),
                                         (300, 320, 20000, 16, 4, 4.0)])
def test_several_strips(M, N, H, V, K, P, T):
    """d of more than 8 MB: P strips, the last one narrower; the strip count changes dX's rounding alone."""
    a = make(N, H, V, K, seed=P)
    out, one = run(M, *a, P=P, T=T), run(M, *a, P=1, T=T)
    compare(out, *a, T)
    assert all(torch.equal(out[i], one[i]) for i in (0, 1, 2, 4))
    unit = M.VocabDistill(M.DistillConfig(N=N, H=H, V=V, K=K, P=P, temperature=T))
    b = make(7, H, V, K, seed=P + 1)          # fewer tokens in the same workspace: one strip
    compare(run(M, *b, T=T, unit=unit), *b, T)
    assert all(torch.equal(p, q) for p, q in zip(out, run(M, *a, T=T, unit=unit)))


@pytest.mark.parametrize("N,H,V,P", [(40, 64, 6000, 1), (300, 128, 9000, 2), (256, 320, 5121, 1), (1, 64, 20000, 3)])
def test_shares_of_a_long_strip(M, N, H, V, P):
    """Few tiles of dX and many classes: K is split, the last share and strip are short or empty."""
    a = make(N, H, V, 5, seed=V)
    out = run(M, *a, P=P)
    compare(out, *a, 1.0)
    assert all(torch.equal(p, q) for p, q in zip(out, run(M, *a, P=P)))


def test_fp32_weight_gradient(M):
    a = make(200, 128, 600, 8)
    out = run(M, *a, P=2, dt=torch.float32)
    assert out[4].dtype == torch.float32
    compare(out, *a, 1.0)


def test_outputs_on_16_bytes(M):
    """Every pointer 16 bytes off a 32-byte boundary, the workspace's too."""
    from top_softmax_router_gb300 import _lib
    X, W, ids, t, g = (v.cuda() for v in make(70, 64, 300, 4, seed=12))

    def off(n, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        flat = torch.zeros(n * size + 64, dtype=torch.uint8, device="cuda")
        return flat[16:16 + n * size].view(dtype)

    X2, W2 = off(X.numel(), X.dtype).view_as(X).copy_(X), off(W.numel(), W.dtype).view_as(W).copy_(W)
    cfg = M.DistillConfig(N=70, H=64, V=300, K=4, P=2)
    ref = M.VocabDistill(cfg)
    loss, lse, _ = ref.forward(X, W, ids, t)
    for dt in (torch.bfloat16, torch.float32):
        want = ref.backward(X, W, ids, t, lse, g, dW_dtype=dt)
        kd = M.VocabDistill(cfg)
        kd.ws = off(kd.ws.numel() + 256, torch.uint8)
        got = kd.forward(X2, W2, ids, t)
        assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
        dX, dW = off(X.numel(), X.dtype), off(W.numel(), dt)
        _lib.check(_lib.load().moe_distill_backward(
            kd._c(70), X2.data_ptr(), W2.data_ptr(), ids.data_ptr(), t.data_ptr(), lse.data_ptr(), g.data_ptr(),
            dX.data_ptr(), dW.data_ptr(), 1 if dt == torch.bfloat16 else 0, kd.ws.data_ptr(), kd.ws.numel(),
            torch.cuda.current_stream().cuda_stream), "moe_distill_backward")
        assert torch.equal(dX.view_as(want[0]), want[0]) and torch.equal(dW.view_as(want[1]), want[1])


def test_rows_with_fewer_entries_or_none(M):
    X, W, ids, t, g = make(140, 128, 700, 12, seed=3)
    ids[0] = -1
    ids[1, 1:] = -1
    t[2] = -float("inf")
    t[3, ::2] = -float("inf")
    ids[64:96] = -1                     # a whole bucket group without entries
    ids[5, 3:7] = -1
    t[5, 4] = float("nan")              # in a place that is no entry
    t[7] = torch.finfo(torch.bfloat16).min
    t[8, 1:] = torch.finfo(torch.float32).min
    out = run(M, X, W, ids, t, g, P=2, T=2.0)
    tt = t.clone()
    tt[5, 4] = 0.0
    compare(out, X, W, ids, tt, g, 2.0)
    for r in [0, 2] + list(range(64, 96)):
        assert out[0][r] == 0 and not out[3][r].any()


def test_a_class_may_occur_twice(M):
    X, W, ids, t, g = make(70, 64, 400, 9, seed=4)
    ids[:, 4] = ids[:, 0]
    ids[:, 8] = ids[:, 0]
    ids[3] = ids[3, 0]
    compare(run(M, X, W, ids, t, g), X, W, ids, t, g, 1.0)


def test_entries_on_tile_and_strip_edges(M):
    X, W, ids, t, g = make(260, 64, 1025, 6, seed=5)
    ids[:] = torch.tensor([0, 127, 128, 255, 256, 1024], dtype=torch.int32)
    ids[::2] = torch.tensor([511, 512, 767, 768, 1023, 383], dtype=torch.int32)
    compare(run(M, X, W, ids, t, g, P=4), X, W, ids, t, g, 1.0)


def test_strips_change_little_and_repeats_nothing(M):
    a = make(300, 256, 2000, 16, seed=6)
    one, four, again = run(M, *a, P=1), run(M, *a, P=4), run(M, *a, P=4)
    for i in (0, 1, 2, 4):
        assert torch.equal(one[i], four[i])
    compare(four, *a, 1.0)
    assert all(torch.equal(p, q) for p, q in zip(four, again))


def test_a_sure_student_and_teacher(M):
    """Logits of hundreds: exponentials of the far classes vanish, nothing overflows; teacher = student at zero loss."""
    X, W, ids, t, g = make(64, 128, 500, 8, seed=7, std=60.0)
    compare(run(M, X, W, ids, t, g), X, W, ids, t, g, 1.0)
    X, W, ids, _, g = make(40, 64, 30, 30, seed=8)
    z = (X.double() @ W.double().T).gather(1, ids.long()).float()
    out = run(M, X, W, ids, z, g)
    assert out[0].abs().max() < 1e-5
    compare(out, X, W, ids, z, g, 1.0)


def test_gradient_against_differences(M):
    """A step of one bf16 unit in X and W (both directions) against dX and dW: the difference quotient's rounding is
    1e-5 of a loss of order one over a step of 2^-4, the gradient's own bf16 error 2^-7 of its scale."""
    X, W, ids, t, g = make(3, 64, 40, 4, seed=9)
    kd = M.VocabDistill(M.DistillConfig(N=3, H=64, V=40, K=4, temperature=2.0))
    ids, t, g = ids.cuda(), t.cuda(), torch.ones(3, device="cuda")
    X, W = (X * 4).round().div(4).cuda(), (W * 8).round().div(8).cuda()   # values to which the step adds exactly
    lse = kd.forward(X, W, ids, t)[1]
    dX, dW = kd.backward(X, W, ids, t, lse, g)
    h = 2.0 ** -4
    for which, d in ((0, dX), (1, dW)):
        scale = d.float().abs().max().item()
        for i in range(0, d.numel(), 37):
            vals = []
            for sign in (h, -h):
                a = [X.clone(), W.clone()]
                a[which].view(-1)[i] += sign
                vals.append(kd.forward(a[0], a[1], ids, t)[0].double().sum().item())
            assert abs((vals[0] - vals[1]) / (2 * h) - d.view(-1)[i].item()) <= 2e-2 * scale + 2e-3


def test_bad_classes_are_reported_and_passed_over(M):
    from top_softmax_router_gb300._lib import MoeError
    X, W, ids, t, g = make(50, 64, 300, 4, seed=10)
    bad = ids.clone()
    bad[3, 1], bad[4, 0] = 300, -2
    kd = M.VocabDistill(M.DistillConfig(N=50, H=64, V=300, K=4))
    loss, lse, _ = kd.forward(X.cuda(), W.cuda(), bad.cuda(), t.cuda())
    with pytest.raises(MoeError) as e:
        kd.check()
    assert e.value.code == -6
    ref = ids.clone()
    ref[3, 1] = ref[4, 0] = -1
    want = kd.forward(X.cuda(), W.cuda(), ref.cuda(), t.cuda())
    kd.check()
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])


def test_no_tokens_and_fewer_tokens(M):
    kd = M.VocabDistill(M.DistillConfig(N=400, H=64, V=500, K=6, P=2))
    a = make(0, 64, 500, 6)
    loss, lse, mean, dX, dW = run(M, *a, unit=kd)
    assert loss.shape == (0,) and mean.item() == 0 and dX.shape == (0, 64) and not dW.any()
    for N in (400, 1, 37):
        a = make(N, 64, 500, 6, seed=N)
        compare(run(M, *a, unit=kd), *a, 1.0)


def test_other_stream_and_graph(M):
    X, W, ids, t, g = (v.cuda() for v in make(300, 128, 900, 8, seed=11))
    kd = M.VocabDistill(M.DistillConfig(N=300, H=128, V=900, K=8, P=2))

    def step(stream=None):
        loss, lse, mean = kd.forward(X, W, ids, t, stream=stream)
        return (loss, lse, mean) + kd.backward(X, W, ids, t, lse, g, stream=stream)

    ref = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    kd.check()


@pytest.mark.parametrize("T", [1.0, 0.5, 0.25])
def test_lowest_teacher_logits_at_low_temperatures(M, T):
    """Entries so far below the row's largest that their distance, or that over T, is beyond fp32: their q is 0."""
    X, W, ids, t, g = make(70, 64, 400, 9, seed=13)
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    t[::2, 3:] = low
    t[5] = low
    t[7, 1] = torch.finfo(torch.bfloat16).min
    t[9, 0], t[9, 4] = high, low
    out = run(M, X, W, ids, t, g, T=T)
    assert all(torch.isfinite(v).all() for v in out)
    compare(out, X, W, ids, t, g, T)


@pytest.mark.parametrize("first", [0.0, 1.0])
def test_one_gradient_for_all_rows_but_a_masked_first(M, first):
    """One gradient g for all rows, the first of which may be masked.  p is 2^-8 within 10 % (logits of 0.02), so that p - 1
    is a bf16 value within 4e-4, and g (1 - 2^-8) lies 0.95 of half a step from the next one: rounded as it is, every
    d would be 3.7e-3 off the same way.  Relative to g, d is off by 4e-4 at its entry, and by 2^-8 of p elsewhere, whose
    share of dW is sqrt(512) 2^-8 against 1 or more of the entries: 4e-4 + 0.09 x 2^-8, 8e-4."""
    X, W, ids, t, _ = make(512, 64, 256, 1, seed=14, std=0.02)
    g = torch.full((512,), (1 + 0.95 * 2.0 ** -8) / (1 - 2.0 ** -8) * 2.0 ** -9)
    g[0] *= first
    dW = run(M, X, W, ids, t, g, dt=torch.float32)[4]
    ref = R.distill(f64(X), f64(W), ids.numpy(), f64(t), 1.0, f64(g))[3]
    assert np.linalg.norm(f64(dW) - ref) <= 8e-4 * np.linalg.norm(ref)


@pytest.mark.parametrize("N,H,V,K,P,T", [(70, 1088, 600, 5, 1, 1.0), (33, 2048, 513, 8, 1, 2.0), (130, 2112, 1000, 3, 2, 1.0),
                                         (40, 4096, 700, 16, 1, 4.0), (260, 2112, 10300, 4, 1, 1.0), (520, 1152, 9001, 6, 1, 2.0)])
def test_logits_of_several_accumulators(M, N, H, V, K, P, T):
    """More than 1024 products a logit: two to four accumulators a tile, the last one short, an odd number of them
    carried from tile to tile where there are more tiles than clusters (the last two cases: 82 and 108 tiles)."""
    a = make(N, H, V, K, seed=H + V)
    out = run(M, *a, P=P, T=T)
    compare(out, *a, T)
    assert all(torch.equal(p, q) for p, q in zip(out, run(M, *a, P=P, T=T)))
