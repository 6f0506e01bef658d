"""Expert routing with scores on the GPU against the float64 oracle: indices and counts equal, weights and
gradients within their rounding.

Tolerances (u = 2^-24): a score is at most 4 u (sigmoid) or 42 u (softmax, see the kernel) off relative to itself
or the row's largest; a share of k <= 32 of them adds 34 u; gradients are three such factors and a sum of k terms
of size |dw|: 160 u scale max|dw|, and half a step of the logits' type.  Below 2^-126 fp32's steps are 2^-149
whatever the value: four roundings there (expf, share, scale, store) are 2^-146 with a margin of two.
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


def check(M, logits, bias, k, dw=None, unit=None, view=None, **kw):
    n, E = logits.shape
    r = unit or M.ScoreRouter(M.ScoreRouterConfig(N=n, E=E, k=k, **kw))
    l = logits.cuda() if view is None else view(logits)
    b = None if bias is None else bias.cuda()
    idx, w, counts = r.forward(l, b)
    opt = dict(groups=1, topk_groups=1, score="softmax", renormalize=True, scale=1.0, group_top=2) | kw
    lf = logits.double().numpy()
    ri, rw, rc = R.route(lf, None if bias is None else bias.double().numpy(), k, opt["groups"], opt["topk_groups"],
                         opt["score"], opt["renormalize"], opt["scale"], opt["group_top"])
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.array_equal(counts.cpu().numpy(), rc)
    scale = abs(opt["scale"])
    assert np.all(np.abs(w.double().cpu().numpy() - rw) <= 80 * U * np.abs(rw) + scale * 2.0 ** -146 + (0 if opt["renormalize"] else 42 * U * scale))
    dw = torch.randn(n, k, generator=torch.Generator().manual_seed(7)) if dw is None else dw
    d = r.backward(l, idx, dw.cuda())
    rd = R.route_backward(lf, ri, dw.numpy(), opt["score"], opt["renormalize"], opt["scale"])
    assert d.dtype == logits.dtype and d.is_contiguous()
    half = torch.finfo(logits.dtype).eps / 2
    tiny = 2.0 ** -25 if logits.dtype == torch.float16 else 1e-38
    worst = 160 * U * scale * np.abs(dw.numpy()).max(axis=1, initial=0)[:, None]
    assert np.all(np.abs(d.double().cpu().numpy() - rd) <= worst + half * np.abs(rd) + tiny)
    r.check()
    return idx, w, counts, d


def logits_of(n, E, t="fp32", seed=0, std=1.5):
    return (torch.randn(n, E, generator=torch.Generator().manual_seed(seed)) * std).to(TYPES[t])


def bias_of(E, seed=1, std=0.1):
    return torch.randn(E, generator=torch.Generator().manual_seed(seed)) * std


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("n,E,k,groups,topk_groups,t", [
    (1, 1, 1, 1, 1, "fp32"), (1, 5, 5, 1, 1, "bf16"), (7, 8, 2, 1, 1, "fp32"), (65, 33, 4, 3, 2, "fp16"),
    (200, 64, 8, 8, 4, "fp32"), (130, 60, 6, 4, 3, "bf16"), (50, 384, 8, 8, 4, "fp32"), (33, 896, 16, 1, 1, "fp32"),
    (20, 1024, 32, 32, 9, "fp32"), (40, 160, 6, 20, 5, "fp32"), (64, 32, 3, 32, 4, "fp32"), (9, 510, 7, 2, 1, "fp32")])
def test_against_the_oracle(M, score, renormalize, biased, n, E, k, groups, topk_groups, t):
    check(M, logits_of(n, E, t, seed=n + E), bias_of(E) if biased else None, k, groups=groups, topk_groups=topk_groups,
          score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [True, False])
def test_group_of_its_largest_value(M, score, biased):
    check(M, logits_of(100, 64), bias_of(64) if biased else None, 4, groups=8, topk_groups=3, score=score, group_top=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 8])
def test_many_rows_with_neighbouring_scores(M, score, groups):
    """20,000 rows of 64 scores squeezed together: many pairs closer than fp32 resolves, each to be ordered as in
    exact arithmetic."""
    l = (torch.randn(20000, 64, generator=torch.Generator().manual_seed(3)) * 2e-5).float()
    check(M, l, bias_of(64, std=2e-6), 8, groups=groups, topk_groups=max(1, groups // 2), score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_ties_go_to_the_lower_index(M, score, groups):
    l = torch.randint(-2, 3, (300, 64), generator=torch.Generator().manual_seed(5)).float()
    l[5] = 0.0
    l[6, ::2] = -0.0
    kw = dict(groups=groups, topk_groups=max(1, groups // 2), score=score)
    check(M, l, None, 8, **kw)
    check(M, l, torch.zeros(64), 8, **kw)
    check(M, l.bfloat16(), torch.full((64,), 0.25), 8, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_experts_and_rows(M, score, renormalize, biased, groups):
    """-inf logits: fewer than k experts left, none left; -inf in bf16's lowest value too."""
    l = logits_of(12, 32, seed=8)
    l[0] = -float("inf")
    l[1, 3:] = -float("inf")
    l[2, :30] = -float("inf")
    l[3, 8:16] = -float("inf")
    l[4] = torch.finfo(torch.bfloat16).min
    l[5, ::2] = torch.finfo(torch.bfloat16).min
    out = check(M, l, bias_of(32) if biased else None, 4, groups=groups, topk_groups=max(1, groups // 2), score=score,
                renormalize=renormalize)
    assert not out[1][0].any() and not out[3][0].any()


def test_a_bias_of_minus_infinity_closes_an_expert(M):
    b = bias_of(16)
    b[3] = b[7] = -float("inf")
    idx, _, counts, _ = check(M, logits_of(200, 16), b, 5, score="sigmoid")
    assert counts[3] == 0 and counts[7] == 0


def test_nan_ranks_last_and_stays_in_its_row(M):
    l = logits_of(6, 16, seed=2)
    ref = M.ScoreRouter(M.ScoreRouterConfig(N=6, E=16, k=4, score="sigmoid")).forward(l.cuda(), bias_of(16).cuda())
    bad = l.clone()
    bad[2, 5] = float("nan")
    for score in ("sigmoid", "softmax"):
        r = M.ScoreRouter(M.ScoreRouterConfig(N=6, E=16, k=4, score=score))
        for b in (None, bias_of(16).cuda()):
            idx, w, _ = r.forward(bad.cuda(), b)
            row = idx[2].tolist()
            assert len(set(row)) == 4 and all(0 <= e < 16 for e in row)
            if score == "sigmoid":
                assert 5 not in row and torch.isfinite(w).all()
            assert torch.isfinite(w[[0, 1, 3, 4, 5]]).all()
            if score == "sigmoid" and b is not None:
                assert torch.equal(idx[[0, 1, 3, 4, 5]], ref[0][[0, 1, 3, 4, 5]])


def test_strided_logits_and_fewer_rows(M):
    def view(v):
        wide = torch.full((v.shape[0], v.shape[1] + 5), float("nan"), dtype=v.dtype, device="cuda")
        wide[:, 2:2 + v.shape[1]] = v.cuda()
        return wide[:, 2:2 + v.shape[1]]
    kw = dict(groups=4, topk_groups=2, score="sigmoid")
    unit = M.ScoreRouter(M.ScoreRouterConfig(N=3000, E=40, k=6, **kw))
    for n in (3000, 1, 0, 255):
        check(M, logits_of(n, 40, "bf16", seed=n), bias_of(40), 6, unit=unit, view=view, **kw)


def test_large_logits(M):
    l = logits_of(100, 48, std=40.0)
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            check(M, l, None, 4, score=score, renormalize=renormalize)


def test_gradient_against_differences(M):
    """Central differences of sum(weights dw) at a step of 2^-7 and fp32 outputs: 2e-3 of the gradient's scale (a step
    that changes the choice is passed over)."""
    dw = torch.randn(4, 3, generator=torch.Generator().manual_seed(1)).cuda()
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            r = M.ScoreRouter(M.ScoreRouterConfig(N=4, E=12, k=3, score=score, renormalize=renormalize, scale=1.5))
            l, b = logits_of(4, 12, seed=6).cuda(), bias_of(12).cuda()
            idx = r.forward(l, b)[0]
            d = r.backward(l, idx, dw)
            h = 2.0 ** -7
            for i in range(48):
                e = torch.zeros(48, device="cuda")
                e[i] = h
                up, dn = r.forward(l + e.view(4, 12), b), r.forward(l - e.view(4, 12), b)
                if torch.equal(up[0], idx) and torch.equal(dn[0], idx):
                    diff = ((up[1].double() - dn[1].double()) * dw.double()).sum() / (2 * h)
                    assert abs(diff - d.view(-1)[i]) <= 2e-3 * max(1.0, d.abs().max().item())


def test_bad_indices_are_reported(M):
    from top_softmax_router_gb300._lib import MoeError
    r = M.ScoreRouter(M.ScoreRouterConfig(N=4, E=12, k=3))
    l = logits_of(4, 12).cuda()
    idx = r.forward(l)[0]
    dw = torch.ones(4, 3, device="cuda")
    ref = r.backward(l, idx, dw)
    bad = idx.clone()
    bad[1, 0], bad[2, 1] = 12, -1
    got = r.backward(l, bad, dw)
    with pytest.raises(MoeError) as e:
        r.check()
    assert e.value.code == -6 and torch.equal(got[[0, 3]], ref[[0, 3]])


def test_other_stream_and_graph(M):
    l, b = logits_of(5000, 64, "bf16").cuda(), bias_of(64).cuda()
    dw = torch.randn(5000, 6, device="cuda")
    r = M.ScoreRouter(M.ScoreRouterConfig(N=5000, E=64, k=6, groups=8, topk_groups=4, score="sigmoid"))
    ref = r.forward(l, b)
    ref += (r.backward(l, ref[0], dw),)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = r.forward(l, b, stream=s)
    got += (r.backward(l, got[0], dw, stream=s),)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = r.forward(l, b)
        got += (r.backward(l, got[0], dw),)
    for _ in range(2):
        g.replay()
    assert all(torch.equal(p, q) for p, q in zip(ref, got))


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("E,groups", [(24, 1), (64, 8)])
def test_sigmoid_logits_far_below_zero(M, renormalize, biased, E, groups):
    """Scores below fp32's range: renormalised weights are shares of exp(l) there, and the gradient is theirs."""
    l = logits_of(18, E, seed=11, std=3.0)
    l += torch.tensor([-20.0, -60, -85, -95, -105, -200, -600, -690, 0])[:, None].repeat(2, 1)
    l[9:, ::2] = -float("inf")                       # half the experts masked
    l[17] = -float("inf")
    l[17, [1, 5, 9]] = torch.tensor([-100.0, -101.5, 0.5])
    kw = dict(groups=groups, topk_groups=max(1, groups // 2), score="sigmoid", renormalize=renormalize, scale=2.5)
    _, w, _, _ = check(M, l, bias_of(E) if biased else None, 4, **kw)
    if renormalize and not biased:
        total = w[:17].double().sum(dim=1)
        assert (total - 2.5).abs().max() <= 2.5 * 40 * U


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 8), (40, 4), (256, 32)])
def test_group_scores_of_large_biases_that_cancel(M, score, E, groups):
    """The group's first expert has a bias of 1000, the others of -1000: a group's score is what is left of their sum."""
    b = torch.full((E,), -1000.0)
    b[::E // groups] = 1000.0
    l = logits_of(3000, E, seed=12, std=0.05)
    check(M, l, b, 3, groups=groups, topk_groups=groups // 2, score=score)
