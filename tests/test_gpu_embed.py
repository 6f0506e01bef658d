"""Token embedding and its gradient on the GPU against the float64 oracle.

Tolerances (u = 2^-24): the lookup is one fp32 product and one rounding to the table's type; a gradient row is an
fp32 sum of its run, at most 32 terms in a piece and then the pieces: u (32 + pieces) sum|terms| + 2 u for the
scale and the addition.
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


def make(n, v, h, t, seed=0, hot=0.0, id_type=torch.int64):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, v, (n,), generator=g)
    if hot:
        ids = torch.where(torch.rand(n, generator=g) < hot, torch.tensor(v // 2), ids)
    table = torch.randn(v, h, generator=g).to(TYPES[t])
    dy = torch.randn(n, h, generator=g).to(TYPES[t])
    return ids.to(id_type), table, dy


def check_grad(got, ids, dy, v, scale, padding=-1, into=None):
    i, d = ids.cpu().numpy(), dy.double().cpu().numpy()
    base = None if into is None else into.double().cpu().numpy()
    ref = R.embed_backward(i, d, v, scale, padding, base)
    mass = R.embed_backward(i, np.abs(d), v, abs(scale), padding)
    n = np.bincount(i[(i >= 0) & (i < v)], minlength=v)[:, None]
    bound = U * (np.minimum(n, 32) + n / 32 + 4) * mass + 2 * U * np.abs(ref)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= bound + (0 if base is None else 2 * U * np.abs(base)))


@pytest.mark.parametrize("t", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,v,h,scale,hot", [
    (1, 1, 1, 1.0, 0), (1, 7, 8, 2.5, 0), (5, 3, 40, 1.0, 0), (64, 10, 33, 0.5, 0), (65, 1, 64, 1.0, 0),
    (300, 1000, 128, 45.25, 0), (1000, 50, 96, 1.0, 0.6), (4096, 1024, 24, 1.0, 0.3), (8192, 1023, 17, 3.0, 0.5),
    (8193, 5000, 16, 1.0, 0.4), (20000, 70000, 8, 2.0, 0.2), (30000, 2, 40, 1.0, 0), (3, 1500000, 1, 1.0, 0)])
def test_against_the_oracle(M, t, n, v, h, scale, hot):
    ids, table, dy = make(n, v, h, t, seed=n + v + h, hot=hot, id_type=torch.int64 if n % 2 else torch.int32)
    ids, table, dy = ids.cuda(), table.cuda(), dy.cuda()
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=n, V=v, H=h, scale=scale))
    y = emb.forward(ids, table)
    assert torch.equal(y, (table[ids.long()].float() * scale).to(table.dtype))
    g = emb.backward(ids, dy)
    check_grad(g, ids, dy, v, scale)
    assert torch.equal(g, emb.backward(ids, dy))          # the same bits again
    base = torch.randn(v, h, device="cuda")
    into = base.clone()
    assert emb.backward(ids, dy, into=into) is into
    check_grad(into, ids, dy, v, scale, into=base)
    absent = torch.ones(v, dtype=torch.bool, device="cuda")
    absent[ids.long()] = False
    assert torch.equal(into[absent], base[absent])
    emb.check()


@pytest.mark.parametrize("runs", [[32], [33], [31, 34], [1, 32, 1], [33, 33], [33, 31], [95, 1, 32], [64], [65], [63, 66], [1, 64, 1], [64, 64], [65, 65], [128, 1], [10, 200, 3, 64, 70],
                                  [8192], [8191, 2], [5000, 5000, 7]])
def test_runs_at_the_edges_of_pieces(M, runs):
    """Sorted runs that start, end and fill pieces of 32 places in every way, in shuffled order."""
    ids = torch.cat([torch.full((r,), 3 * i + 1) for i, r in enumerate(runs)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))].cuda()
    v = 3 * len(runs) + 2
    dy = torch.randn(len(ids), 72, device="cuda").bfloat16()
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=len(ids), V=v, H=72))
    check_grad(emb.backward(ids, dy), ids, dy, v, 1.0)


def test_the_sum_does_not_depend_on_how_many_tokens_surround_it(M):
    """Integers small enough that every order of an fp32 sum is exact: gradients must be equal, at both sort forms."""
    for n in (8000, 50000):
        ids, _, _ = make(n, 900, 1, "fp32", seed=n, hot=0.5)
        dy = torch.randint(-8, 9, (n, 12), generator=torch.Generator().manual_seed(n)).float().cuda()
        emb = M.TokenEmbedding(M.EmbeddingConfig(N=n, V=900, H=12))
        ref = torch.zeros(900, 12, dtype=torch.float64, device="cuda").index_add_(0, ids.cuda(), dy.double())
        assert torch.equal(emb.backward(ids.cuda(), dy).double(), ref)


@pytest.mark.parametrize("n,v,h", [(65536, 900, 4), (65537, 400, 8), (66000, 1, 4), (150000, 70000, 4), (70001, 600000, 1)])
def test_many_tokens(M, n, v, h):
    """The sort's last length in one cluster, and beyond it; integers, so that every order of the sums is exact."""
    ids, _, _ = make(n, v, 1, "fp32", seed=n, hot=0.1)
    ids[::5000] = -1 if n % 2 else v
    dy = torch.randint(-4, 5, (n, h), generator=torch.Generator().manual_seed(n)).float().cuda()
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=n, V=v, H=h))
    ok = (ids >= 0) & (ids < v)
    ref = torch.zeros(v, h, dtype=torch.float64, device="cuda").index_add_(0, ids[ok].cuda(), dy[ok.cuda()].double())
    assert torch.equal(emb.backward(ids.cuda(), dy).double(), ref)
    base = torch.ones(v, h, device="cuda")
    assert torch.equal(emb.backward(ids.cuda(), dy, into=base).double(), ref + 1)


def test_padding_id_has_no_gradient(M):
    ids, table, dy = (t.cuda() for t in make(500, 20, 16, "bf16", seed=2))
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=500, V=20, H=16, padding_idx=7))
    assert torch.equal(emb.forward(ids, table), table[ids])
    check_grad(emb.backward(ids, dy), ids, dy, 20, 1.0, padding=7)
    base = torch.ones(20, 16, device="cuda")
    assert torch.equal(emb.backward(ids, dy, into=base)[7], torch.ones(16, device="cuda"))


@pytest.mark.parametrize("bad", [-1, 20, 2 ** 31 - 1, -2 ** 31, 2 ** 40])
def test_ids_outside_the_table_are_reported(M, bad):
    from top_softmax_router_gb300._lib import MoeError
    ids, table, dy = (t.cuda() for t in make(70, 20, 16, "fp32", seed=2))
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=70, V=20, H=16))
    ids[3] = bad
    y = emb.forward(ids, table)
    with pytest.raises(MoeError) as e:
        emb.check()
    assert e.value.code == -6 and not y[3].any() and torch.equal(y[4:], table[ids[4:]])
    g = emb.backward(ids, dy)
    with pytest.raises(MoeError):
        emb.check()
    check_grad(g, ids, dy, 20, 1.0)
    emb.check()


def test_strided_gradient_and_fewer_tokens(M):
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=20000, V=300, H=40))
    for n, pad in ((20000, 8), (777, 3), (1, 1)):
        ids, _, dy = make(n, 300, 40, "bf16", seed=n)
        wide = torch.full((n, 40 + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :40] = dy.cuda()
        check_grad(emb.backward(ids.cuda(), wide[:, :40]), ids, dy, 300, 1.0)


def test_no_tokens(M):
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=8, V=30, H=16))
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    table = torch.randn(30, 16, device="cuda")
    assert emb.forward(ids, table).shape == (0, 16)
    dy = torch.empty(0, 16, device="cuda")
    assert not emb.backward(ids, dy).any()
    base = torch.ones(30, 16, device="cuda")
    assert torch.equal(emb.backward(ids, dy, into=base.clone()), base)


def test_other_stream_and_graph(M):
    ids, table, dy = (t.cuda() for t in make(9000, 400, 64, "bf16", seed=8, hot=0.3))
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=9000, V=400, H=64))
    ref = emb.forward(ids, table), emb.backward(ids, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = emb.forward(ids, table, stream=s), emb.backward(ids, dy, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = emb.forward(ids, table), emb.backward(ids, dy)
    ids.copy_(ids.flip(0))
    g.replay()
    assert torch.equal(got[0], table[ids])
    check_grad(got[1], ids, dy, 400, 1.0)
