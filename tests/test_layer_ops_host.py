"""Refusals of the layer operators, on the host: bad shapes, types, pointers and workspaces are errors before any
launch, from C and from Python."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import top_softmax_router_gb300.build as B
    B.build()
    from top_softmax_router_gb300 import _lib
    return _lib


FAKE = ctypes.c_void_p(4096)      # never dereferenced: the checks fail first
ODD = ctypes.c_void_p(4097)
INVALID, SHAPE, SMALL = -1, -2, -3


def ref(s):
    return ctypes.byref(s)


@pytest.mark.parametrize("cfg,code", [((-1, 8, 1e-5), INVALID), ((4, 0, 1e-5), INVALID), ((4, 8, -1e-5), INVALID),
                                      ((4, 8, float("nan")), INVALID), ((4, 8, float("inf")), INVALID),
                                      ((4, 16385, 1e-5), SHAPE), ((4, 16384, 0.0), 0)])
def test_norm_shapes(lib, cfg, code):
    assert lib.load().moe_layernorm_workspace_bytes(ref(lib.LayerNormConfig(*cfg)), None) == code


def test_norm_arguments(lib):
    L, c = lib.load(), lib.LayerNormConfig(4, 8, 1e-5)

    def fwd(x=FAKE, ldx=8, w=None, b=None, y=FAKE, t=0, p=0):
        return L.moe_layernorm_forward(ref(c), x, ldx, w, b, y, None, None, t, p, None)

    assert fwd(x=None) == fwd(y=None) == fwd(ldx=7) == fwd(t=3) == fwd(t=-1) == fwd(t=1, p=2) == INVALID
    assert fwd(x=ODD) == fwd(w=ODD) == fwd(b=ODD) == fwd(y=ODD) == INVALID
    assert L.moe_layernorm_forward(None, FAKE, 8, None, None, FAKE, None, None, 0, 0, None) == INVALID

    def bwd(x=FAKE, ldx=8, mean=FAKE, rstd=FAKE, dy=FAKE, lddy=8, dx=FAKE, dw=FAKE, ws=FAKE, n=1 << 20, t=0):
        return L.moe_layernorm_backward(ref(c), x, ldx, None, mean, rstd, dy, lddy, dx, dw, None, t, 0, ws, n, None)

    assert bwd(x=None) == bwd(mean=None) == bwd(rstd=None) == bwd(dy=None) == bwd(ldx=1) == bwd(lddy=7) == INVALID
    assert bwd(ws=None) == bwd(ws=ODD) == bwd(dx=ODD) == bwd(dw=ODD) == bwd(t=9) == INVALID
    assert bwd(n=16) == SMALL


@pytest.mark.parametrize("cfg,code", [((-1, 8, 8, -1, 1.0), INVALID), ((4, 0, 8, -1, 1.0), SHAPE),
                                      ((4, 8, 0, -1, 1.0), SHAPE), ((4, 8, 8, -2, 1.0), INVALID),
                                      ((4, 8, 8, -1, float("inf")), INVALID), ((1 << 25, 8, 8, -1, 1.0), SHAPE),
                                      ((4, 1 << 30, 8, -1, 1.0), SHAPE), ((4, 8, (1 << 20) + 1, -1, 1.0), SHAPE)])
def test_embed_shapes(lib, cfg, code):
    assert lib.load().moe_embed_workspace_bytes(ref(lib.EmbedConfig(*cfg)), None, None) == code


def test_embed_arguments(lib):
    L, c = lib.load(), lib.EmbedConfig(4, 8, 8, -1, 1.0)

    def fwd(ids=FAKE, it=1, table=FAKE, y=FAKE, t=0, ws=FAKE, n=1 << 20):
        return L.moe_embed_forward(ref(c), ids, it, table, y, t, ws, n, None)

    assert fwd(ids=None) == fwd(table=None) == fwd(y=None) == fwd(ws=None) == fwd(it=2) == fwd(t=5) == INVALID
    assert fwd(ids=ODD) == fwd(ids=ctypes.c_void_p(4100)) == fwd(table=ODD) == fwd(ws=ODD) == INVALID
    assert fwd(n=8) == SMALL

    def bwd(ids=FAKE, it=0, dy=FAKE, ld=8, t=0, dW=FAKE, acc=0, ws=FAKE, n=1 << 24):
        return L.moe_embed_backward(ref(c), ids, it, dy, ld, t, dW, acc, ws, n, None)

    assert bwd(ids=None) == bwd(dy=None) == bwd(dW=None) == bwd(ld=7) == bwd(acc=2) == bwd(it=7) == bwd(ws=ODD) == INVALID
    assert bwd(n=256) == SMALL


@pytest.mark.parametrize("cfg,code", [
    ((-1, 8, 2, 1, 1, 2, 0, 1, 1.0), INVALID), ((4, 0, 2, 1, 1, 2, 0, 1, 1.0), INVALID),
    ((4, 8, 0, 1, 1, 2, 0, 1, 1.0), INVALID), ((4, 8, 2, 0, 1, 2, 0, 1, 1.0), INVALID),
    ((4, 8, 2, 1, 0, 2, 0, 1, 1.0), INVALID), ((4, 8, 2, 1, 1, 3, 0, 1, 1.0), INVALID),
    ((4, 8, 2, 1, 1, 2, 2, 1, 1.0), INVALID), ((4, 8, 2, 1, 1, 2, 0, 2, 1.0), INVALID),
    ((4, 8, 2, 1, 1, 2, 0, 1, float("nan")), INVALID), ((4, 1025, 2, 1, 1, 2, 0, 1, 1.0), SHAPE),
    ((4, 8, 2, 3, 1, 2, 0, 1, 1.0), SHAPE), ((4, 8, 2, 2, 3, 2, 0, 1, 1.0), SHAPE),
    ((4, 8, 5, 2, 1, 2, 0, 1, 1.0), SHAPE), ((4, 64, 33, 1, 1, 2, 0, 1, 1.0), SHAPE),
    ((4, 64, 2, 64, 64, 2, 0, 1, 1.0), SHAPE), ((4, 1024, 32, 32, 1, 2, 1, 1, 1.0), 0)])
def test_scores_shapes(lib, cfg, code):
    assert lib.load().moe_scores_workspace_bytes(ref(lib.ScoresConfig(*cfg)), None) == code


def test_scores_arguments(lib):
    L, c = lib.load(), lib.ScoresConfig(4, 8, 2, 1, 1, 2, 0, 1, 1.0)

    def fwd(l=FAKE, ld=8, t=0, b=None, idx=FAKE, w=FAKE, ws=FAKE, n=256):
        return L.moe_scores_forward(ref(c), l, ld, t, b, idx, w, None, ws, n, None)

    assert fwd(l=None) == fwd(ld=7) == fwd(t=4) == fwd(b=ODD) == fwd(idx=None) == fwd(w=None) == fwd(ws=None) == INVALID
    assert fwd(n=255) == SMALL

    def bwd(l=FAKE, ld=8, t=0, idx=FAKE, dw=FAKE, d=FAKE, ws=FAKE, n=256):
        return L.moe_scores_backward(ref(c), l, ld, t, idx, dw, d, ws, n, None)

    assert bwd(l=None) == bwd(ld=7) == bwd(idx=None) == bwd(dw=ODD) == bwd(d=None) == bwd(ws=ODD) == INVALID
    assert bwd(n=0) == SMALL


@pytest.mark.parametrize("cfg,code", [
    ((-1, 64, 10, 2, 1, 1.0), INVALID), ((4, 64, 10, 2, 1, 0.0), INVALID), ((4, 64, 10, 2, 1, -1.0), INVALID),
    ((4, 64, 10, 2, 1, float("nan")), INVALID), ((4, 64, 10, 2, 1, 1e-45), INVALID), ((4, 65, 10, 2, 1, 1.0), SHAPE),
    ((4, 64, 0, 2, 1, 1.0), SHAPE), ((4, 64, (1 << 20) + 1, 2, 1, 1.0), SHAPE), ((4, 64, 10, 257, 1, 1.0), SHAPE),
    ((4, 64, 10, 0, 1, 1.0), SHAPE), ((4, 64, 10, 2, 11, 1.0), SHAPE), ((4, 64, 10, 2, 0, 1.0), SHAPE),
    ((4, 64, 1 << 20, 256, 1, 1.0), 0)])
def test_distill_shapes(lib, cfg, code):
    assert lib.load().moe_distill_workspace_bytes(ref(lib.DistillConfig(*cfg)), None, None) == code


@pytest.mark.parametrize("H,V,P", [(64, 70000, 1), (64, 70000, 9), (1024, 32000, 4), (4096, 65536, 4), (320, 5000, 2), (64, 100, 3)])
def test_a_distill_workspace_serves_fewer_tokens(lib, H, V, P):
    f, b, last = ctypes.c_size_t(), ctypes.c_size_t(), (0, 0)
    for n in list(range(0, 600, 7)) + [1023, 1024, 1025, 2048, 5000, 8192, 30000]:
        assert lib.load().moe_distill_workspace_bytes(ref(lib.DistillConfig(n, H, V, 8, P, 1.0)), ref(f), ref(b)) == 0
        assert f.value >= last[0] and b.value >= last[1]
        last = f.value, b.value


def test_distill_arguments(lib):
    L, c = lib.load(), lib.DistillConfig(4, 64, 10, 2, 1, 1.0)

    def fwd(X=FAKE, W=FAKE, ids=FAKE, t=FAKE, loss=FAKE, lse=FAKE, ws=FAKE, n=1 << 24):
        return L.moe_distill_forward(ref(c), X, W, ids, t, loss, lse, None, ws, n, None)

    assert fwd(X=None) == fwd(W=None) == fwd(ids=None) == fwd(t=ODD) == fwd(loss=None) == fwd(lse=None) == INVALID
    assert fwd(X=ctypes.c_void_p(4104)) == fwd(ws=None) == INVALID
    assert fwd(n=256) == SMALL

    def bwd(X=FAKE, W=FAKE, ids=FAKE, lse=FAKE, g=FAKE, dX=FAKE, dW=FAKE, t=1, ws=FAKE, n=1 << 24):
        return L.moe_distill_backward(ref(c), X, W, ids, FAKE, lse, g, dX, dW, t, ws, n, None)

    assert bwd(X=None) == bwd(W=ODD) == bwd(ids=None) == bwd(lse=None) == bwd(g=None) == bwd(dX=None) == INVALID
    assert bwd(dW=ctypes.c_void_p(4104)) == bwd(t=2) == bwd(ws=None) == INVALID
    assert bwd(n=256) == SMALL


def test_python_refuses_host_tensors_types_and_shapes(lib):
    import top_softmax_router_gb300 as M
    ln = M.LayerNorm(M.LayerNormConfig(N=4, H=8), device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ln.forward(torch.zeros(4, 8))
    with pytest.raises(TypeError):
        ln.forward([[0.0] * 8])
    with pytest.raises(ValueError, match="at most 4"):
        ln.forward(torch.zeros(5, 8))
    emb = M.TokenEmbedding(M.EmbeddingConfig(N=4, V=9, H=8), device="cpu")
    with pytest.raises(TypeError, match="ids"):
        emb.forward(torch.zeros(4), torch.zeros(9, 8))
    with pytest.raises(ValueError, match="CUDA"):
        emb.forward(torch.zeros(4, dtype=torch.int64), torch.zeros(9, 8))
    r = M.ScoreRouter(M.ScoreRouterConfig(N=4, E=8, k=2), device="cpu")
    with pytest.raises(TypeError, match="logits"):
        r.forward(torch.zeros(4, 8, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        r.forward(torch.zeros(4, 8))
    with pytest.raises(ValueError, match="score"):
        M.ScoreRouter(M.ScoreRouterConfig(N=4, E=8, k=2, score="relu"), device="cpu")
    from top_softmax_router_gb300._lib import MoeError
    with pytest.raises(MoeError):
        M.ScoreRouter(M.ScoreRouterConfig(N=4, E=8, k=9), device="cpu")
