"""Refusals of the 8-bit blocks, the RMS norm and the products by expert, on the host: bad shapes, types, pointers and
workspaces are errors before any launch, from C and from Python."""
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
OFF8 = ctypes.c_void_p(4104)
INVALID, SHAPE, SMALL = -1, -2, -3


def ref(s):
    return ctypes.byref(s)


def test_blocks8(lib):
    L = lib.load()

    def pack(x=FAKE, ld=8, t=0, n=4, h=8, c=FAKE, s=FAKE):
        return L.moe_blocks8_pack(x, ld, t, n, h, c, s, None)

    assert pack(x=None) == pack(ld=7) == pack(t=3) == pack(n=-1) == pack(h=0) == pack(c=None) == pack(s=None) == pack(x=ODD) == INVALID
    assert pack(h=(1 << 20) + 1, ld=1 << 21) == pack(n=1 << 31) == SHAPE
    assert pack(n=0, x=None) == 0

    def unpack(c=FAKE, s=FAKE, n=4, h=8, y=FAKE, t=1):
        return L.moe_blocks8_unpack(c, s, n, h, y, t, None)

    assert unpack(c=None) == unpack(s=None) == unpack(y=None) == unpack(y=ODD) == unpack(t=-1) == unpack(n=-1) == unpack(h=0) == INVALID
    assert unpack(n=1 << 31) == SHAPE and unpack(n=0, c=None) == 0

    def weight(w=FAKE, t=1, E=1, O=8, K=8, c=FAKE, s=FAKE):
        return L.moe_blocks8_pack_weight(w, t, E, O, K, c, s, None)

    assert weight(w=None) == weight(t=9) == weight(E=-1) == weight(O=-1) == weight(K=0) == weight(c=None) == weight(s=None) == weight(w=ODD) == INVALID
    assert weight(K=(1 << 20) + 1) == weight(O=(1 << 20) + 1) == weight(E=1 << 20, O=1 << 20, K=1 << 20) == SHAPE
    assert weight(E=0, w=None) == weight(O=0, w=None) == 0


@pytest.mark.parametrize("cfg,code", [((-1, 8, 1e-6), INVALID), ((4, 0, 1e-6), INVALID), ((4, 8, -1e-6), INVALID),
                                      ((4, 8, float("nan")), INVALID), ((4, 8, float("inf")), INVALID),
                                      ((4, 16385, 1e-6), SHAPE), ((4, 16384, 0.0), 0)])
def test_rms_shapes(lib, cfg, code):
    assert lib.load().moe_rmsnorm_workspace_bytes(ref(lib.RmsNormConfig(*cfg)), None) == code


def test_rms_arguments(lib):
    L, c = lib.load(), lib.RmsNormConfig(4, 8, 1e-6)

    def fwd(x=FAKE, ldx=8, r=FAKE, ldr=8, w=None, h=FAKE, y=FAKE, q=FAKE, s=FAKE, rstd=FAKE, t=0, p=0):
        return L.moe_rmsnorm_forward(ref(c), x, ldx, r, ldr, w, h, y, q, s, rstd, t, p, None)

    assert fwd(x=None) == fwd(ldx=7) == fwd(ldr=7) == fwd(t=3) == fwd(t=1, p=2) == fwd(q=None) == fwd(s=None) == INVALID
    assert fwd(x=ODD) == fwd(r=ODD) == fwd(w=ODD) == fwd(h=ODD) == fwd(y=ODD) == fwd(rstd=ODD) == fwd(r=None) == INVALID
    assert L.moe_rmsnorm_forward(None, FAKE, 8, None, 8, None, None, FAKE, None, None, None, 0, 0, None) == INVALID

    def bwd(h=FAKE, ldh=8, w=None, rstd=FAKE, dy=FAKE, ldy=8, dh=FAKE, lddh=8, dx=FAKE, dw=FAKE, t=0, p=0, ws=FAKE, n=1 << 20):
        return L.moe_rmsnorm_backward(ref(c), h, ldh, w, rstd, dy, ldy, dh, lddh, dx, dw, t, p, ws, n, None)

    assert bwd(h=None) == bwd(ldh=1) == bwd(rstd=None) == bwd(dy=None) == bwd(ldy=7) == bwd(lddh=7) == bwd(t=9) == INVALID
    assert bwd(ws=None) == bwd(ws=ODD) == bwd(dx=ODD) == bwd(dw=ODD) == bwd(dh=ODD) == bwd(w=ODD) == bwd(h=ODD) == INVALID
    assert bwd(n=16) == SMALL


@pytest.mark.parametrize("H", [8, 256, 264, 1000, 7168, 7176, 16384])
def test_an_rms_workspace_serves_fewer_rows(lib, H):
    b, last = ctypes.c_size_t(), 0
    for n in list(range(0, 3000, 37)) + [10 ** 5]:
        assert lib.load().moe_rmsnorm_workspace_bytes(ref(lib.RmsNormConfig(n, H, 0.0)), ref(b)) == 0
        assert b.value >= last
        last = b.value


@pytest.mark.parametrize("cfg,code", [
    ((-1, 16, 16, 1, 0), INVALID), ((4, 0, 16, 1, 0), INVALID), ((4, 16, 0, 1, 0), INVALID), ((4, 16, 16, 0, 0), INVALID),
    ((4, 16, 16, 1, 2), INVALID), ((4, 24, 16, 1, 0), SHAPE), ((4, 16, 8, 1, 0), SHAPE), ((4, 16, 16, 1025, 0), SHAPE),
    ((4, (1 << 20) + 16, 16, 1, 0), SHAPE), ((1 << 30, 1 << 20, 16, 1, 0), SHAPE), ((4, 1 << 20, 1 << 20, 1024, 0), SHAPE),
    ((4, 1 << 20, 16, 1024, 1), 0), ((0, 16, 16, 1, 0), 0)])
def test_linear_shapes(lib, cfg, code):
    assert lib.load().moe_linear_workspace_bytes(ref(lib.LinearConfig(*cfg)), None, None) == code


def test_linear_arguments(lib):
    L, c, c8, cE = lib.load(), lib.LinearConfig(4, 16, 32, 1, 0), lib.LinearConfig(4, 16, 32, 1, 1), lib.LinearConfig(4, 16, 32, 3, 1)

    def fwd(c=c, x=FAKE, ld=16, xs=None, w=FAKE, ws_=None, off=FAKE, y=FAKE, ws=FAKE, n=1 << 26):
        return L.moe_linear_forward(ref(c), x, ld, xs, w, ws_, off, y, ws, n, None)

    assert fwd(x=None) == fwd(w=None) == fwd(y=None) == fwd(ws=None) == fwd(ws=OFF8) == fwd(x=OFF8) == fwd(w=OFF8) == fwd(y=OFF8) == INVALID
    assert fwd(xs=FAKE) == fwd(ws_=FAKE) == fwd(ld=15) == fwd(ld=20) == fwd(off=ODD) == fwd(c=cE, off=None) == INVALID
    assert fwd(xs=FAKE, ws_=FAKE, ld=24) == INVALID and fwd(n=1 << 20) == SMALL
    assert L.moe_linear_forward(None, FAKE, 16, None, FAKE, None, None, FAKE, FAKE, 1 << 26, None) == INVALID

    def bwd(c=c8, x=FAKE, ld=16, xs=FAKE, w=FAKE, ws_=FAKE, off=FAKE, dy=FAKE, dx=FAKE, dw=FAKE, t=0, ws=FAKE, n=1 << 26):
        return L.moe_linear_backward(ref(c), x, ld, xs, w, ws_, off, dy, dx, dw, t, ws, n, None)

    assert bwd(x=None) == bwd(w=None) == bwd(dy=None) == bwd(ws=None) == bwd(x=OFF8) == bwd(w=OFF8) == bwd(dy=OFF8) == INVALID
    assert bwd(dx=OFF8) == bwd(dw=OFF8) == bwd(t=2) == bwd(ld=32) == bwd(off=ODD) == bwd(c=cE, off=None) == INVALID
    assert bwd(c=c) == bwd(c=c, xs=None) == bwd(c=c, ws_=None) == INVALID          # no room for 8 bits
    assert bwd(n=1 << 20) == SMALL
    assert bwd(c=lib.LinearConfig(0, 16, 32, 1, 1), dw=None, x=None, dy=None) == 0


@pytest.mark.parametrize("blocks8", [0, 1])
def test_a_linear_workspace_serves_fewer_rows(lib, blocks8):
    f, b, last = ctypes.c_size_t(), ctypes.c_size_t(), (0, 0)
    for n in list(range(0, 600, 7)) + [5000, 131072]:
        assert lib.load().moe_linear_workspace_bytes(ref(lib.LinearConfig(n, 272, 144, 5, blocks8)), ref(f), ref(b)) == 0
        assert f.value >= last[0] and b.value >= last[1]
        last = f.value, b.value


def test_python_refuses_host_tensors_types_and_shapes(lib):
    import top_softmax_router_gb300 as M
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        M.Checkpoint8(M.Checkpoint8Config(N=4, H=0))
    ck = M.Checkpoint8(M.Checkpoint8Config(N=4, H=8))
    with pytest.raises(ValueError, match="CUDA"):
        ck.pack(torch.zeros(4, 8))
    with pytest.raises(TypeError, match="x"):
        ck.pack(torch.zeros(4, 8, dtype=torch.float64))
    with pytest.raises(ValueError, match="at most 4"):
        ck.pack(torch.zeros(5, 8))
    with pytest.raises(TypeError, match="codes"):
        ck.unpack(torch.zeros(4, 8), torch.zeros(4, 1))
    with pytest.raises(TypeError, match="w"):
        M.pack_weight8(torch.zeros(4, 8))
    rms = M.RMSNorm(M.RMSNormConfig(N=4, H=8), device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        rms.forward(torch.zeros(4, 8))
    with pytest.raises(TypeError):
        rms.forward([[0.0] * 8])
    lin = M.ExpertLinear(M.ExpertLinearConfig(N=4, K=16, O=32, E=2), device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        lin.forward(torch.zeros(4, 16, dtype=bf), torch.zeros(2, 32, 16, dtype=bf))
    with pytest.raises(TypeError, match="x"):
        lin.forward(torch.zeros(4, 16), torch.zeros(2, 32, 16, dtype=bf))
    with pytest.raises(ValueError, match="both or neither"):
        lin.forward(torch.zeros(4, 16, dtype=bf), torch.zeros(2, 32, 16, dtype=bf), x_scales=torch.zeros(4, 1))
    with pytest.raises(TypeError, match="dy"):
        lin.backward(None, None, torch.zeros(4, 32))
    with pytest.raises(TypeError, match="x: expected bfloat16"):
        M.rms_norm_linear8(torch.zeros(4, 8), None, None, rms, lin)


@pytest.mark.parametrize("cfg,code", [((2 ** 31 - 4096, 16, 16, 1, 0), 0), ((2 ** 31 - 4095, 16, 16, 1, 0), SHAPE), ((2 ** 31 - 1, 16, 16, 3, 0), SHAPE),
                                      ((2 ** 30, 144, 16, 1, 1), SHAPE), ((2 ** 30 - 1, 144, 16, 1, 1), 0), ((2 ** 30, 16, 144, 1, 1), SHAPE), ((2 ** 30, 144, 144, 1, 0), 0)])
def test_linear_rows_that_32_bits_cannot_count(lib, cfg, code):
    """A kernel's row, plus a tile, or plus the rows that all its warps zero in a step, has to stay below 2^31; so have the
    blocks of an operand that is packed or restored."""
    assert 2 ** 31 - 4096 + 76 * 16 + 256 < 2 ** 31
    assert lib.load().moe_linear_workspace_bytes(ref(lib.LinearConfig(*cfg)), None, None) == code


def test_sizes_past_32_bits_are_refused(lib):
    """Their lower bits alone would be another shape."""
    import top_softmax_router_gb300 as M
    big = 2 ** 32 + 16
    for make in (lambda: M.ExpertLinear(M.ExpertLinearConfig(N=big, K=16, O=16), device="cpu"),
                 lambda: M.ExpertLinear(M.ExpertLinearConfig(N=4, K=big, O=16), device="cpu"),
                 lambda: M.RMSNorm(M.RMSNormConfig(N=big, H=8), device="cpu"),
                 lambda: M.LayerNorm(M.LayerNormConfig(N=big, H=8), device="cpu")):
        with pytest.raises(ValueError, match="out of range"):
            make()
    with pytest.raises(ValueError, match="out of range"):
        M.pack_weight8(torch.empty(1, dtype=torch.bfloat16).expand(2 ** 32 + 1, 1, 1))
