"""8-bit blocks on the GPU against the oracle: codes, scales and restored values are those of the definition, bit for bit
(the scale is a power of two, so that nothing but the rounding to e4m3 rounds)."""
import numpy as np
import pytest
import torch

from gpu_util import lib_api, need_gpu
from oracle import blocks8_ref as R

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def M():
    need_gpu()
    return lib_api()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rows(n, h, t, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))
    x[torch.rand(n, h, generator=g) < 0.02] *= 30
    x[:, : h // 3] *= 2.0 ** -9          # below the codes' ordinary numbers in part
    return x.to(TYPES[t])


def check(M, x, unit=None, place=lambda t: t.cuda()):
    n, h = x.shape
    u = unit or M.Checkpoint8(M.Checkpoint8Config(N=n, H=h))
    c, s = u.pack(place(x))
    rc, rs = R.pack(host(x))
    assert c.dtype == torch.float8_e4m3fn and s.dtype == torch.float8_e8m0fnu
    assert np.array_equal(host(c), rc, equal_nan=True) and np.array_equal(host(s), rs)
    for t in TYPES.values():
        y = u.unpack(c, s, t)
        want = torch.from_numpy(R.unpack(rc, rs)).to(t)
        assert y.dtype == t and np.array_equal(host(y), host(want), equal_nan=True)
    return c, s


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n,h", [(1, 1), (1, 128), (3, 129), (5, 1000), (2, 1001), (70, 64), (33, 2048), (300, 136), (9, 7168), (1, 20000)])
def test_against_the_oracle(M, t, n, h):
    check(M, rows(n, h, t, seed=n + h))


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,first", [(8, 0), (3, 0), (16, 8), (5, 3)])
def test_strided_rows(M, t, pad, first):
    def place(v):
        wide = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=v.dtype, device="cuda")
        view = wide[:, first:first + v.shape[1]]
        view.copy_(v)
        return view
    check(M, rows(19, 264, t, seed=3), place=place)


def test_every_magnitude(M):
    """Blocks whose largest value runs through the type, each exactly at 448 x 2^e, just above it, and 0."""
    e = torch.arange(-149, 128, dtype=torch.float64)
    top = torch.cat([1.75 * 2.0 ** e[e < 127], 1.7500001 * 2.0 ** e[e < 127], 2.0 ** e, torch.tensor([0.0, 3.3895e38, 3.4e38])])
    x = torch.zeros(len(top), 128, dtype=torch.float64)
    x[:, 5] = top
    x[:, 7] = -top * 0.4
    x[:, 100] = top * 2.0 ** -12
    check(M, x.float())


def test_what_is_no_number(M):
    x = rows(6, 300, "bf16", seed=4)
    x[0, 3], x[1, 200], x[2, 299] = float("nan"), float("inf"), float("-inf")
    x[3] = float("nan")
    x[4, :128] = 0
    check(M, x)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("E,O,K", [(1, 1, 1), (1, 128, 128), (2, 129, 200), (3, 16, 1040), (1, 257, 77), (5, 200, 136)])
def test_weights(M, t, E, O, K):
    w = rows(E * O, K, t, seed=O).view(E, O, K)
    c, s = M.pack_weight8(w.cuda())
    rc, rs = R.pack_weight(host(w))
    assert np.array_equal(host(c), rc) and np.array_equal(host(s), rs)


def test_none_fewer_and_another_stream(M):
    u = M.Checkpoint8(M.Checkpoint8Config(N=50, H=260))
    c, s = u.pack(torch.empty(0, 260, device="cuda"))
    assert c.shape == (0, 260) and s.shape == (0, 3) and u.unpack(c, s).shape == (0, 260)
    check(M, rows(7, 260, "bf16"), unit=u)
    side = torch.cuda.Stream()
    x = rows(50, 260, "bf16").cuda()
    side.wait_stream(torch.cuda.current_stream())
    c, s = u.pack(x, stream=side)
    y = u.unpack(c, s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, u.unpack(*u.pack(x)))


def test_a_large_checkpoint(M):
    """More than 2^31 elements: the row's offset needs 64 bits."""
    n, h = 300_000, 7168
    x = torch.zeros(n, h, dtype=torch.bfloat16, device="cuda")
    x[-3:] = rows(3, h, "bf16", seed=9).cuda()
    u = M.Checkpoint8(M.Checkpoint8Config(N=n, H=h))
    c, s = u.pack(x)
    rc, rs = R.pack(host(x[-3:]))
    assert np.array_equal(host(c[-3:]), rc) and np.array_equal(host(s[-3:]), rs)
    assert np.array_equal(host(u.unpack(c, s)[-3:]), R.unpack(rc, rs))


def test_fp16_at_the_top_of_its_range(M):
    """The finite fp16 values whose nearest code would stand for 65536, an infinity there: restored in fp16 they are finite,
    and off by at most 2^-4 as every other."""
    top = torch.arange(0x7A00, 0x7C00, dtype=torch.int16).view(torch.float16)      # 49152 .. 65504
    x = torch.stack([top.view(4, 128), -top.view(4, 128)]).view(8, 128)
    x[5, 64:] = 1.0
    u = M.Checkpoint8(M.Checkpoint8Config(N=8, H=128))
    c, s = u.pack(x.cuda())
    rc, rs = R.pack(host(x))
    assert np.array_equal(host(s), rs) and np.array_equal(host(c), np.where((rs == 2.0 ** 8) & (np.abs(rc) == 256), np.sign(rc) * 240, rc))
    y = host(u.unpack(c, s, torch.float16))
    assert np.all(np.isfinite(y)) and np.all(np.abs(y - host(x)) <= 2.0 ** -4 * np.abs(host(x)))
