"""Products grouped by expert on the GPU against the float64 oracle, in bf16 and in 8 bits, forward and backward.

Tolerances, from the arithmetic before any run.  The tensor cores add 16 products of bf16 (32 of e4m3) at a time to an
fp32 accumulator and cut off towards zero: each addition, and each of the products as they are lined up, is off by at most
2^-23 of the largest partial sum, which the sum of the terms' magnitudes S bounds.
  y, dx   sums of K (O) terms, then shares added in fp32: (K / 16 + 32) 2^-23 S, and half a step of bf16 (2^-8 |y|)
  dw      1024 rows to an accumulator, those added in fp32: (min(n, 1024) / 16 + 32 + n / 1024) 2^-23 S, and half a step of
          its type
Operands in 8 bits are compared with the values that they stand for; dx with the product of dy's codes.
"""
import numpy as np
import pytest
import torch

from gpu_util import lib_api, need_gpu
from oracle import blocks8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    need_gpu()
    return lib_api()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ends(counts, lead=0):
    return [lead + sum(counts[:i]) for i in range(len(counts) + 1)]


class Case:
    """Inputs on the device, and their values in fp64."""

    def __init__(self, M, n, K, O, off=None, x8=False, w8=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.off_host = [0, n] if off is None else off
        E = len(self.off_host) - 1
        x = (torch.randn(n, K, generator=g) * torch.exp(torch.randn(n, 1, generator=g))).bfloat16()
        w = (torch.randn(E, O, K, generator=g) * K ** -0.5).bfloat16()
        dy = torch.randn(n, O, generator=g).bfloat16()
        inside = torch.zeros(n, dtype=torch.bool)
        inside[self.off_host[0]:self.off_host[-1]] = True
        self.inside = inside.numpy()
        self.x, self.w, self.dy = x.cuda(), w.cuda(), dy.cuda()
        self.off = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
        self.xs = self.ws = None
        X, W, D = host(x), host(w), host(dy)
        self.d_dw = D
        if x8:
            X = R.unpack(*R.pack(X))
            self.x, self.xs = M.Checkpoint8(M.Checkpoint8Config(N=n, H=K)).pack(self.x)
        if w8:
            W, D = R.unpack_weight(*R.pack_weight(W)), R.unpack(*R.pack(D))
            self.w, self.ws = M.pack_weight8(self.w)
        # what belongs to nobody is no number
        self.x.view(torch.uint8 if x8 else torch.int16)[~inside] = 0x7F if x8 else 0x7FC0
        self.dy[~inside] = float("nan")
        X, D, self.d_dw = (np.where(self.inside[:, None], a, 0) for a in (X, D, self.d_dw))
        self.X, self.W, self.D = X, W, D
        self.n, self.K, self.O, self.E = n, K, O, E

    def unit(self, M):
        return M.ExpertLinear(M.ExpertLinearConfig(N=self.n, K=self.K, O=self.O, E=self.E, blocks8=self.xs is not None or self.ws is not None))


def near(got, ref, size, terms, half):
    got = host(got)
    assert np.all(np.isfinite(got))
    bad = np.abs(got - ref) > (terms / 16 + 32) * 2.0 ** -23 * size + half * np.abs(ref) + 1e-37
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref).max())


def check(M, c, unit=None, forward=True, backward=True, dw_dtype=torch.float32):
    u = unit or c.unit(M)
    out = []
    if forward:
        y = u.forward(c.x, c.w, c.off, c.xs, c.ws)
        near(y, *R.linear(c.X, c.W, c.off_host), c.K, 2.0 ** -8)
        assert torch.all(y[torch.from_numpy(~c.inside)] == 0)
        out.append(y)
    if backward:
        dx, dw = u.backward(c.x, c.w, c.dy, c.off, c.xs, c.ws, dw_dtype=dw_dtype)
        near(dx, *R.linear_dx(c.D, c.W, c.off_host), c.O, 2.0 ** -8)
        assert torch.all(dx[torch.from_numpy(~c.inside)] == 0)
        assert dw.dtype == dw_dtype
        near(dw, *R.linear_dw(c.d_dw, c.X, c.off_host, c.E), min(c.n, 1024) + c.n / 64, torch.finfo(dw_dtype).eps / 2)
        out += [dx, dw]
    u.check()
    return out


KINDS = {"bf16": {}, "e4m3": dict(x8=True, w8=True)}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n,K,O", [(1, 16, 16), (1, 128, 256), (2, 144, 272), (8, 7168, 256), (1, 4096, 16), (127, 1040, 400), (128, 64, 128),
                                   (129, 256, 64), (256, 512, 512), (257, 640, 48), (300, 16, 2064), (1000, 2048, 320), (2100, 128, 144)])
def test_dense(M, kind, n, K, O):
    check(M, Case(M, n, K, O, **KINDS[kind], seed=n + K))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("counts,lead,tail", [([5], 0, 0), ([0, 0, 3], 0, 0), ([256, 256], 0, 0), ([1, 255, 257, 0, 64], 3, 9),
                                              ([0, 0, 0], 4, 1), ([700, 15, 16, 17, 63, 65, 300], 0, 31), ([1] * 70, 1, 0), ([1100, 1, 2050], 0, 0)])
def test_by_expert(M, kind, counts, lead, tail):
    off = ends(counts, lead)
    check(M, Case(M, off[-1] + tail, 320, 272, off, **KINDS[kind], seed=len(counts)))


@pytest.mark.parametrize("dw", [torch.float32, torch.bfloat16])
def test_a_checkpoint_beside_bf16_weights(M, dw):
    off = ends([100, 0, 333, 7])
    check(M, Case(M, 450, 272, 144, off, x8=True), forward=False, dw_dtype=dw)
    check(M, Case(M, 450, 272, 144, off, x8=True, w8=True), dw_dtype=dw)
    check(M, Case(M, 450, 272, 144, off), dw_dtype=dw)
    check(M, Case(M, 450, 272, 144, off, w8=True), forward=False, dw_dtype=dw)


@pytest.mark.parametrize("kind", list(KINDS))
def test_many_experts(M, kind):
    counts = [(7 * i) % 5 for i in range(1024)]
    off = ends(counts)
    check(M, Case(M, off[-1], 64, 48, off, **KINDS[kind]))


def test_no_rows(M):
    for off in (None, torch.zeros(2, dtype=torch.int32, device="cuda")):
        u = M.ExpertLinear(M.ExpertLinearConfig(N=8, K=32, O=16))
        x, w, dy = torch.empty(0, 32, device="cuda").bfloat16(), torch.zeros(1, 16, 32, device="cuda").bfloat16(), torch.empty(0, 16, device="cuda").bfloat16()
        assert u.forward(x, w, off).shape == (0, 16)
        dx, dw = u.backward(x, w, dy, off)
        assert dx.shape == (0, 32) and torch.all(dw == 0)


@pytest.mark.parametrize("kind", list(KINDS))
def test_strided_x(M, kind):
    c = Case(M, 200, 256, 128, **KINDS[kind])
    wide = torch.zeros(200, 256 + 48, dtype=c.x.dtype, device="cuda")
    wide.view(torch.uint8).fill_(0x7F)
    view = wide[:, 16:272]
    view.view(torch.uint8).copy_(c.x.view(torch.uint8)) if kind == "e4m3" else view.copy_(c.x)
    u = c.unit(M)
    assert torch.equal(u.forward(view, c.w, None, c.xs, c.ws), u.forward(c.x, c.w, None, c.xs, c.ws))
    if kind == "bf16":
        for p, q in zip(u.backward(view, c.w, c.dy), u.backward(c.x, c.w, c.dy)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("kind", list(KINDS))
def test_a_unit_serves_fewer_rows_and_repeats_its_bits(M, kind):
    big = Case(M, 900, 512, 256, ends([300, 0, 600]), **KINDS[kind])
    small = Case(M, 9, 512, 256, ends([2, 4, 3]), **KINDS[kind], seed=1)
    u = big.unit(M)
    for c in (big, small, big, small):
        for p, q in zip(check(M, c, u), check(M, c, u)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("kind", list(KINDS))
def test_a_row_that_holds_no_number_stays_alone(M, kind):
    c = Case(M, 300, 384, 144, **KINDS[kind])
    u = c.unit(M)
    y = u.forward(c.x, c.w, None, c.xs, c.ws)
    if kind == "bf16":
        c.x[77, 5] = float("nan")
        c.x[130, 383] = float("inf")
    else:
        c.x.view(torch.uint8)[77, 5] = 0x7F
        c.xs.view(torch.uint8)[130, 2] = 255
    z = u.forward(c.x, c.w, None, c.xs, c.ws)
    keep = torch.ones(300, dtype=torch.bool)
    keep[[77, 130]] = False
    assert torch.equal(y[keep], z[keep]) and torch.all(torch.isnan(z[77])) and not torch.any(torch.isfinite(z[130]))


@pytest.mark.parametrize("off", [[0, 5, 4, 10], [-1, 3, 4, 10], [0, 3, 4, 11], [0, 2000000000, 4, 10]])
def test_offsets_that_are_none_are_reported(M, off):
    from top_softmax_router_gb300._lib import MoeError
    u = M.ExpertLinear(M.ExpertLinearConfig(N=10, K=64, O=64, E=3))
    x, w, dy = torch.randn(10, 64, device="cuda").bfloat16(), torch.randn(3, 64, 64, device="cuda").bfloat16(), torch.randn(10, 64, device="cuda").bfloat16()
    bad = torch.tensor(off, dtype=torch.int32, device="cuda")
    for call in (lambda o: u.forward(x, w, o), lambda o: u.backward(x, w, dy, o, want_dw=False), lambda o: u.backward(x, w, dy, o, want_dx=False)):
        call(bad)
        with pytest.raises(MoeError):
            u.check()
        call(torch.tensor([0, 3, 4, 10], dtype=torch.int32, device="cuda"))
        u.check()


def test_other_streams_and_graphs(M):
    """A call on a side stream, and a captured step replayed on new contents, give the eager bits."""
    a, b = (Case(M, 70, 512, 256, ends([40, 30]), x8=True, w8=True, seed=s) for s in (1, 2))
    u = a.unit(M)
    want = [check(M, c, u) for c in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = u.forward(a.x, a.w, a.off, a.xs, a.ws, stream=side)
    dx, dw = u.backward(a.x, a.w, a.dy, a.off, a.xs, a.ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip((y, dx, dw), want[0]))
    names = ("x", "w", "dy", "off", "xs", "ws")
    held = {k: getattr(a, k).clone() for k in names}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy = u.forward(held["x"], held["w"], held["off"], held["xs"], held["ws"])
        gdx, gdw = u.backward(held["x"], held["w"], held["dy"], held["off"], held["xs"], held["ws"])
    for c, w in ((b, want[1]), (a, want[0])):
        for k in names:
            held[k].copy_(getattr(c, k))
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip((gy, gdx, gdw), w))
    u.check()


def test_waits_that_may_run_out_leave_the_context_usable(M):
    """A wait limit far below a copy's time: the calls end as ever or report the timeout; the next, after check(), gives
    the usual bits."""
    from top_softmax_router_gb300._lib import MoeError
    for kind in KINDS.values():
        for n in (20, 900):
            c = Case(M, n, 2048, 272, **kind)
            u = c.unit(M)
            want = check(M, c, u)
            M.set_wait_limit_ns(1000)
            try:
                u.forward(c.x, c.w, c.off, c.xs, c.ws)
                u.backward(c.x, c.w, c.dy, c.off, c.xs, c.ws)
                try:
                    u.check()
                except MoeError:
                    pass
            finally:
                M.set_wait_limit_ns(0)
            assert all(torch.equal(p, q) for p, q in zip(want, check(M, c, u)))


def test_large_offsets(M):
    """x and y of more than 2^32 bytes: the last rows."""
    n, K, O = 1_200_000, 2048, 2048
    g = torch.Generator().manual_seed(0)
    x = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
    w = (torch.randn(2, O, K, generator=g) * K ** -0.5).bfloat16().cuda()
    x[-5:] = torch.randn(5, K, generator=g).bfloat16().cuda()
    off = torch.tensor([0, n - 3, n], dtype=torch.int32, device="cuda")
    u = M.ExpertLinear(M.ExpertLinearConfig(N=n, K=K, O=O, E=2))
    y = u.forward(x, w, off)
    u.check()
    ref, size = R.linear(host(x[-5:]), host(w), [0, 2, 5])
    near(y[-5:], ref, size, K, 2.0 ** -8)
    assert torch.all(y[:-256] == 0)


def test_a_thread_of_its_own(M):
    """The first call of a thread that has used no CUDA yet (as autograd's has not), and two threads in turn."""
    import threading
    c = Case(M, 70, 272, 144, ends([40, 30]), x8=True, w8=True)
    u = c.unit(M)
    want, got = check(M, c, u), []
    stream = torch.cuda.current_stream()
    for _ in range(2):
        t = threading.Thread(target=lambda: got.append((u.forward(c.x, c.w, c.off, c.xs, c.ws, stream=stream),
                                                        *u.backward(c.x, c.w, c.dy, c.off, c.xs, c.ws, stream=stream))))
        t.start()
        t.join()
    assert len(got) == 2 and all(torch.equal(p, q) for g in got for p, q in zip(g, want))


CLUSTERS = 76                                    # of a GB300


def shares_of(tiles, blocks):
    """Into how many shares a tile of so many K blocks is split."""
    return max(1, min(CLUSTERS // tiles, blocks // 4)) if tiles else 1


@pytest.mark.parametrize("n,K,O", [(2500, 1536, 1536), (2500, 2560, 2560)])
def test_weight_gradients_of_several_accumulators(M, n, K, O):
    """More than 1024 rows to a share, so that dw's fp32 sums over accumulators are formed; with two shares to a tile (36
    tiles), and with more tiles than clusters (100)."""
    tiles, blocks = -(-K // 256) * -(-O // 256), -(-n // 64)
    per = -(-blocks // shares_of(tiles, blocks))
    assert per > 16 and (tiles > CLUSTERS or shares_of(tiles, blocks) > 1)
    check(M, Case(M, n, K, O), forward=False)
    check(M, Case(M, n, K, O, x8=True), forward=False, dw_dtype=torch.bfloat16)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("counts", [None, [257, 300, 513, 0, 300], [256] * 9])
def test_clusters_with_several_full_tiles(M, kind, counts):
    """y and dx of more than two rounds of tiles (a cluster's second and third accumulator, rows of both CTAs), each of more
    than four K blocks."""
    n = 2300 if counts is None else sum(counts)
    off = None if counts is None else ends(counts)
    rows = sum(-(-c // 256) for c in (counts or [n]))
    for K, O in ((1040, 4112), (4112, 1040)):
        c = Case(M, n, K, O, off, **KINDS[kind], seed=n)
        u = c.unit(M)
        y = u.forward(c.x, c.w, c.off, c.xs, c.ws)
        near(y, *R.linear(c.X, c.W, c.off_host), K, 2.0 ** -8)
        dx, _ = u.backward(c.x, c.w, c.dy, c.off, c.xs, c.ws, want_dw=False)
        near(dx, *R.linear_dx(c.D, c.W, c.off_host), O, 2.0 ** -8)
        u.check()
        assert rows * -(-max(K, O) // 256) > 2 * CLUSTERS and min(K, O) > 4 * 128
        del u


def values8(codes, scales):
    """The fp64 values of codes [n, k] with one scale for 128 of a row, or [E, o, k] with one for 128 x 128."""
    s = scales.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]
    return codes.double() * (s if codes.dim() == 2 else s.repeat_interleave(128, 1)[:, :codes.shape[1]])


@pytest.mark.parametrize("what", ["y", "dx"])
@pytest.mark.parametrize("kind,length", [("bf16", 1 << 16), ("e4m3", 1 << 17)])
def test_long_sums_are_not_cut_to_one_side(M, kind, length, what):
    """Positive terms, as many tiles as clusters and one more (so that none is split): the sums' mean error, one-sided where
    additions are cut off towards zero.  An accumulator takes 1024 products in bf16, 64 additions (4096 in e4m3, 128), each
    off by at most 2^-23 of it, its products by another 32 such steps; the accumulators are added in fp32.  Against the
    correctly rounded value an error of mean B moves the share B / 2^-8 of the values by a step of at most 2^-7: five sigmas
    of that beside it."""
    n, few = 77 * 256, 64
    g = torch.Generator(device="cuda").manual_seed(1)

    def positive(*shape):
        v = torch.rand(*shape, device="cuda", generator=g, dtype=torch.bfloat16).add_(0.5)
        return v.mul_(torch.exp2(torch.rand(*shape[:-1], 1, device="cuda", generator=g)).bfloat16())   # spread over a binade

    a = positive(n, length)
    K, O = (length, few) if what == "y" else (few, length)
    b = positive(1, few, length) / length                      # [1, few, length]: W itself for y, its transpose for dx
    w = b.contiguous() if what == "y" else b.transpose(1, 2).contiguous()
    u = M.ExpertLinear(M.ExpertLinearConfig(N=n, K=K, O=O, blocks8=kind == "e4m3" and what == "dx"))
    ck = M.Checkpoint8(M.Checkpoint8Config(N=n, H=length))
    codes, scales = ck.pack(a) if kind == "e4m3" else (None, None)
    wc, ws = M.pack_weight8(w) if kind == "e4m3" else (w, None)
    if what == "y":
        got = u.forward(a if kind == "bf16" else codes, wc, None, scales, ws)
    else:
        got = u.backward(None, wc, a, None, None, ws, want_dw=False)[0]
    u.check()
    W = (w.double() if kind == "bf16" else values8(wc, ws))[0]
    W = W.t() if what == "y" else W                            # [length, few]
    total = 0.0
    for r in range(0, n, 1024):
        at = slice(r, min(n, r + 1024))
        ref = (a[at].double() if kind == "bf16" else values8(codes[at], scales[at])) @ W
        total += ((got[at].double() - ref.bfloat16().double()) / ref).sum().item()
    products, additions = (1024, 64) if kind == "bf16" else (4096, 128)
    bound = (additions + 32) * 2.0 ** -23 + length / products * 2.0 ** -24
    assert abs(total / got.numel()) <= bound + 5 * (bound * 2.0 ** -6 / got.numel()) ** 0.5


def test_a_check_clears_on_the_stream_it_checked(M):
    """check(stream) while the current stream is busy: what a later call on `stream` reports is not wiped."""
    from top_softmax_router_gb300._lib import MoeError
    u = M.ExpertLinear(M.ExpertLinearConfig(N=10, K=64, O=64, E=3))
    x, w = torch.randn(10, 64, device="cuda").bfloat16(), torch.randn(3, 64, 64, device="cuda").bfloat16()
    bad = torch.tensor([0, 5, 4, 10], dtype=torch.int32, device="cuda")
    side, busy = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    u.forward(x, w, bad, stream=side)
    with torch.cuda.stream(busy):
        torch.cuda._sleep(400_000_000)             # cycles: a fifth of a second
        with pytest.raises(MoeError):
            u.check(stream=side)
        u.forward(x, w, bad, stream=side)
    torch.cuda.synchronize()
    with pytest.raises(MoeError):
        u.check(stream=side)
    u.check()


@pytest.mark.parametrize("kind,K,O", [("e4m3", 7168, 2048), ("bf16", 3584, 2048), ("bf16", 7168, 2048), ("e4m3", 2048, 256), ("bf16", 320, 272)])
def test_no_share_is_empty(M, kind, K, O):
    """A tile's shares have K blocks each: as many places of the workspace are written as there are such shares."""
    c = Case(M, 8, K, O, **KINDS[kind])
    u = c.unit(M)
    places = u.ws[:M.linear_workspace_bytes(u.cfg)[0]][-CLUSTERS * 256 * 256 * 4:].view(torch.float32).view(CLUSTERS, -1)
    places.fill_(float("nan"))
    near(u.forward(c.x, c.w, None, c.xs, c.ws), *R.linear(c.X, c.W, c.off_host), K, 2.0 ** -8)
    tiles, blocks = -(-O // 256), -(-K // (128 if kind == "e4m3" else 64))
    per = -(-blocks // shares_of(tiles, blocks))
    per = -(-per // 4) * 4 if kind == "e4m3" else per
    shares = -(-blocks // per)
    assert (~torch.isnan(places)).any(dim=1).sum().item() == (tiles * shares if shares > 1 else 0)


@pytest.mark.parametrize("kind", list(KINDS))
def test_gradients_past_2_to_31_elements(M, kind):
    """x, dy and dx of more than 2^31 elements: the last rows, and what they give dw."""
    n, K, O = 1_100_000, 2048, 2048
    g = torch.Generator().manual_seed(4)
    x, dy = (torch.zeros(n, 2048, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = (torch.randn(2, O, K, generator=g) * K ** -0.5).bfloat16().cuda()
    x[-5:], dy[-5:] = torch.randn(5, K, generator=g).bfloat16().cuda(), torch.randn(5, O, generator=g).bfloat16().cuda()
    off = torch.tensor([0, n - 3, n], dtype=torch.int32, device="cuda")
    X, W, D, xs, ws = host(x[-5:]), host(w), host(dy[-5:]), None, None
    d_dw = D
    if kind == "e4m3":
        X, W, D = R.unpack(*R.pack(X)), R.unpack_weight(*R.pack_weight(W)), R.unpack(*R.pack(D))
        x, xs = M.Checkpoint8(M.Checkpoint8Config(N=n, H=K)).pack(x)
        w, ws = M.pack_weight8(w)
    u = M.ExpertLinear(M.ExpertLinearConfig(N=n, K=K, O=O, E=2, blocks8=kind == "e4m3"))
    if kind == "e4m3":
        y = u.forward(x, w, off, xs, ws)
        near(y[-5:], *R.linear(X, W, [0, 2, 5]), K, 2.0 ** -8)
        del y
    dx, dw = u.backward(x, w, dy, off, xs, ws)
    u.check()
    near(dx[-5:], *R.linear_dx(D, W, [0, 2, 5]), O, 2.0 ** -8)
    assert not dx[:-5].any()
    near(dw, *R.linear_dw(d_dw, X, [0, 2, 5], 2), 5, 2.0 ** -24)


def test_weights_past_2_to_31_elements(M):
    """The last experts' rows and gradients."""
    E, n, K, O = 520, 20, 2048, 2048
    g = torch.Generator().manual_seed(5)
    off_host = [0] * (E - 2) + [5, 5, 20]
    x, dy = torch.randn(n, K, generator=g).bfloat16().cuda(), torch.randn(n, O, generator=g).bfloat16().cuda()
    w = torch.zeros(E, O, K, dtype=torch.bfloat16, device="cuda")
    w[-3:] = (torch.randn(3, O, K, generator=g) * K ** -0.5).bfloat16().cuda()
    off = torch.tensor(off_host, dtype=torch.int32, device="cuda")
    X, W, D, last = host(x), host(w[-3:]), host(dy), off_host[-4:]
    u = M.ExpertLinear(M.ExpertLinearConfig(N=n, K=K, O=O, E=E))
    near(u.forward(x, w, off), *R.linear(X, W, last), K, 2.0 ** -8)
    dx, dw = u.backward(x, w, dy, off)
    u.check()
    near(dx, *R.linear_dx(D, W, last), O, 2.0 ** -8)
    near(dw[-3:], *R.linear_dw(D, X, last, 3), n, 2.0 ** -24)
    assert not dw[:-3].any()
    wc, ws = M.pack_weight8(w)
    rc, rs = R.pack_weight(W)
    assert np.array_equal(host(wc[-3:]), rc) and np.array_equal(host(ws[-3:]), rs)
