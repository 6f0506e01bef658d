"""The 8-bit oracle pinned on the CPU: to torch's e4m3 conversion, to the scale's definition, to differences."""
import numpy as np
import torch

from oracle import blocks8_ref as R


def test_codes_are_torchs_e4m3():
    v = np.concatenate([np.linspace(-448, 448, 20001), np.geomspace(2.0 ** -12, 448, 5000), [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    v = torch.tensor(v, dtype=torch.float32)
    want = v.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3(v.double().numpy()), want)


def test_scales_are_the_smallest_that_hold_the_largest():
    a = np.concatenate([np.geomspace(1e-35, 3e38, 4001), 448 * 2.0 ** np.arange(-100, 100), 448 * 2.0 ** np.arange(-100, 100) * (1 + 2.0 ** -20)])
    s = R.scale_of(a)
    assert np.all(a <= 448 * s) and np.all(a > 224 * s)
    assert R.scale_of(0.0) == 1.0 and R.scale_of(1e-45) == 2.0 ** -127


def test_packing_is_off_by_at_most_half_a_step():
    g = np.random.default_rng(0)
    x = g.standard_normal((7, 300)) * np.exp(g.standard_normal((7, 300)))
    c, s = R.pack(x)
    v = R.unpack(c, s)
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * np.repeat(s, 128, axis=1)[:, :300]))
    w = g.standard_normal((2, 200, 140))
    c, s = R.pack_weight(w)
    assert s.shape == (2, 2, 2) and np.all(np.abs(R.unpack_weight(c, s) - w) <= 2.0 ** -4 * np.abs(w) + 2.0 ** -10 * s.max())


def test_what_is_no_number_leaves_its_block_alone():
    x = np.array([[1.0, np.nan, np.inf, -3.0, -np.inf] + [0.0] * 200])
    c, s = R.pack(x)
    v = R.unpack(c, s)
    assert np.array_equal(np.isnan(v[0, :5]), [False, True, True, False, True])
    assert v[0, 0] == 1 and v[0, 3] == -3 and s[0, 1] == 1


def test_rms_gradients_against_differences():
    g = np.random.default_rng(1)
    h, w, dy, dh = g.standard_normal((3, 9)), g.standard_normal(9), g.standard_normal((3, 9)), g.standard_normal((3, 9))
    dx, dw = R.rms_backward(h, w, dy, dh, 1e-3)

    def f(a, b):
        return (R.rms_forward(a, b, 1e-3)[0] * dy).sum() + (a * dh).sum()

    for i in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[i] = 1e-5
        assert abs((f(h + d, w) - f(h - d, w)) / 2e-5 - dx[i]) < 1e-8
    for i in range(9):
        d = np.zeros(9)
        d[i] = 1e-5
        assert abs((f(h, w + d) - f(h, w - d)) / 2e-5 - dw[i]) < 1e-8


def test_products_by_expert_against_autograd():
    g = torch.Generator().manual_seed(2)
    off = [1, 4, 4, 9]
    x = torch.randn(10, 5, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(3, 6, 5, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(10, 6, generator=g, dtype=torch.float64)
    y = torch.stack([x[n] @ w[0 if n < 4 else 2].t() if 1 <= n < 9 else torch.zeros(6, dtype=torch.float64) for n in range(10)])
    (y * dy).sum().backward()
    X, W, D = x.detach().numpy(), w.detach().numpy(), dy.numpy()
    assert np.allclose(R.linear(X, W, off)[0], y.detach().numpy(), atol=1e-13)
    assert np.allclose(R.linear_dx(D, W, off)[0], x.grad.numpy(), atol=1e-13)
    assert np.allclose(R.linear_dw(D, X, off, 3)[0], w.grad.numpy(), atol=1e-13)
