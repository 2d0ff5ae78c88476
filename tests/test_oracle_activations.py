"""CPU pins of oracle/activations.py: the 8-bit form against torch's own e4m3
cast and brute force, and every gradient against central differences."""
import numpy as np
import pytest
import torch

from oracle import activations as oa


def rng(*key):
    return np.random.default_rng(np.random.SeedSequence(list(key)))


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = oa.e4m3_values()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rounding_is_to_the_nearest_value(fmt):
    values = np.unique(oa.e4m3_values()[~np.isnan(oa.e4m3_values())]) if fmt == "e4m3" else np.arange(-127, 128.0)
    v = np.concatenate([rng(1).uniform(-oa.TOP[fmt], oa.TOP[fmt], 4000), rng(2).normal(0, 0.01, 4000), values,
                        (values[1:] + values[:-1]) / 2])
    got = oa.act8_round(v, fmt)
    best = np.abs(v[:, None] - values[None, :]).min(axis=1)
    assert np.array_equal(np.abs(v - got), best)
    if fmt == "e4m3":
        want = torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()
        exact = v == v.astype(np.float32)            # where the detour over fp32 rounds nothing
        assert np.array_equal(got[exact], want[exact])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_exponent_is_the_least_that_fits(fmt):
    top = oa.TOP[fmt]
    edges = [top * 2.0 ** k for k in (-125, -120, -119, -3, 0, 1, 100)]
    amax = np.array([0.0, 1e-45, 2.0 ** -126, 1.0, 3.3e38] + edges + [np.nextafter(e, np.inf) for e in edges] +
                    [np.nextafter(e, 0) for e in edges])
    for a, k in zip(amax, oa.act8_exponent(amax, fmt)):
        assert k >= -120 and a <= top * 2.0 ** k
        assert k == -120 or a > top * 2.0 ** (k - 1)


def test_values_of_a_packed_block_are_exact_in_bf16():
    x = np.concatenate([rng(3).normal(0, 10.0 ** e, (4, 96)) for e in (-41, -38, -20, 0, 20, 37)])
    for fmt in oa.TOP:
        v, _ = oa.act8(x, fmt)
        assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)


def differences(f, x, eps=1e-6):
    """Central differences of the scalar function f at x."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        at = x[i]
        x[i] = at + eps
        hi = f(x)
        x[i] = at - eps
        lo = f(x)
        x[i] = at
        g[i] = (hi - lo) / (2 * eps)
    return g


# Central differences of a smooth function of order one with eps = 1e-6: truncation
# ~eps^2, cancellation ~2^-52 / eps = 2e-10 times the function's size (below 100 here).
DIFF_TOL = 1e-7


def test_norm_gradient_against_differences():
    r = rng(4)
    x, res, w, dy = r.normal(size=(3, 7)), r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=(3, 7))
    dh = r.normal(size=(3, 7))

    def loss(x_, res_, w_):
        h = x_ + res_
        return (oa.rms_norm(h, w_, 1e-6)[0] * dy).sum() + (h * dh).sum()

    h = x + res
    dx, dw = oa.rms_norm_backward(dy, h, w, oa.rms_norm(h, w, 1e-6)[1], dh)
    assert np.abs(dx - differences(lambda v: loss(v, res, w), x)).max() < DIFF_TOL
    assert np.abs(dx - differences(lambda v: loss(x, v, w), res)).max() < DIFF_TOL
    assert np.abs(dw - differences(lambda v: loss(x, res, v), w)).max() < DIFF_TOL


def test_weight_gradient_against_differences():
    r = rng(5)
    x, w, dy = r.normal(size=(6, 5)), r.normal(size=(4, 5)), r.normal(size=(6, 4))
    assert np.abs(oa.weight_grad(dy, x) - differences(lambda v: ((x @ v.T) * dy).sum(), w)).max() < DIFF_TOL


def test_expert_path_against_differences():
    r = rng(6)
    T, K, E, D, M = 5, 2, 3, 4, 3
    idx = np.array([[0, 2], [2, -1], [1, 0], [7, 2], [0, 1]])
    offsets, source, position = oa.expert_sort(idx, E)
    assert offsets.tolist() == [0, 3, 5, 8] and source[8:].tolist() == [-1, -1]
    x, w, dout = r.normal(size=(T, D)), r.normal(size=(T, K)), r.normal(size=(T, M))
    W = r.normal(size=(E, M, D))

    def forward(x_, w_, W_):
        y = np.zeros((T * K, M))
        for e in range(E):
            for row in range(offsets[e], offsets[e + 1]):
                y[row] = W_[e] @ x_[source[row] // K]
        return y

    def loss(x_, w_, W_):
        return (oa.expert_combine(forward(x_, w_, W_), position, w_) * dout).sum()

    y = forward(x, w, W)
    dy, dw = oa.expert_combine_backward(dout, y, position, w, np.zeros_like(y))
    assert np.abs(dw - differences(lambda v: loss(x, v, W), w)).max() < DIFF_TOL
    xs = x[source.clip(0) // K]
    dW = oa.expert_weight_grad(dy, xs, offsets)
    assert np.abs(dW - differences(lambda v: loss(x, w, v), W)).max() < DIFF_TOL
    dxs = np.zeros((T * K, D))
    for e in range(E):
        dxs[offsets[e]:offsets[e + 1]] = dy[offsets[e]:offsets[e + 1]] @ W[e]
    dx = oa.expert_combine(dxs, position, np.ones((T, K)))   # the gather's gradient
    assert np.abs(dx - differences(lambda v: loss(v, w, W), x)).max() < DIFF_TOL
