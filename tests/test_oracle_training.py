"""The float64 definitions of the FP8 training operators against independent facts: torch's casts, closed
forms and central differences (CPU)."""
import numpy as np
import pytest
import torch

from oracle import training as O

CAST = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_codes_against_torch(fmt):
    every = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(every).view(CAST[fmt]).double().numpy()
    np.testing.assert_array_equal(O.decode_fp8(every, fmt), want)
    fin = np.unique(want[np.isfinite(want)])
    mid = (fin[1:] + fin[:-1]) / 2                     # ties
    v = np.concatenate([fin, mid, np.nextafter(mid, np.inf), np.nextafter(mid, -np.inf),
                        np.random.default_rng(0).normal(size=4000) * 10.0 ** np.random.default_rng(1).uniform(-8, 3, 4000)])
    v = v.astype(np.float32)                           # torch rounds once from fp32
    v = np.clip(v, -O.FORMATS[fmt][2], O.FORMATS[fmt][2])
    got = O.decode_fp8(O.encode_fp8(v.astype(np.float64), fmt), fmt)
    np.testing.assert_array_equal(got, torch.from_numpy(v).to(CAST[fmt]).double().numpy())
    assert O.decode_fp8(O.encode_fp8(np.array([1e30, -1e30]), fmt), fmt).tolist() == [O.FORMATS[fmt][2], -O.FORMATS[fmt][2]]


@pytest.mark.parametrize("top", [448.0, 57344.0])
def test_scale_exponent_is_the_smallest(top):
    rng = np.random.default_rng(2)
    for a in list(10.0 ** rng.uniform(-37, 37, 500)) + [top * 2.0 ** q for q in range(-100, 100, 7)] + [2.0 ** -149]:
        p = O.scale_exp(float(a), top)
        assert a <= top * 2.0 ** p and (p == -126 or a > top * 2.0 ** (p - 1))
    assert O.scale_exp(0.0, top) == 0


def test_product_of_blocks_in_closed_form():
    # one value per block: out = sum over blocks of 128 * sa * sb (the last block is short)
    a, b = np.ones((3, 300)), np.ones((2, 300))
    sa = np.array([[1, 2, 4], [1, 1, 1], [0, 0, 8]], float)
    sb = np.array([[1, 1, 1], [2, 0, 1]], float)
    out, mag = O.gemm(a, sa, b, sb)
    want = np.array([[128 + 256 + 4 * 44, 256 + 4 * 44], [300, 256 + 44], [8 * 44, 8 * 44]], float)
    np.testing.assert_array_equal(out, want)
    np.testing.assert_array_equal(mag, want)
    np.testing.assert_array_equal(O.dequant(np.ones((130, 1)), np.array([[2.0], [3.0]]))[:, 0], [2.0] * 128 + [3.0] * 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_loss_of_even_and_collapsed_routing(score):
    E, k = 8, 2
    l = np.zeros((16, E))
    even = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(16)])
    assert O.balance_loss(l, even, coef=0.5, score=score)[0] == pytest.approx(0.5)
    l[:, :2] = 60.0 if score == "softmax" else 0.0
    if score == "sigmoid":
        l[:, 2:] = -800.0
    assert O.balance_loss(l, np.tile([0, 1], (16, 1)), score=score)[0] == pytest.approx(E / k)
    assert O.balance_loss(np.full((4, E), -np.inf), np.zeros((4, k), int), score=score)[0] == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("packed", [False, True])
def test_balance_gradient_against_differences(score, packed):
    rng = np.random.default_rng(3)
    T, E, k = 11, 5, 2
    l = rng.normal(size=(T, E))
    ids = np.argsort(-l, 1)[:, :k]
    kw = {"coef": 0.3, "score": score}
    if packed:
        kw |= {"offsets": [1, 4, 4, 9], "mask": rng.random(T) > 0.3}
    grad, _ = O.balance_grad(1.7, l, ids, **kw)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = l.copy(), l.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = 1.7 * (O.balance_loss(up, ids, **kw)[0] - O.balance_loss(dn, ids, **kw)[0]) / (2 * h)
            assert abs(d - grad[t, e]) < 1e-8


def test_linear_layer_gradients_against_differences():
    # the three products of a linear layer: dx = dy W and dW = dy^T x, by differences of sum(dy * x W^T)
    rng = np.random.default_rng(4)
    x, w, dy = rng.normal(size=(3, 5)), rng.normal(size=(4, 5)), rng.normal(size=(3, 4))
    one = lambda r: np.ones((r, 1))   # noqa: E731
    dx = O.gemm(dy, one(3), w.T, one(5))[0]
    dw = O.gemm(dy.T, one(4), x.T, one(5))[0]
    f = lambda: float((dy * O.gemm(x, one(3), w, one(4))[0]).sum())   # noqa: E731
    for arr, g in ((x, dx), (w, dw)):
        for i in np.ndindex(arr.shape):
            v = arr[i]
            arr[i] = v + 1e-6
            up = f()
            arr[i] = v - 1e-6
            d = (up - f()) / 2e-6
            arr[i] = v
            assert abs(d - g[i]) < 1e-8
