"""The bar on errors ahead of the last rounding tells fp32's accuracy from one more rounding to bf16: the down product
and the combine on the CPU, with the mistakes planted in the model."""
import numpy as np
import torch

from rounding import BAR, excess, half_step


def bf(v):
    return torch.from_numpy(np.asarray(v, np.float32)).bfloat16().double().numpy()


def model(seed, T=12, H=512, F=384, k=4):
    rng = np.random.default_rng(seed)
    a, b = rng.standard_normal((2, T, k, F))
    h = (0.25 * a / (1 + np.exp(-a)) * b).astype(np.float32).astype(np.float64)
    w = rng.standard_normal((k, F, H)) / F ** 0.5
    return h, w


def pairs(h, w):
    return np.matmul(h.transpose(1, 0, 2), w).transpose(1, 0, 2)     # [T, k, H]


def rows8(h, w):
    """The pairs' products of h's 8-bit rows."""
    D = np.abs(h).max(-1, keepdims=True)
    return pairs(np.rint(127 * h / D) * (D / 127), w)


def test_half_step():
    v = np.array([1.0, 1.9921875, 2.0, -3.0, 0.75, 2.0 ** -100])
    assert (half_step(v) == np.array([2.0 ** -8, 2.0 ** -8, 2.0 ** -7, 2.0 ** -7, 2.0 ** -9, 2.0 ** -108])).all()
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 1000)) * 3
    assert (excess(bf(x), x) == 0).all()


def test_the_low_part_of_h_counts():
    h, w = model(1)
    w = bf(w)
    ref = pairs(h, w).sum(1)
    hi = bf(h)
    lo = bf(h - hi)
    assert excess(bf(pairs(hi + lo, w).sum(1)), ref).max() < BAR / 5
    assert excess(bf(pairs(hi, w).sum(1)), ref).min() > 5 * BAR


def test_the_8_bit_layer_with_fewer_bits():
    """A pair's output rounded before the sum, and h rounded before its rows are quantised, fail in every token."""
    h, w = model(2)
    ref = rows8(h, w)
    y = ref.sum(1)
    assert excess(bf(ref.astype(np.float32).astype(np.float64).sum(1)), y).max() < BAR / 5
    assert excess(bf(bf(ref).sum(1)), y).min() > 5 * BAR
    assert excess(bf(rows8(bf(h), w).sum(1)), y).min() > 5 * BAR
