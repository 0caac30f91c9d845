"""Pins of the fp64 oracle of the training-step operators: central differences, torch's double
arithmetic and brute force (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import train as ot


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 8, 16])
def test_qk_norm_rope_backward_against_central_differences(interleaved, rot):
    rng = np.random.default_rng(1 + rot)
    x = rng.standard_normal((2, 3, 2, 16))
    gamma = 1 + 0.3 * rng.standard_normal(16)
    dy = rng.standard_normal(x.shape)
    pos = np.array([[0, 5, 9], [1000, 3, 7]])
    freq = 100.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    f = lambda x, gamma: float((dy * ot.qk_norm_rope(x, gamma, pos, freq, 1e-3,
                                                     interleaved)).sum())
    dx, dg = ot.qk_norm_rope_backward(x, gamma, pos, freq, 1e-3, interleaved, dy)
    # central differences of step h: truncation h^2 f''' / 6, rounding 2^-53 |f| / h
    h = 1e-5
    for at in [(0, 0, 0, 0), (1, 2, 1, 15), (0, 1, 1, 7), (1, 0, 0, 8)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, gamma) - f(x - e, gamma)) / (2 * h) - dx[at]) <= 1e-8
    for j in (0, 7, 8, 15):
        e = np.zeros(16)
        e[j] = h
        assert abs((f(x, gamma + e) - f(x, gamma - e)) / (2 * h) - dg[j]) <= 1e-8


def test_rotation_keeps_pair_lengths_and_turns_back():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 4, 3, 32))
    pos = np.array([[0, 1, 77, 123456]])
    freq = 10000.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        y = ot.rotate(x, pos, freq, inter)
        assert np.array_equal(y[..., 16:], x[..., 16:])
        assert np.allclose(y[:, 0], x[:, 0], rtol=0, atol=1e-15)
        assert np.abs(ot.rotate(y, pos, freq, inter, back=True) - x).max() <= 1e-14
    # one pair by hand: position 1, frequency 1
    y = ot.rotate(x, pos, freq, True)
    assert np.allclose(y[0, 1, 0, 0], x[0, 1, 0, 0] * np.cos(1) - x[0, 1, 0, 1] * np.sin(1))


def test_adamw_against_torch_in_double():
    rng = np.random.default_rng(5)
    w = torch.tensor(rng.standard_normal(50), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([w], lr=0.01, betas=(0.8, 0.96), eps=1e-10, weight_decay=0.1)
    wo, m, v = w.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 5):
        g = rng.standard_normal(50)
        w.grad = torch.from_numpy(g)
        opt.step()
        wo, m, v = ot.adamw(wo, g, m, v, t, 0.01, 0.8, 0.96, 1e-10, 0.1)
    assert np.abs(w.detach().numpy() - wo).max() <= 1e-13


def test_e4m3_codes_against_torch():
    assert len(ot.E4M3_VALUES) == 127 and ot.E4M3_VALUES[-1] == 448
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ot.E4M3_VALUES)
    rng = np.random.default_rng(6)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.uniform(-5, 2.6, 4000),
                        (ot.E4M3_VALUES[1:] + ot.E4M3_VALUES[:-1]) / 2, [0.0, 448.0, -448.0]])
    x = np.clip(x.astype(np.float32), -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ot.encode_e4m3(x), want)


def test_block_scales_and_norm():
    x = np.zeros(600)
    x[3], x[300], x[599] = -4.48, 1e-40, 0.5
    s = ot.block_scales(x)
    assert s.shape == (3,) and np.allclose(s, [0.01, 0.0, 0.5 / 448])
    assert np.allclose(ot.dequantize_blocks(np.ones(600), s)[[0, 255, 256, 512]],
                       [0.01, 0.01, 0.0, 0.5 / 448])
    norm, factor = ot.grad_norm([np.full(9, 2.0), np.array([8.0])], 1.0)
    assert norm == 10.0 and abs(factor - 1 / (10 + 1e-6)) <= 1e-15
    assert ot.grad_norm([np.ones(1)], 5.0)[1] == 1.0


def test_scale_as_a_product_is_one_unit_from_the_quotient():
    """The 8-bit format's scale, amax times 1/448 rounded to fp32: 1/448 is off by 0.75 2^-24 of
    itself, at most 0.75 units of the product's last place, which rounding turns into one at most."""
    rng = np.random.default_rng(9)
    x = (rng.random(1 << 20) + 1).astype(np.float32)
    c = np.float32(1 / 448)
    assert abs(float(c) * 448 - 1) <= 0.751 * 2.0 ** -24
    product, quotient = x * c, x / np.float32(448)
    apart = np.abs(product.view(np.int32) - quotient.view(np.int32))
    assert apart.max() == 1
