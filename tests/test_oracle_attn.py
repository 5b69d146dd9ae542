"""Pins of the attention layer's fp64 definitions (oracle/attn.py), on the CPU."""
import numpy as np
import pytest
import torch

import oracle.attn as oa


def test_e4m3_codes_agree_with_torch():
    x = torch.randn(20000, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    x = (x * torch.pow(2.0, torch.randint(-12, 8, x.shape).double())).clamp(-448, 448).float()
    ties = torch.tensor([2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 0.0, -0.0, 448.0, -448.0, 2.0 ** -9])
    x = torch.cat([x, ties])
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oa.e4m3_code(x.double().numpy()), want)
    assert np.array_equal(oa.e4m3_value(want), torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


def test_row_scales_are_the_smallest_powers_of_two():
    for amax in (448.0, 448.0000001, 1.0, 7.0, 7.03125, 2.0 ** -130, 0.0, 3e38):
        code, byte = oa.quantise_row(np.array([amax, -amax / 3, 0.0]))
        e = byte - 127
        assert oa.EXP_MIN <= e <= oa.EXP_MAX
        if 448 * 2.0 ** oa.EXP_MIN < amax <= 448 * 2.0 ** oa.EXP_MAX:
            assert 448 * 2.0 ** (e - 1) < amax <= 448 * 2.0 ** e
        v = oa.row_value(code, byte)
        if amax <= 448 * 2.0 ** oa.EXP_MAX:  # half a step of e4m3, 2^-10 of the scale below its normal range
            assert np.all(np.abs(v - [amax, -amax / 3, 0.0]) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** (e - 10)))
        # every value is a normal bf16 number
        b = torch.from_numpy(v).to(torch.bfloat16).double().numpy()
        assert np.array_equal(b, v)
    for bad in (np.nan, np.inf, -np.inf):
        code, byte = oa.quantise_row(np.array([1.0, bad]))
        assert byte == 255 and not code.any() and np.isnan(oa.row_value(code, byte)).all()


def test_attention_of_one_key_and_of_equal_keys():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((3, 1, 8)), rng.standard_normal((3, 1, 8))
    q = rng.standard_normal((3, 2, 8))
    o, lse, _, _ = oa.attention(q, k, v, 0.3)
    assert np.allclose(o[0], v[0], atol=1e-15) and np.allclose(lse[0], (q[0] @ k[0, 0]) * 0.3, atol=1e-14)
    k[:] = k[0]
    o, _, _, _ = oa.attention(q, k, v, 0.3)
    assert np.allclose(o[2], v[:, 0].mean(0), atol=1e-15)
    o, _, _, _ = oa.attention(q, k, v, 0.3, window=2)
    assert np.allclose(o[2], v[1:, 0].mean(0), atol=1e-15) and np.allclose(o[0], v[0], atol=1e-15)


@pytest.mark.parametrize("with_residual_grad", [False, True])
def test_norm_gradients_agree_with_differences(with_residual_grad):
    rng = np.random.default_rng(3)
    R, d, eps = 3, 8, 1e-5
    x, r, w = rng.standard_normal((R, d)), rng.standard_normal((R, d)), rng.standard_normal(d)
    dy, ds = rng.standard_normal((R, d)), rng.standard_normal((R, d)) * with_residual_grad

    def loss(x, r, w):
        s, _, y = oa.add_rmsnorm(x, r, w, eps)
        return np.sum(dy * y) + np.sum(ds * s)

    s, rstd, _ = oa.add_rmsnorm(x, r, w, eps)
    dx, dw = oa.add_rmsnorm_grads(dy, s, w, rstd, ds)
    h = 1e-6
    for a, grad in ((x, dx), (r, dx), (w, dw)):
        num = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = loss(x, r, w)
            a[i] = keep - h
            num[i] = (up - loss(x, r, w)) / (2 * h)
            a[i] = keep
        # central differences: third derivative times h^2 / 6, and 2^-53 |loss| / h
        assert np.max(np.abs(num - grad)) < 1e-7
