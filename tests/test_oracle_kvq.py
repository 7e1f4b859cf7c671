"""Pins of the quantised-cache oracle (oracle/kvq.py) against hand-derived
values and the properties of the affine format, and of its attention against
PyTorch's float64 scaled dot-product attention."""
import numpy as np
import pytest
import torch

from helpers import bits as raw
from oracle import kvq


def _bf16(a):
    return raw(torch.as_tensor(np.asarray(a, np.float32)).to(torch.bfloat16))


def test_bf16_round_matches_torch():
    x = np.random.default_rng(1).standard_normal(20000).astype(np.float32) * np.float32(10.0) ** np.random.default_rng(2).integers(-30, 30, 20000)
    np.testing.assert_array_equal(kvq.bf16_round(x), _bf16(x))


def test_codes_of_a_ramp():
    # 0..63: scale bf16(63 / 15) = 4.1875, bias 0; code = rint(x / 4.1875), at most 15
    c, sb = kvq.quantise(_bf16(np.arange(64.0)), 4)
    assert kvq.bf16_value(sb)[0].tolist() == [4.1875, 0.0]
    want = np.minimum(np.rint(np.arange(64) / 4.1875), 15)
    np.testing.assert_array_equal(c[0], want)
    # 8 bits: scale bf16(63 / 255) = 0.2470703125
    c, sb = kvq.quantise(_bf16(np.arange(64.0)), 8)
    assert kvq.bf16_value(sb)[0, 0] == np.float32(0.2470703125)
    np.testing.assert_array_equal(c[0], np.minimum(np.rint(np.arange(64) / 0.2470703125), 255))


def test_nibble_order_and_round_trip():
    codes = np.arange(64, dtype=np.uint8) % 16
    q = kvq.pack(codes, 4)
    assert q[0] == 0x10 and q[1] == 0x32 and q[7] == 0xFE  # even channel low
    np.testing.assert_array_equal(kvq.unpack(q, 4), codes)


def test_equal_values_are_kept_exactly():
    x = _bf16(np.full(64, -3.25))
    for b in (4, 8):
        c, sb = kvq.quantise(x, b)
        assert (c == 0).all() and kvq.bf16_value(sb)[0].tolist() == [0.0, -3.25]
        np.testing.assert_array_equal(kvq.values(kvq.pack(c, b), sb, b), np.full(64, -3.25))


@pytest.mark.parametrize("bits", [4, 8])
def test_error_is_within_half_a_step(bits):
    # the scale is rounded by at most 2^-8 of itself, so the largest code's value is off
    # by L 2^-8 scale at most where the range was rounded down (the code is clamped)
    x = _bf16(np.random.default_rng(3).standard_normal((50, 256)))
    c, sb = kvq.quantise(x, bits)
    s = np.repeat(kvq.bf16_value(sb)[..., 0].astype(np.float64), 64, -1).reshape(50, 256)
    err = np.abs(kvq.values(kvq.pack(c, bits), sb, bits) - kvq.bf16_value(x).astype(np.float64))
    L = 2 ** bits - 1
    assert (err <= s * (0.5 + max(0.0, L * 2.0 ** -8 - 0.5)) * (1 + 1e-6)).all()


def test_extreme_ranges_stay_finite():
    big = np.zeros(64, np.float32)
    big[0], big[1] = 3.0e38, -3.0e38
    c, sb = kvq.quantise(_bf16(big), 4)
    assert np.isfinite(kvq.bf16_value(sb)).all() and c[0, 0] == 15 and c[0, 1] == 0
    # a range whose step is below the smallest normal number: codes 0, the bias alone
    tiny = np.zeros(64, np.float32)
    tiny[5] = 2.0 ** -126
    c, sb = kvq.quantise(_bf16(tiny), 8)
    assert (c == 0).all() and (sb == 0).all()


def test_attention_matches_torch_float64():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((5, 8, 64)), rng.standard_normal((40, 2, 64)), rng.standard_normal((40, 2, 64))
    got = kvq.attend(q, k, v, np.full(5, 40))
    Q = torch.from_numpy(q).transpose(0, 1)
    K, V = (torch.from_numpy(np.repeat(x, 4, 1)).transpose(0, 1) for x in (k, v))
    ref = torch.nn.functional.scaled_dot_product_attention(Q, K, V).transpose(0, 1).numpy()
    np.testing.assert_allclose(got, ref, rtol=1e-11, atol=1e-12)
    # limits: no token gives zeros, one token gives its value row
    got = kvq.attend(q, k, v, np.array([0, 1, 2, 39, 40]))
    assert (got[0] == 0).all()
    np.testing.assert_array_equal(got[1, 5], v[0, 1])
    ref = torch.nn.functional.scaled_dot_product_attention(Q[:, 3:4], K[:, :39], V[:, :39])[:, 0].numpy()
    np.testing.assert_allclose(got[3], ref, rtol=1e-11, atol=1e-12)
