"""Pins of the oracle for the 8-bit cache and windowed attention: closed forms,
library routines and brute force (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import attention as oattn, bf16 as obf, cache8 as o8, window as owin


def test_e4m3_magnitudes_are_the_formats():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o8.e4m3_magnitudes(), t)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_bf16_value_rounds_as_the_library_does(fmt):
    """Vectors of one loud value that fixes E = 0, and every finite bf16 up to it."""
    bits = np.arange(0x7F80, dtype=np.uint16)
    keep = obf.to_f64(bits) <= o8.LIMIT[fmt]
    b = np.concatenate([bits[keep], bits[keep] | 0x8000, obf.from_f64(o8.LIMIT[fmt])]).astype(np.uint16)
    codes, E = o8.quantise(b[None], fmt)
    assert E.tolist() == [0]
    y = torch.from_numpy(obf.to_f64(b).astype(np.float32))
    ref = y.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else torch.round(y).to(torch.int8).view(torch.uint8)
    assert np.array_equal(codes[0], ref.numpy())


@pytest.mark.parametrize("fmt,amax,E", [
    ("e4m3", 448.0, 0), ("e4m3", 450.0, 1), ("e4m3", 449.0, 1), ("e4m3", 1.0, -8), ("e4m3", 1.75, -8), ("e4m3", 2.0, -7),
    ("e4m3", 0.0, -100), ("e4m3", 2.0 ** -120, -100), ("e4m3", 3.3895313892515355e38, 119),
    ("int8", 127.0, 0), ("int8", 127.5, 1), ("int8", 128.0, 1), ("int8", 1.0, -6), ("int8", 0.9921875, -7), ("int8", 0.99609375, -6),
    ("int8", 0.0, -100), ("int8", 3.3895313892515355e38, 121), ("e4m3", np.inf, -128), ("int8", np.nan, -128)])
def test_exponents(fmt, amax, E):
    x = np.array([[0.0, -amax, 0.0]])
    assert o8.exponent(x, fmt).tolist() == [E]
    codes, e = o8.quantise(obf.from_f64(x), fmt)
    v = o8.values(codes, e, fmt)
    if E == -128:
        assert np.isnan(v).all() and not codes.any()
    else:
        assert np.isfinite(obf.to_f64(obf.from_f64(v))).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_held_values_are_bf16_numbers_within_half_a_step(fmt):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(300, 64)) * np.exp(rng.normal(size=(300, 1)) * 20)
    b = obf.from_f64(x)
    x = obf.to_f64(b)
    codes, E = o8.quantise(b, fmt)
    v = o8.values(codes, E, fmt)
    assert np.array_equal(obf.to_f64(obf.from_f64(v)), v)
    scale = 2.0 ** E.astype(float)[:, None]
    half = 0.5 * scale if fmt == "int8" else np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale)
    assert (np.abs(v - x) <= half).all()
    again, E2 = o8.quantise(obf.from_f64(v), fmt)
    assert np.array_equal(o8.values(again, E2, fmt), v)


def test_visible_keys():
    assert owin.visible(9, 12, 0, 0).tolist() == [True] * 10 + [False] * 2
    assert np.nonzero(owin.visible(9, 12, 3, 0))[0].tolist() == [7, 8, 9]
    assert np.nonzero(owin.visible(9, 12, 3, 2))[0].tolist() == [0, 1, 7, 8, 9]
    assert np.nonzero(owin.visible(9, 12, 1, 0))[0].tolist() == [9]
    assert np.nonzero(owin.visible(2, 12, 3, 9))[0].tolist() == [0, 1, 2]
    assert np.nonzero(owin.visible(9, 12, 3, 8))[0].tolist() == list(range(10))


def test_a_window_that_covers_everything_is_plain_attention():
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(size=(4, 64)), rng.normal(size=(30, 2, 64)), rng.normal(size=(30, 2, 64))
    qb, kb, vb = obf.from_f64(q[None]), obf.from_f64(k[None]), obf.from_f64(v[None])
    q, k, v = obf.to_f64(qb)[0], obf.to_f64(kb)[0], obf.to_f64(vb)[0]
    for n in (1, 7, 30):
        ref = obf.to_f64(oattn.decode(qb, kb, vb, [n]))[0]
        for window, sinks in ((0, 0), (n, 0), (100, 3), (1, n)):
            assert np.array_equal(obf.to_f64(obf.from_f64(owin.row(q, k, v, n - 1, window, sinks))), ref)
    assert not owin.row(q, k, v, -1, 4, 1).any()
    assert np.allclose(owin.row(q, k, v, 20, 1, 0), np.repeat(v[20], 2, axis=0))
