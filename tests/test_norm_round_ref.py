"""CPU tests of the plain rounding (tests/norm_round.py) that the norm's outputs are compared with."""
import numpy as np
import pytest
import torch

import norm_round as nr

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def numbers(n=200000):
    g = np.random.Generator(np.random.PCG64(1))
    v = g.standard_normal(n) * 2.0 ** g.integers(-155, 130, n).astype(np.float64)
    v[::2] = g.standard_normal(n // 2) * 2.0 ** g.integers(-30, 18, n // 2).astype(np.float64)
    v[:6] = [0.0, 65519.99, 65520.0, -65520.0, np.inf, np.nan]
    return v


def test_fp16_and_fp32_as_numpy_converts():
    v = numbers()
    with np.errstate(over="ignore"):
        assert np.array_equal(nr.once(v, "f16"), v.astype(np.float16).astype(np.float64), equal_nan=True)
        assert np.array_equal(nr.once(v, "f32"), v.astype(np.float32).astype(np.float64), equal_nan=True)


def test_bf16_as_torch_converts_32_bit_numbers():
    with np.errstate(over="ignore"):
        f = numbers().astype(np.float32)
    want = torch.from_numpy(f).to(torch.bfloat16).double().numpy()
    assert np.array_equal(nr.once(f.astype(np.float64), "bf16"), want, equal_nan=True)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_numbers_beside_middles_tell_one_rounding_from_two(kind):
    w, y = nr.beside_middles(kind, np.random.Generator(np.random.PCG64(2)), 1000)
    assert np.isfinite(w).all()
    with np.errstate(over="ignore"):
        twice = nr.once(y.astype(np.float32).astype(np.float64), kind)
    assert nr.off(nr.once(y, kind), y, kind) == 0
    assert nr.off(twice, y, kind) > 100
    cut = np.trunc(y / nr.step(y, kind)) * nr.step(y, kind)  # towards zero: about half are wrong
    assert nr.off(cut, y, kind) > len(y) // 4


def test_either_neighbour_only_at_a_middle():
    y = np.array([1 + 2.0 ** -11, 1 + 2.0 ** -11 + 2.0 ** -40, 1 + 2.0 ** -10])
    assert nr.off(np.array([1.0, 1 + 2.0 ** -10, 1 + 2.0 ** -10]), y, "f16") == 0
    assert nr.off(np.array([1 + 2.0 ** -10, 1.0, 1.0]), y, "f16") == 2
    assert nr.off(np.array([np.inf, 65504.0]), np.array([65520.0, 65520.0]), "f16") == 0
    assert nr.off(np.array([np.inf, 65504.0]), np.array([65519.0, 65521.0]), "f16") == 2
