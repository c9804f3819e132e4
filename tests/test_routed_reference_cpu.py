"""The plain form of the row quantisation, and that its test rows tell a division from a product with a reciprocal."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import routed_reference as ref

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_even(dtype):
    for row in ref.tie_rows(dtype):
        assert np.array_equal(torch.from_numpy(row).to(dtype).double().numpy(), row)
        q, scale = ref.quantize(row[None])
        want = [round(Fraction(127) * Fraction(v) / Fraction(row[0])) for v in row]     # exact, ties to even
        assert q[0].tolist() == want
        assert scale[0] == np.float32(row[0]) / np.float32(127)


@pytest.mark.parametrize("exponent", [-149, -140, -126, -1, 0, 60, 126])
def test_the_range_of_float32(exponent):
    """Subnormal and largest maxima: powers of two times the same integers quantise to the same."""
    base = np.array([[1.0, 0.5, -0.5, 0.25, 0.0, -1.0]]) if exponent > -148 else np.array([[1.0, 0, 0, 1, -1, 1]])
    row = np.ldexp(base, exponent).astype(np.float32).astype(np.float64)
    assert np.array_equal(ref.quantize(row)[0], ref.quantize(base)[0])
    assert not ref.quantize(0 * row)[0].any()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_a_reciprocal_alone_would_be_noticed(dtype):
    wrong = 0
    for row in ref.tie_rows(dtype):
        x = row.astype(np.float32)
        near = np.rint(x * (np.float32(127) / x[0])).astype(np.int8)
        wrong += int((near != ref.quantize(row[None])[0][0]).sum())
    assert wrong > 0                               # one is enough for a test of equality


def test_a_reciprocal_alone_would_be_noticed_in_random_rows():
    """bfloat16 has ties only where the reciprocal is exact; its random rows come close enough to others."""
    x = torch.from_numpy(np.random.default_rng(0).standard_normal((600, 1032)).astype(np.float32)).bfloat16()
    x = x.float().numpy()
    near = np.rint(x * (np.float32(127) / np.abs(x).max(1, keepdims=True))).astype(np.int8)
    assert int((near != ref.quantize(x.astype(np.float64))[0]).sum()) > 0
