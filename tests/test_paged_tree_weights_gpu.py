"""Tree attention with weights so small that their 16-bit type hardly holds them."""
import numpy as np
import pytest

import paged_tree_ref as ref
from test_paged_tree_gpu import Case, _bits, _round, _wide

pytestmark = pytest.mark.gpu

LAYOUTS = [(4, 1), (129, 1), (16, 4), (40, 1)]  # rows held four times, once, four times, once


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", LAYOUTS)
@pytest.mark.parametrize("ctx", [30, 100, 700])
def test_small_fp16_weights_count(cuda_lib, d, hq, hkv, ctx):
    """One key with a weight near 1, all others with one of 2^-25.3, which fp16
    does not hold: together they are what the outputs consist of, the strong
    key's value being zero.

    Bound: the weights are held with 2^7 as the unit, in which 2^-25.3 lies above
    fp16's least normal number by 2^-4.3 of it, so each is off by at most 2^-25
    of that unit, 2^-32 (subnormal steps of 2^-24, half a step), a 2^-6.7 part of
    itself; the exponential adds 2^-20 of it at arguments up to 2^5, the sum of at
    most 1000 products in 32 bits 2^-14, the output's rounding 2^-11.
    """
    n = 2
    c = Case([(ctx, n)], hq, hkv, d, "fp16", tree="chain", seed=61)
    c.q[:], c.k[:] = 0, 0
    c.q[:, :, 0] = _round(np.asarray([1.0]), "fp16")[0]
    c.k[c.tables[0, 0], :, 0, 5, 0] = _round(np.asarray([17.546875]), "fp16")[0]
    c.v[:] = _round(1024.0 * (1 + np.random.default_rng(62).random(c.v.shape)), "fp16")
    c.v[c.tables[0, 0], :, :, 5] = 0
    got = _wide(c.run(cuda_lib, scale=1.0), "fp16")
    want = c.want(1.0)[0]
    rows = slice(0, n)
    part = 2.0 ** -6.7 + 2.0 ** -20 + 2.0 ** -14 + 2.0 ** -11
    assert (np.abs(got - want)[rows] <= part * want[rows] + 2.0 ** -25).all(), \
        float((np.abs(got - want)[rows] / want[rows]).max())


def test_bf16_weights_are_not_biased(cuda_lib):
    """bf16 has the exponents of 32 bits: nothing there to hold up."""
    c = Case([(100, 2)], 4, 1, 64, "bf16", tree="chain", seed=65)
    c.q[:], c.k[:] = 0, 0
    c.q[:, :, 0] = _round(np.asarray([1.0]), "bf16")[0]
    c.k[c.tables[0, 0], :, 0, 5, 0] = _round(np.asarray([60.0]), "bf16")[0]
    c.v[c.tables[0, 0], :, :, 5] = 0
    c.check(cuda_lib, scale=1.0)
    assert ref.bound(*c.want(1.0), "bf16", 64)[:2].max() < 1e-20
    assert np.abs(_wide(_bits(c.launch(cuda_lib, scale=1.0)), "bf16")[:2]).max() > 1e-28
