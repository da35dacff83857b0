"""Attention over the 8-bit cache where a query, a softmax scale or a key scale is very large or small, and another
makes up for it."""
import numpy as np
import pytest

import paged_q8_ref as ref
from paged_q8_winners import check_winners, winners
from test_paged_q8_gpu import HALF, LEAST, TYPES, batch, check_attn, dev, torch, upload, wide

pytestmark = pytest.mark.gpu

ROWS = [(40, 1), (333, 2), (3, 9), (0, 1)]


def inputs(kind, width, d=128, hq=8, hkv=2, seed=97, low=-9, high=-5):
    rng, lens, cu, tables, blocks = batch(ROWS, seed=seed, width=width)
    return rng, lens, cu, tables, ref.new_cache(rng, blocks, hkv, d, kind, low, high), rng.standard_normal((13, hq, d))


# powers of two of the queries, the softmax scale and the key scales, which make up for each other
POWERS = [(80, 0, -80), (75, 0, -84), (0, 97, -100), (0, 60, -60), (50, -100, 50), (60, -126, 66), (-100, -20, 120),
          (-100, 0, 100), (0, -110, 110), (-120, 120, 0), (120, -120, 0), (100, 40, -140), (-60, -60, 120), (-66, -66, 132), (0, 0, 0)]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("width", [23, 300])
@pytest.mark.parametrize("powers", POWERS, ids=str)
def test_factors_that_make_up_for_each_other(cuda_lib, powers, width, kind):
    of_q, of_scale, of_key = powers
    rng, lens, cu, tables, cache, q = inputs(kind, width)
    cache[2][:] = cache[2].astype(np.float64) * 2.0 ** of_key
    scale = max(2.0 ** of_scale / 11, 2.0 ** -126)
    check_attn(cuda_lib, q * 2.0 ** of_q, cache, tables, lens, cu, kind, "bf16", scale)
    if of_q == 0:
        check_attn(cuda_lib, q, cache, tables, lens, cu, kind, "fp16", scale)


@pytest.mark.parametrize("d,hq,hkv", [(64, 6, 2), (256, 4, 1), (128, 3, 3), (128, 24, 1)])
def test_rows_and_pages_of_all_sizes_in_one_tile(cuda_lib, d, hq, hkv):
    """Query heads 2^90 apart, on pages whose keys are small, zero, or large for the small rows alone."""
    rng, lens, cu, tables, cache, q = inputs("e4m3", 40, d, hq, hkv)
    q[:, ::2] *= 2.0 ** 90
    cache[2][:] *= np.float32(2.0 ** -90)
    cache[2][rng.random(cache[2].shape) < 0.1] = 0
    check_attn(cuda_lib, q, cache, tables, lens, cu, "e4m3", "bf16")
    q[:, ::2] = 0
    cache[2][:] *= np.float32(2.0 ** 90)
    check_attn(cuda_lib, q, cache, tables, lens, cu, "e4m3", "bf16")
    q[:, 1::2] *= 2.0 ** -90
    cache[2][:] *= np.float32(2.0 ** 90)
    check_attn(cuda_lib, q, cache, tables, lens, cu, "e4m3", "bf16")


@pytest.mark.parametrize("scale,low,high", [(1.0, 100, 112), (2.0 ** 126 / 3, -40, -35), (2.0 ** 40, 60, 72), (1e-30, 127, 115)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("width", [23, 300])
def test_pages_whose_large_scales_differ(cuda_lib, width, dtype, scale, low, high):
    """Scores near the largest 32-bit numbers, from pages whose key scales are powers of two apart."""
    rng, lens, cu, tables, cache, q = inputs("int8", width)
    cache[2][:] = np.where(rng.random(cache[2].shape) < 0.5, 2.0 ** low, 2.0 ** high)
    cache[0][:] = rng.integers(0, 20, cache[0].shape)  # scores below 2^126
    q = dev(q, TYPES[dtype])
    got = cuda_lib.paged_attn_q8(q, *upload(cache, "int8"), dev(tables), dev(lens), dev(cu), scale)
    cuda_lib.check()
    want, decided = winners(wide(q), cache, tables, lens, cu, "int8", scale)
    assert decided.mean() > 0.4
    check_winners(wide(got), want, decided, HALF[dtype], LEAST[dtype])


@pytest.mark.parametrize("of_q,of_scale,of_key", [(0, 126, 30), (0, 126, -7), (100, 100, 100), (126, 126, 126), (0, 120, 120),
                                                  (126, 126, -140), (20, 97, -20)])
@pytest.mark.parametrize("width", [23, 300])
def test_scores_past_32_bits(cuda_lib, width, of_q, of_scale, of_key):
    """Scores that no 32-bit number holds: the largest has all the weight, among pages of all scales."""
    rng, lens, cu, tables, cache, q = inputs("int8", width)
    cache[2][:] = np.exp2(of_key + rng.integers(-5, 2, cache[2].shape))
    q = dev(np.clip(q, -1.9, 1.9) * 2.0 ** of_q, torch.bfloat16)
    got = cuda_lib.paged_attn_q8(q, *upload(cache, "int8"), dev(tables), dev(lens), dev(cu), 2.0 ** of_scale)
    cuda_lib.check()
    want, decided = winners(wide(q), cache, tables, lens, cu, "int8", 2.0 ** of_scale, fold=2.0 ** -18)
    assert decided.mean() > 0.9
    check_winners(wide(got), want, decided, HALF["bf16"], LEAST["bf16"])


def test_equal_scores_past_32_bits_share_the_weight(cuda_lib):
    """Contexts of one key, repeated, and rows that see nothing but scores below all numbers."""
    rng, lens, cu, tables, cache, q = inputs("int8", 23)
    k, v, ks, vs = cache
    k[:], v[:] = 3, rng.integers(1, 60, (1, 2, 128, 1))
    ks[:], vs[:] = 2.0 ** 120, 0.25
    for sign in (1.0, -1.0):
        x = dev(np.abs(q) * sign, torch.bfloat16)
        got = wide(cuda_lib.paged_attn_q8(x, *upload(cache, "int8"), dev(tables), dev(lens), dev(cu), 2.0 ** 126))
        want = np.repeat(v[0].astype(np.float64)[:, :, 0], 4, axis=0) * 0.25
        # equal weights are powers of two; their sum and the quotient are off by 32-bit steps, which the values'
        # six bits, held in eight, round away
        assert (got == want[None]).all()
    cuda_lib.check()


@pytest.mark.parametrize("of_q,of_scale,low,high", [(29, 29, 45, 60), (24, 19, 36, 70), (0, 29, 45, 90), (29, 0, 45, 100),
                                                    (24, 20, 35, 37), (30, 29, 46, 47), (-30, 29, 46, 126)])
@pytest.mark.parametrize("width", [23, 300])
def test_pages_on_both_sides_of_large(cuda_lib, width, of_q, of_scale, low, high):
    """Pages of key scales that are just not large beside such that are, under rows and softmax scales of both kinds."""
    rng, lens, cu, tables, cache, q = inputs("int8", width)
    cache[2][:] = np.where(rng.random(cache[2].shape) < 0.5, 2.0 ** low, 2.0 ** high)
    q = dev(np.clip(q, -1.9, 1.9) * 2.0 ** of_q, torch.bfloat16)
    got = cuda_lib.paged_attn_q8(q, *upload(cache, "int8"), dev(tables), dev(lens), dev(cu), 2.0 ** of_scale)
    cuda_lib.check()
    want, decided = winners(wide(q), cache, tables, lens, cu, "int8", 2.0 ** of_scale, fold=2.0 ** -18)
    assert decided.mean() > 0.9
    check_winners(wide(got), want, decided, HALF["bf16"], LEAST["bf16"])
