"""Attention over the 8-bit cache where scores are so large that their last bit is a factor of many powers of two."""
import numpy as np
import pytest

import paged_q8_ref as ref
from paged_q8_winners import check_winners, winners
from test_paged_q8_gpu import HALF, LEAST, TYPES, batch, dev, torch, upload, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("width", [33, 700])
@pytest.mark.parametrize("scale", [2.0 ** 17 / 3, 2.0 ** 23 / 3, 2.0 ** 31 / 3, 2.0 ** 60 / 3])
def test_large_scores(cuda_lib, scale, width, kind, dtype):
    rng, lens, cu, tables, blocks = batch([(40, 1), (500, 1), (290, 3)], seed=95, width=width)
    cache = ref.new_cache(rng, blocks, 2, 128, kind, -7, -6)
    q = dev(rng.standard_normal((5, 8, 128)), TYPES[dtype])
    got = cuda_lib.paged_attn_q8(q, *upload(cache, kind), dev(tables), dev(lens), dev(cu), scale)
    cuda_lib.check()
    want, decided = winners(wide(q), cache, tables, lens, cu, kind, scale)
    assert decided.mean() > 0.5
    check_winners(wide(got), want, decided, HALF[dtype], LEAST[dtype])


@pytest.mark.parametrize("exponent", [-149, -60, 100])
def test_large_scores_beside_pages_of_other_value_scales(cuda_lib, exponent):
    """The keys that come close have values of another size than the key that wins."""
    rng, lens, cu, tables, blocks = batch([(600, 2)], seed=96)
    cache = k, v, ks, vs = ref.new_cache(rng, blocks, 1, 128, "int8", -7, -6)
    q = dev(rng.standard_normal((2, 4, 128)), torch.bfloat16)
    i = dev(tables), dev(lens), dev(cu)
    scale = 2.0 ** 33 / 3
    want, _ = winners(wide(q), cache, tables, lens, cu, "int8", scale)
    won = {tuple(row) for row in want.reshape(-1, 128)}
    for b in range(blocks):  # pages without a winner
        if not any(tuple(x * vs[b, 0]) in won for x in ref.decode(v[b, 0], "int8").T):
            vs[b] = 2.0 ** exponent
    want, decided = winners(wide(q), cache, tables, lens, cu, "int8", scale)
    assert decided.mean() > 0.5
    got = cuda_lib.paged_attn_q8(q, *upload(cache, "int8"), *i, scale)
    cuda_lib.check()
    check_winners(wide(got), want, decided, HALF["bf16"], LEAST["bf16"])
