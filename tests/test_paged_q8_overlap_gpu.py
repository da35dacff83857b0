"""Buffers of the 8-bit cache that lie side by side are not taken for overlapping ones."""
import numpy as np
import pytest

import paged_q8_ref as ref
from test_paged_q8_gpu import batch, codes, dev, new_rows, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("swap", [False, True])
def test_write_to_halves_of_one_buffer(cuda_lib, swap):
    rng, lens, cu, tables, blocks = batch([(3, 30), (0, 16)], seed=130)
    cache = ref.new_cache(rng, blocks, 2, 64, "e4m3")
    both = codes(np.stack([cache[0].reshape(blocks, -1), cache[1].reshape(blocks, -1)]), "e4m3")
    scales = dev(np.stack(cache[2:]))
    a, b = (1, 0) if swap else (0, 1)
    kv = new_rows(rng, 46, 2, 64, "bf16")
    mine = both[a].view(cache[0].shape), both[b].view(cache[1].shape), scales[a], scales[b]
    apart = [t.clone() for t in mine]
    i = dev(tables), dev(lens), dev(cu)
    cuda_lib.paged_attn_cache_write_q8(kv, -kv, *mine, *i)
    cuda_lib.paged_attn_cache_write_q8(kv, -kv, *apart, *i)
    cuda_lib.check()
    for x, y in zip(mine, apart):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
