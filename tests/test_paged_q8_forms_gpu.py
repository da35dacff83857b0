"""One long context among short ones behind a wide table is not one warp's alone."""
import numpy as np
import pytest

from test_paged_q8_gpu import dev, torch

pytestmark = pytest.mark.gpu


def shortest_us(f):
    f()
    times = []
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(3):
            f()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) / 3 * 1e3)
    return min(times)


@pytest.mark.parametrize("hq,hkv,seqs", [(32, 8, 152), (16, 16, 76), (16, 4, 304)])
def test_a_long_context_among_short_ones(cuda_lib, seqs, hq, hkv):
    """As many pairs as there are computing warps, and a few more: about the same work, so about the same time (where
    one warp had the long context alone the first took 37 times as long)."""
    d, pages = 128, 4096
    took = []
    for n in (seqs, seqs + 2):
        lens = np.asarray([16 * pages] + [100] * (n - 1), dtype=np.int32)
        tables = np.zeros((n, pages), dtype=np.int32)
        tables[0] = np.random.default_rng(1).permutation(pages)
        tables[1:, :7] = pages + np.arange(7)  # a prefix that all the others share
        k = torch.zeros((pages + 7, hkv, d // 16, 16, 16), dtype=torch.int8, device="cuda").random_(-60, 60)
        v = torch.zeros((pages + 7, hkv, d, 16), dtype=torch.int8, device="cuda").random_(-60, 60)
        scale = torch.full((pages + 7, hkv), 2.0 ** -6, device="cuda")
        q = torch.randn((n, hq, d), device="cuda").bfloat16()
        t, size = dev(tables), dev(lens)
        took.append(shortest_us(lambda: cuda_lib.paged_attn_q8(q, k, v, scale, scale, t, size)))
    cuda_lib.check()
    assert took[0] < 4 * took[1] + 50
