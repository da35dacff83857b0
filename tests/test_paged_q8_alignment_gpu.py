"""The 8-bit cache in buffers that begin where the header allows and no better: 16 bytes past a 32-byte
boundary, arrays of int32 and float 4 bytes past a 16-byte one."""
import pytest

import paged_q8_ref as ref
from test_paged_q8_gpu import WRITES, batch, dev, new_rows, torch, upload

pytestmark = pytest.mark.gpu


def past(t, by):
    """t in memory that begins `by` bytes past a 256-byte boundary, contiguous as before."""
    raw = torch.empty(t.numel() * t.element_size() + 256, dtype=torch.uint8, device="cuda")
    at = -raw.data_ptr() % 256 + by
    out = raw[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    out.view(torch.uint8).copy_(t.view(torch.uint8))
    assert out.data_ptr() % 256 == by and out.is_contiguous()
    return out


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [0, 3, 6])
@pytest.mark.parametrize("by", [16, 48])
def test_least_alignment(cuda_lib, by, rows, d, kind):
    rng, lens, cu, tables, blocks = batch(WRITES[rows], seed=120 + rows)
    total = int(cu[-1])
    here = upload(ref.new_cache(rng, blocks, 2, d, kind), kind)
    key, value, q = (new_rows(rng, total, h, d, "bf16") for h in (2, 2, 8))
    i = [dev(tables), dev(lens), dev(cu)]
    there = [past(t, by) for t in here[:2]] + [past(t, 4) for t in here[2:]]
    j = [past(t, 4) for t in i]
    cuda_lib.paged_attn_cache_write_q8(key, value, *here, *i)
    cuda_lib.paged_attn_cache_write_q8(past(key, by), past(value, by), *there, *j)
    cuda_lib.check()
    for a, b in zip(here, there):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    pair = past(torch.zeros_like(key), by), past(torch.zeros_like(key), by)
    cuda_lib.paged_attn_cache_read_q8(*there, *j, out=pair)
    for a, b in zip(cuda_lib.paged_attn_cache_read_q8(*here, *i, total), pair):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = past(torch.zeros_like(q), by)
    cuda_lib.paged_attn_q8(past(q, by), *there, *j, out=out)
    assert torch.equal(out, cuda_lib.paged_attn_q8(q, *here, *i))
    cuda_lib.check()
