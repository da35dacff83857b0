"""Scales below 32 bits' normal numbers, which the C call takes (the binding's
begin at 2^-126): all weights are equal, and rows that see nothing are zero."""
import ctypes

import pytest

from test_paged_tree_gpu import Case, _bits, _dev, _wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
@pytest.mark.parametrize("scale", [2.0 ** -149, 1e-40, 2.0 ** -127])
def test_subnormal_scale(cuda_lib, d, dtype, scale):
    import torch
    hq, hkv = 4, 2
    c = Case([(10, 8), (300, 2), (20, 5)], hq, hkv, d, dtype, seed=66)
    c.lens[0] = 5  # fewer tokens than drafts: rows that see nothing
    q, k, v = (_dev(x, dtype) for x in (c.q, c.k, c.v))
    ints = [_dev(x) for x in (c.tables, c.lens, c.cu, c.parents)]
    lib = cuda_lib.load()
    ws = torch.empty(lib.paged_attn_tree_workspace_size(d), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0)
    s = ctypes.c_void_p(int(torch.cuda.current_stream().cuda_stream))
    assert lib.paged_attn_tree(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), *(t.data_ptr() for t in ints), 3, c.total, hq, hkv,
        d, 16, c.tables.shape[1], c.k.shape[0], scale, 1 if dtype == "fp16" else 0, out.data_ptr(),
        ws.data_ptr(), ws.numel(), s) == 0
    cuda_lib.check()
    got = _wide(_bits(out), dtype)
    c.compare(got, want=c.want(scale))
    assert (got[:2] == 0).all()
