"""Of several reports the check returns the one that its header names first,
whichever word holds it (the test build, whose waits end after 50 ms)."""
import ctypes

import numpy as np
import pytest

from test_paged_tree_gpu import Case, _dev
from test_paged_tree_timeout import waitlib  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_a_timeout_comes_before_a_bad_page(waitlib):  # noqa: F811
    import torch
    from variable_length_prefill_gb300._binding import ERR_BAD_BLOCK_TABLE, ERR_DEVICE_TIMEOUT
    hq, hkv, d = 8, 2, 128
    c = Case([(300, 1), (40, 1)], hq, hkv, d, "bf16", tree=None, seed=91, behind=0)
    q, k, v = (_dev(x, "bf16") for x in (c.q, c.k, c.v))
    tables, lens, cu = _dev(c.tables), _dev(c.lens), _dev(c.cu)
    bad = torch.full_like(tables, -1)
    out = torch.empty_like(q)
    ws = torch.empty(waitlib.paged_attn_tree_workspace_size(d), dtype=torch.uint8, device="cuda")
    s = ctypes.c_void_p(int(torch.cuda.current_stream().cuda_stream))
    p = lambda *ts: [t.data_ptr() for t in ts]  # noqa: E731
    sizes = (c.tables.shape[1], c.k.shape[0])

    def decode(table):
        assert waitlib.paged_attn_decode(*p(q, k, v, table, lens), 2, hq, hkv, d, 16, *sizes, 0,
                                         out.data_ptr(), s) == 0

    def tree(withheld):
        waitlib.attn_varlen_test_withhold(withheld)
        try:
            assert waitlib.paged_attn_tree(*p(q, k, v, tables, lens, cu), None, 2, 2, hq, hkv, d, 16,
                                           *sizes, 0.0, 0, *p(out, ws), ws.numel(), s) == 0
        finally:
            waitlib.attn_varlen_test_withhold(0)

    decode(tables)
    tree(0)
    assert waitlib.attn_varlen_check(s) == 0
    decode(bad)
    assert waitlib.attn_varlen_check(s) == ERR_BAD_BLOCK_TABLE
    decode(bad)
    tree(1)
    assert waitlib.attn_varlen_check(s) == ERR_DEVICE_TIMEOUT
    decode(tables)
    tree(0)
    assert waitlib.attn_varlen_check(s) == 0
    assert np.isfinite(out.float().cpu().numpy()).all()
