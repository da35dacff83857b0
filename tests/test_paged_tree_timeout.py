"""The bounded waits of the tree attention kernel giving up, run on purpose.

As for the attention kernel (test_wait_timeout.py): the test build waits 50 ms
and can withhold the first keys of the first row tile, which are then neither
copied nor announced.  The wait for them runs out, every role of the CTA stops, the call
returns, the check reports ATTN_VARLEN_ERR_DEVICE_TIMEOUT once, and the next
call is right."""
import ctypes
import time

import numpy as np
import pytest

from test_paged_tree_gpu import Case, _bits, _dev, _wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def waitlib(cuda_lib):
    from variable_length_prefill_gb300 import _binding
    lib = ctypes.CDLL(cuda_lib.build(variant="testhooks"))
    for name, (res, args) in _binding.SYMBOLS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    lib.attn_varlen_test_withhold.argtypes = [ctypes.c_int]
    lib.attn_varlen_test_withhold.restype = None
    yield lib
    lib.attn_varlen_test_withhold(0)


CASES = [
    ([(300, 5), (40, 2)], 8, 2, 128, "bf16"),     # one tile or two a CTA
    ([(6000, 12)] * 6, 16, 8, 128, "bf16"),       # many tiles, several segments
    ([(3000, 40)] * 6, 8, 2, 256, "fp16"),
    ([(900, 3)] * 60, 8, 8, 64, "bf16"),
]


@pytest.mark.parametrize("rows,hq,hkv,d,dtype", CASES, ids=range(len(CASES)))
def test_wait_runs_out_and_is_reported(waitlib, rows, hq, hkv, d, dtype):
    import torch
    from variable_length_prefill_gb300._binding import ERR_DEVICE_TIMEOUT
    c = Case(rows, hq, hkv, d, dtype, seed=50)
    q, k, v = (_dev(x, dtype) for x in (c.q, c.k, c.v))
    ints = [_dev(x) for x in (c.tables, c.lens, c.cu, c.parents)]
    ws = torch.empty(waitlib.paged_attn_tree_workspace_size(d), dtype=torch.uint8, device="cuda")
    s = ctypes.c_void_p(int(torch.cuda.current_stream().cuda_stream))

    def run():
        out = torch.full_like(q, 7.0)
        assert waitlib.paged_attn_tree(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), *(t.data_ptr() for t in ints), len(c.lens),
            c.total, hq, hkv, d, 16, c.tables.shape[1], c.k.shape[0], 0.0,
            1 if dtype == "fp16" else 0, out.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
        return out

    want = run()
    assert waitlib.attn_varlen_check(s) == 0
    waitlib.attn_varlen_test_withhold(1)
    try:
        t0 = time.perf_counter()
        run()
        assert waitlib.attn_varlen_check(s) == ERR_DEVICE_TIMEOUT
        assert time.perf_counter() - t0 < 1.0
    finally:
        waitlib.attn_varlen_test_withhold(0)
    assert waitlib.attn_varlen_check(s) == 0
    again = run()
    assert waitlib.attn_varlen_check(s) == 0
    np.testing.assert_array_equal(_bits(again), _bits(want))
    assert np.isfinite(_wide(_bits(again), dtype)).all()
