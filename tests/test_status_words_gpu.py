"""Device-side reports against checks that run at the same time."""
import numpy as np
import pytest

import paged_cache_ref as ref
from test_paged_cache_gpu import _bf16, _cu, _t

pytestmark = pytest.mark.gpu


def test_a_report_during_a_check_is_not_lost(cuda_lib):
    """A check finds one report while a kernel on another stream, at a moment
    swept over the time of the check, makes a second, of a kind that comes first
    among several: one of this check and the next has to return it."""
    import torch
    rng = np.random.default_rng(53)
    lens = np.asarray([20], dtype=np.int32)
    tables, blocks = ref.tables_for(rng, lens)
    k, v = ref.new_caches(rng, blocks, 1, 64)
    key = rng.integers(0, 1 << 16, (1, 1, 64), dtype=np.uint16)
    gk, gv, gkey, gt, gl = _bf16(k), _bf16(v), _bf16(key), _t(tables), _t(lens)
    bad, cu, refs, row = _t(np.full_like(tables, -1)), _t(_cu([1])), _t(np.ones(blocks, np.int32)), \
        _t(np.asarray([7], np.int32))
    side = torch.cuda.Stream()

    def report():
        try:
            cuda_lib.check()
        except cuda_lib.AttnVarlenError as e:
            return e.code
        return 0

    report()
    torch.cuda.synchronize()
    lost = []
    for i in range(600):
        cuda_lib.paged_attn_cache_free(gt, gl, refs, row)  # a row that is not there: -14
        with torch.cuda.stream(side):
            torch.cuda._sleep(1 + 500 * i)
        cuda_lib.paged_attn_cache_write(gkey, gkey, gk, gv, bad, gl, cu, stream=side)  # -11
        first = report()
        side.synchronize()
        second = report()
        assert first in (-14, -11) and second in (0, -11, -14)
        if -11 not in (first, second):
            lost.append(i)
    assert not lost, f"{len(lost)} reports lost, at steps {lost[:20]}"
