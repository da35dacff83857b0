"""What the paged-cache operators report of calls that go wrong, and that no
report is lost on its way to the check."""
import numpy as np
import pytest

import paged_cache_ref as ref
from test_paged_cache_gpu import _bf16, _bits, _cu, _raises, _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [
    # (length, new tokens) of each sequence; tables of 4 pages, 64 places
    [(65, 1)], [(68, 4)], [(300, 17)], [(2 ** 31 - 1, 1)],
    [(30, 2), (65, 1)], [(70, 3), (64, 9)], [(10, 1)] * 300 + [(65, 1)],
], ids=range(7))
def test_write_wholly_past_the_table(cuda_lib, rows):
    """A sequence none of whose new tokens has a place is reported like one
    whose last tokens have none: the decode step behind a full table."""
    rng = np.random.default_rng(51)
    lens = np.asarray([n for n, _ in rows], dtype=np.int32)
    cu = _cu([n for _, n in rows])
    tables, blocks = ref.tables_for(rng, np.minimum(lens, 64), width=4)
    k, v = ref.new_caches(rng, blocks, 2, 64)
    key = rng.integers(0, 1 << 16, (int(cu[-1]), 2, 64), dtype=np.uint16)
    gk, gv = _bf16(k), _bf16(v)
    cuda_lib.paged_attn_cache_write(_bf16(key), _bf16(key), gk, gv, _t(tables), _t(lens), _t(cu))
    _raises(cuda_lib, -11)
    assert ref.write(key, key, k, v, tables, lens, cu)
    np.testing.assert_array_equal(_bits(gk), k)
    np.testing.assert_array_equal(_bits(gv), v)


def test_write_without_new_tokens_reports_nothing(cuda_lib):
    """A length past the table is the write's business only where it has tokens to place."""
    rng = np.random.default_rng(52)
    lens = np.asarray([20, 90], dtype=np.int32)
    cu = _cu([3, 0])
    tables, blocks = ref.tables_for(rng, np.minimum(lens, 64), width=4)
    k, v = ref.new_caches(rng, blocks, 2, 64)
    key = rng.integers(0, 1 << 16, (3, 2, 64), dtype=np.uint16)
    gk, gv = _bf16(k), _bf16(v)
    cuda_lib.paged_attn_cache_write(_bf16(key), _bf16(key), gk, gv, _t(tables), _t(lens), _t(cu))
    _raises(cuda_lib)
    assert not ref.write(key, key, k, v, tables, lens, cu)
    np.testing.assert_array_equal(_bits(gk), k)
