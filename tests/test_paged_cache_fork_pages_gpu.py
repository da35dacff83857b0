"""Forks of rows whose tables hold ids that are no pages."""
import numpy as np
import pytest

from test_paged_cache_gpu import _bf16, _bits, _pool, _raises, _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-5, 10 ** 6])
@pytest.mark.parametrize("n", [3, 37])
def test_a_bad_last_page_is_copied_as_an_id(cuda_lib, bad, n):
    """The copy of a row whose partial page is none has none either: no page of
    the pool, with what some other row left in it, takes its place."""
    rng = np.random.default_rng(57)
    k, v, tables, lens, refs = _pool(rng, 5, [n, 20], 6)
    last = n // 16
    refs[tables[0, last]] = 0
    tables[0, last] = bad
    dev = [_bf16(k), _bf16(v), _t(tables), _t(lens), _t(refs)]
    cuda_lib.paged_attn_cache_fork(*dev, _t(np.asarray([0, 1], np.int32)), _t(np.asarray([2, 3], np.int32)))
    _raises(cuda_lib, -11)
    fresh = int(np.flatnonzero(refs <= 0)[0])  # for row 1's partial page alone
    tables[2, :last + 1] = tables[0, :last + 1]
    tables[3, 0], tables[3, 1] = tables[1, 0], fresh
    refs[tables[0, :last]] += 1
    refs[tables[1, 0]] += 1
    refs[fresh] = 1
    lens[2:4] = n, 20
    k[fresh], v[fresh] = k[tables[1, 1]], v[tables[1, 1]]
    for got, want in zip(dev[2:], (tables, lens, refs)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    np.testing.assert_array_equal(_bits(dev[0]), k)
    np.testing.assert_array_equal(_bits(dev[1]), v)
