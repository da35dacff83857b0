"""cu_seqlens whose entries lie at the ends of 32 bits: taken as cut to the packed
rows, so such a sequence is empty or gets the rows that there are."""
import numpy as np
import pytest

import paged_cache_ref as ref
from test_paged_cache_gpu import _bf16, _bits, _raises, _t
from test_paged_tree_gpu import Case, _wide

pytestmark = pytest.mark.gpu

LEAST, MOST = -2 ** 31, 2 ** 31 - 1
CUS = [[5, LEAST, 4, 9], [9, LEAST + 3, 2, MOST], [LEAST, 3, LEAST, 6], [MOST, LEAST, MOST, LEAST],
       [1, MOST, LEAST, MOST], [2, 7, MOST, 12]]


def _clip(cu, total):
    return np.clip(np.asarray(cu, dtype=np.int64), 0, total).astype(np.int32)


@pytest.mark.parametrize("cu", CUS, ids=range(len(CUS)))
def test_tree(cuda_lib, cu):
    c = Case([(40, 4), (50, 5), (33, 3)], 4, 2, 64, seed=81, behind=0)
    c.parents[:] = -1
    cut = _clip(cu, c.total)
    rows = [r for a, b in zip(cut, cut[1:]) for r in range(a, b)]
    if len(rows) > len(set(rows)):
        pytest.skip("slices overlap")
    c.lens[:] = [40, 47, 36]
    c.cu[:] = cut
    want = c.want()
    c.cu[:] = cu
    c.compare(_wide(c.run(cuda_lib), "bf16"), want=want)


@pytest.mark.parametrize("cu", CUS, ids=range(len(CUS)))
def test_write_and_accept(cuda_lib, cu):
    rng = np.random.default_rng(82)
    lens = np.asarray([40, 47, 36], dtype=np.int32)
    tables, blocks = ref.tables_for(rng, lens)
    k, v = ref.new_caches(rng, blocks, 2, 64)
    key = rng.integers(0, 1 << 16, (12, 2, 64), dtype=np.uint16)
    gk, gv, gcu = _bf16(k), _bf16(v), _t(np.asarray(cu, dtype=np.int32))
    cuda_lib.paged_attn_cache_write(_bf16(key), _bf16(key), gk, gv, _t(tables), _t(lens), gcu)
    _raises(cuda_lib)
    assert not ref.write(key, key, k, v, tables, lens, _clip(cu, 12))
    np.testing.assert_array_equal(_bits(gk), k)
    np.testing.assert_array_equal(_bits(gv), v)
    # accept knows no total: a slice that ends at 2^31 - 1 counts all before it
    accepted, num = np.zeros((3, 2), dtype=np.int32), np.zeros(3, dtype=np.int32)
    out = cuda_lib.paged_attn_cache_accept(gk, gv, _t(tables), _t(lens), gcu, _t(accepted), _t(num))
    _raises(cuda_lib)
    new, bad, page = ref.accept(k, v, tables, lens, _clip(cu, MOST), accepted, num)
    assert not bad and not page
    np.testing.assert_array_equal(out.cpu().numpy(), new)
