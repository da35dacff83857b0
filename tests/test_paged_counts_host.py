"""Counts of rows, sequences and forks that the kernels' 32-bit loops could not
step over are refused (no GPU: pointers are fakes that no check dereferences)."""
import pytest

import variable_length_prefill_gb300 as vlp
from variable_length_prefill_gb300 import _binding as B

P, BIG = 0x100000, 1 << 40
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("n", [(1 << 30) + 1, MOST - 1000, MOST])
def test_too_many(n):
    lib = vlp.load()
    write = (*(P,) * 7, n, 4, 8, 128, 16, 1, 1, 1024, 128, 1024, 128, None)
    assert lib.paged_attn_cache_write(*write) == B.ERR_INVALID_ARG
    assert lib.paged_attn_cache_fork(*(P,) * 7, 1, n, 8, 128, 16, 1, 1, P, BIG, None) == B.ERR_INVALID_ARG
    assert lib.paged_attn_cache_fork(*(P,) * 7, n, 2, 8, 128, 16, 1, 1, P, BIG, None) == B.ERR_INVALID_ARG
    tree = (*(P,) * 7, n, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, P, 2 * P, BIG, None)
    assert lib.paged_attn_tree(*tree) == B.ERR_INVALID_ARG
