"""An output over the queries is refused by the library itself (no GPU)."""
import pytest

import variable_length_prefill_gb300 as vlp
from variable_length_prefill_gb300 import _binding as B

P, BIG, BYTES = 0x100000, 1 << 40, 4 * 8 * 128 * 2


@pytest.mark.parametrize("shift", [0, 16, BYTES - 16, 16 - BYTES])
def test_out_over_the_queries(shift):
    rc = vlp.load().paged_attn_tree(*(P,) * 7, 1, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, P + shift, P, BIG, None)
    assert rc == B.ERR_INVALID_ARG
