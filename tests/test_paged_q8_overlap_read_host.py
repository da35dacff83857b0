"""Keys and values of the 8-bit cache read into rows that both would write: refused before anything runs."""
import pytest

import variable_length_prefill_gb300 as vlp
from variable_length_prefill_gb300 import _binding as B

# fake addresses, 16-byte aligned and far apart; never dereferenced
KC, VC, KS, VS, TABLES, LENS, CU, KEY = (0x10000000 * (i + 1) for i in range(8))


def _read(by, st, total=4, hkv=8, d=128):
    """Values `by` elements behind the keys."""
    return vlp.load().paged_attn_cache_read_q8(KC, VC, KS, VS, TABLES, LENS, CU, 1, total, hkv, d, 16, 1, 5, 0, 0, KEY,
                                               KEY + 2 * by, *st, *st, None)


@pytest.mark.parametrize("by,st,args", [
    (0, (1024, 128), {}), (128, (1024, 128), {}), (2048 + 128 * 7, (1024, 128), {}), (-1024, (1024, 128), {}),
    (120, (2048, 128), {}), (1016, (2048, 128), {}), (2048 * 3 - 8, (2048, 128), {}),  # halves of a fused row, a little off
    (2040, (256, 1024), dict(total=4, hkv=8)), (-8, (64, 256), dict(d=64)),
    (8, (0, 128), dict(total=1)), (120, (512, 0), dict(hkv=1)), (512, (512, 0), dict(hkv=1)),
])
def test_read_refuses_rows_that_keys_and_values_share(by, st, args):
    assert _read(by, st, **args) == B.ERR_INVALID_ARG


def test_read_refuses_one_buffer_under_two_layouts():
    assert vlp.load().paged_attn_cache_read_q8(KC, VC, KS, VS, TABLES, LENS, CU, 1, 4, 8, 128, 16, 1, 5, 0, 0, KEY, KEY,
                                               1024, 128, 128, 512, None) == B.ERR_INVALID_ARG
