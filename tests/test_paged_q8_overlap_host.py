"""Buffers of the 8-bit cache that share memory where two of them are written: refused before anything runs."""
import pytest

import variable_length_prefill_gb300 as vlp
from variable_length_prefill_gb300 import _binding as B

# fake addresses, 16-byte aligned and far apart; never dereferenced
KEY, VALUE, KC, VC, KS, VS, TABLES, LENS, CU = (0x10000000 * (i + 1) for i in range(9))
NB, HKV, D = 5, 8, 128
ST = (1024, 128, 1024, 128)


def _write(kc=KC, vc=VC, ks=KS, vs=VS):
    return vlp.load().paged_attn_cache_write_q8(KEY, VALUE, kc, vc, ks, vs, TABLES, LENS, CU, 1, 4, HKV, D, 16, 1, NB, 0,
                                                0, *ST, None)


@pytest.mark.parametrize("by", [0, 4, 4 * NB * HKV - 4])
def test_write_refuses_scales_that_share_memory(by):
    assert _write(vs=KS + by) == B.ERR_INVALID_ARG
    assert _write(ks=VS + by) == B.ERR_INVALID_ARG


@pytest.mark.parametrize("by", [0, 16, NB * HKV * D * 16 - 16])
def test_write_refuses_caches_that_share_memory(by):
    assert _write(vc=KC + by) == B.ERR_INVALID_ARG
    assert _write(kc=VC + by) == B.ERR_INVALID_ARG
