"""Argument checks of the paged-cache operators, and the reference they are
tested against.  No GPU needed: pointers are fakes that no check dereferences."""
import numpy as np
import pytest

import paged_cache_ref as ref
import variable_length_prefill_gb300 as vlp
from variable_length_prefill_gb300 import _binding as B

P = 0x100000
S8 = (1024, 128, 1024, 128)


@pytest.mark.parametrize("args,code", [
    # (key, value, k, v, tables, lens, cu, S, total, Hkv, D, bs, W, blocks, strides, stream)
    ((P,) * 7 + (-1, 4, 8, 128, 16, 1, 1) + S8 + (None,), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, -4, 8, 128, 16, 1, 1) + S8 + (None,), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 0, 128, 16, 1, 1) + S8 + (None,), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 96, 16, 1, 1) + S8 + (None,), B.ERR_UNSUPPORTED_DIM),
    ((P,) * 7 + (1, 4, 8, 128, 32, 1, 1) + S8 + (None,), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 128, 16, 0, 1) + S8 + (None,), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 128, 16, 1, 0) + S8 + (None,), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 1 << 20, 128, 16, 1, 1) + S8 + (None,), B.ERR_INVALID_ARG),
    ((None,) + (P,) * 6 + (1, 4, 8, 128, 16, 1, 1) + S8 + (None,), B.ERR_INVALID_ARG),
    ((P,) * 6 + (None,) + (1, 4, 8, 128, 16, 1, 1) + S8 + (None,), B.ERR_INVALID_ARG),
    ((P + 8,) + (P,) * 6 + (1, 4, 8, 128, 16, 1, 1) + S8 + (None,), B.ERR_MISALIGNED),
    ((P,) * 3 + (P + 8,) + (P,) * 3 + (1, 4, 8, 128, 16, 1, 1) + S8 + (None,), B.ERR_MISALIGNED),
    ((P,) * 6 + (P + 2,) + (1, 4, 8, 128, 16, 1, 1) + S8 + (None,), B.ERR_MISALIGNED),
    ((P,) * 7 + (1, 4, 8, 128, 16, 1, 1, 1024, 128, 1028, 128, None), B.ERR_MISALIGNED),
    ((P,) * 7 + (1, 4, 8, 128, 16, 1, 1, 1024, -128, 1024, 128, None), B.ERR_INVALID_ARG),
    ((None,) * 7 + (0, 4, 8, 128, 16, 1, 1) + S8 + (None,), B.OK),
    ((None,) * 7 + (3, 0, 8, 128, 16, 1, 1) + S8 + (None,), B.OK),
])
def test_write_arguments(args, code):
    assert vlp.load().paged_attn_cache_write(*args) == code


@pytest.mark.parametrize("args,code", [
    # (k, v, tables, lens, cu, accepted, num, S, A, Hkv, D, bs, W, blocks, out, stream)
    ((P,) * 7 + (-1, 4, 8, 128, 16, 1, 1, P, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 0, 8, 128, 16, 1, 1, P, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 80, 16, 1, 1, P, None), B.ERR_UNSUPPORTED_DIM),
    ((P,) * 7 + (1, 4, 8, 128, 8, 1, 1, P, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 128, 16, 1, 1, None, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 128, 16, 1, 1, P + 1, None), B.ERR_MISALIGNED),
    ((P + 4,) + (P,) * 6 + (1, 4, 8, 128, 16, 1, 1, P, None), B.ERR_MISALIGNED),
    ((None,) * 7 + (0, 4, 8, 128, 16, 1, 1, None, None), B.OK),
])
def test_accept_arguments(args, code):
    assert vlp.load().paged_attn_cache_accept(*args) == code


@pytest.mark.parametrize("args,code", [
    # (tables, lens, refs, rows, n, S, bs, W, blocks, stream)
    ((P,) * 4 + (-1, 2, 16, 1, 1, None), B.ERR_INVALID_ARG),
    ((P,) * 4 + (1, 0, 16, 1, 1, None), B.ERR_INVALID_ARG),
    ((P,) * 4 + (1, 2, 4, 1, 1, None), B.ERR_INVALID_ARG),
    ((P, P, None, P, 1, 2, 16, 1, 1, None), B.ERR_INVALID_ARG),
    ((P, P, P, P + 2, 1, 2, 16, 1, 1, None), B.ERR_MISALIGNED),
    ((None,) * 4 + (0, 2, 16, 1, 1, None), B.OK),
])
def test_free_arguments(args, code):
    assert vlp.load().paged_attn_cache_free(*args) == code


@pytest.mark.parametrize("args,code", [
    # (k, v, tables, lens, refs, src, dst, n, S, Hkv, D, bs, W, blocks, ws, bytes, stream)
    ((P,) * 7 + (-1, 2, 8, 128, 16, 1, 1, P, 1 << 20, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 0, 8, 128, 16, 1, 1, P, 1 << 20, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 2, 8, 128, 16, 1, 1, None, 1 << 20, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 2, 8, 128, 16, 1, 1, P, 4 * 6 - 1, None), B.ERR_WORKSPACE_SMALL),
    ((P,) * 7 + (1, 2, 8, 72, 16, 1, 1, P, 1 << 20, None), B.ERR_UNSUPPORTED_DIM),
    ((None,) * 7 + (0, 2, 8, 128, 16, 1, 1, None, 0, None), B.OK),
])
def test_fork_arguments(args, code):
    assert vlp.load().paged_attn_cache_fork(*args) == code


@pytest.mark.parametrize("args,code", [
    # (k, v, tables, lens, refs, S, Hkv, D, bs, W, blocks, tables_out, refs_out, ws, bytes, stream)
    ((P,) * 5 + (-1, 8, 128, 16, 1, 4, P, P, P, 1 << 20, None), B.ERR_INVALID_ARG),
    ((P,) * 5 + (1, 8, 128, 16, 1, 4, P, None, P, 1 << 20, None), B.ERR_INVALID_ARG),
    ((P,) * 5 + (1, 8, 128, 16, 1, 4, P, P, P, 4 * 14 - 1, None), B.ERR_WORKSPACE_SMALL),
    ((P,) * 5 + (1, 8, 128, 16, 1, 4, P, P, P + 2, 1 << 20, None), B.ERR_MISALIGNED),
    ((None,) * 5 + (0, 8, 128, 16, 1, 4, None, None, None, 0, None), B.OK),
])
def test_compact_arguments(args, code):
    assert vlp.load().paged_attn_cache_compact(*args) == code


def test_workspace_sizes():
    lib = vlp.load()
    assert lib.paged_attn_cache_fork_workspace_size(-1, 4) == 0
    assert lib.paged_attn_cache_fork_workspace_size(3, 5) == 4 * 16
    assert lib.paged_attn_cache_compact_workspace_size(-1) == 0
    assert lib.paged_attn_cache_compact_workspace_size(10) == 4 * 32


def test_binding_refuses_what_does_not_fit():
    """Host tensors, mismatched caches and index arrays, before any launch."""
    torch = pytest.importorskip("torch")
    bf = dict(dtype=torch.bfloat16)
    k, v = torch.zeros((4, 2, 8, 16, 8), **bf), torch.zeros((4, 2, 64, 16), **bf)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        vlp.paged_attn_cache_compact(k, v, i(1, 2), i(1), i(4))
    with pytest.raises(ValueError, match="does not fit"):
        vlp.paged_attn_cache_compact(k, v[:, :1], i(1, 2), i(1), i(4))
    with pytest.raises(ValueError, match="bf16"):
        vlp.paged_attn_cache_fork(k.float(), v.float(), i(1, 2), i(1), i(4), i(1), i(1))
    with pytest.raises(ValueError):
        vlp.paged_attn_cache_free(i(1, 2), i(1), i(4), i(1))


# ------------------------------------------------------- the reference itself
def test_reference_write_is_what_decode_reads():
    """A written token is found where the paged decode's oracle looks for it."""
    import oracle
    from workloads import bf16_bits_to_f64, round_to_bf16_bits
    rng = np.random.default_rng(1)
    lens = np.asarray([37, 5], dtype=np.int32)
    tables, blocks = ref.tables_for(rng, lens, fill=0)
    x = lambda *s: round_to_bf16_bits(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    k, v, key, value, q = (x(blocks, 2, 16, 16, 8), x(blocks, 2, 128, 16), x(42, 2, 128),
                           x(42, 2, 128), x(2, 4, 128))
    ref.write(key, value, k, v, tables, lens, np.asarray([0, 37, 42]))
    got = oracle.paged_decode(q, k, v, tables, lens, "bf16")
    for i, (lo, hi) in enumerate([(0, 37), (37, 42)]):
        for h in range(4):
            s = bf16_bits_to_f64(key[lo:hi, h // 2]) @ bf16_bits_to_f64(q[i, h]) / 128 ** 0.5
            w = np.exp(s - s.max())
            np.testing.assert_allclose(got[i, h], w / w.sum() @ bf16_bits_to_f64(value[lo:hi, h // 2]),
                                       rtol=1e-9, atol=1e-12)


def test_reference_fork_free_compact_closed_forms():
    rng = np.random.default_rng(2)
    k, v = ref.new_caches(rng, 6, 1, 64)
    tables = np.asarray([[4, 2, -1], [-1, -1, -1]], dtype=np.int32)
    lens, refs = np.asarray([20, 0], dtype=np.int32), np.asarray([0, 0, 1, 0, 1, 0], dtype=np.int32)
    assert ref.fork(k, v, tables, lens, refs, [0], [1]) == (False, False)
    assert tables.tolist() == [[4, 2, -1], [4, 0, -1]] and refs.tolist() == [1, 0, 1, 0, 2, 0]
    assert (k[0] == k[2]).all() and lens.tolist() == [20, 20]
    data = [k[4].copy(), v[2].copy()]
    t, r = ref.compact(k, v, tables, lens, refs)
    assert t.tolist() == [[1, 2, -1], [1, 0, -1]] and r.tolist() == [1, 2, 1, 0, 0, 0]
    assert (k[1] == data[0]).all() and (v[2] == data[1]).all()
    assert not ref.free(t, lens, r, [0, 1, 1]) and r.tolist() == [0] * 6
