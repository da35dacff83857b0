"""Argument checks of the tree attention and pins of its reference (no GPU)."""
import numpy as np
import pytest

import paged_cache_ref as cref
import paged_tree_ref as ref
import variable_length_prefill_gb300 as vlp
from variable_length_prefill_gb300 import _binding as B

P = 0x100000
BIG = 1 << 40


@pytest.mark.parametrize("args,code", [
    # (q, k, v, tables, lens, cu, parents, S, total, Hq, Hkv, D, bs, W, blocks, scale, dtype, out,
    #  ws, bytes, stream)
    ((P,) * 7 + (-1, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, -4, 8, 2, 128, 16, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 3, 128, 16, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 0, 128, 16, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 2, 72, 16, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_UNSUPPORTED_DIM),
    ((P,) * 7 + (1, 4, 8, 2, 128, 32, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 2, 128, 16, 1, 1, 0.0, 2, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 2, 128, 16, 1, 1, float("nan"), 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 1 << 30, 8, 2, 128, 16, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 2, 128, 16, 1 << 27, 1, 0.0, 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 2, 128, 16, 1, 1, float("inf"), 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 2, 128, 16, 1, 1, 2.0 ** 127, 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, None, P, BIG, None), B.ERR_INVALID_ARG),
    ((P,) * 7 + (1, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, P, None, BIG, None), B.ERR_INVALID_ARG),
    ((None,) + (P,) * 6 + (1, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_INVALID_ARG),
    ((P + 8,) + (P,) * 6 + (1, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_MISALIGNED),
    ((P,) * 6 + (P + 2,) + (1, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, P, P, BIG, None), B.ERR_MISALIGNED),
    ((P,) * 7 + (1, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, P, P + 8, BIG, None), B.ERR_MISALIGNED),
    ((P,) * 7 + (1, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, P, P, 15, None), B.ERR_WORKSPACE_SMALL),
    ((None,) * 7 + (0, 4, 8, 2, 128, 16, 1, 1, 0.0, 0, None, None, 0, None), B.OK),
    ((None,) * 7 + (3, 0, 8, 2, 128, 16, 1, 1, 0.0, 0, None, None, 0, None), B.OK),
])
def test_arguments(args, code):
    assert vlp.load().paged_attn_tree(*args) == code


def test_workspace_size():
    lib = vlp.load()
    assert lib.paged_attn_tree_workspace_size(96) == 0
    assert all(lib.paged_attn_tree_workspace_size(d) >= 16 for d in (64, 128, 256))


def _setup(rows, seed=0, hq=4, hkv=2, d=64):
    rng = np.random.default_rng(seed)
    lens = np.asarray([c + n for c, n in rows], dtype=np.int32)
    cu = np.concatenate([[0], np.cumsum([n for _, n in rows])]).astype(np.int32)
    tables, blocks = cref.tables_for(rng, lens, fill=0)
    q = rng.standard_normal((int(cu[-1]), hq, d))
    k, v = rng.standard_normal((blocks, hkv, d // 8, 16, 8)), rng.standard_normal((blocks, hkv, d, 16))
    return q, k, v, tables, lens, cu


def _dense(k, v, tables, i, n):
    pos = np.arange(n)
    key = k[tables[i, pos // 16], :, :, pos % 16, :].reshape(n, k.shape[1], -1)
    return key, v[tables[i, pos // 16], :, :, pos % 16]


def test_reference_chain_is_causal_attention():
    torch = pytest.importorskip("torch")
    q, k, v, tables, lens, cu = _setup([(20, 7), (0, 5), (33, 1)])
    out = ref.tree(q, k, v, tables, lens, cu, None)[0]
    for i in range(3):
        key, val = _dense(k, v, tables, i, lens[i])
        n = cu[i + 1] - cu[i]
        mask = torch.ones(n, int(lens[i]), dtype=torch.bool).tril(int(lens[i]) - int(n))
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).transpose(0, 1)  # noqa: E731
        want = torch.nn.functional.scaled_dot_product_attention(
            t(q[cu[i]:cu[i + 1]]), t(key).repeat_interleave(2, 0), t(val).repeat_interleave(2, 0),
            attn_mask=mask)
        np.testing.assert_allclose(out[cu[i]:cu[i + 1]], want.transpose(0, 1).numpy(), rtol=1e-10,
                                   atol=1e-12)


def test_reference_branch_is_its_path_alone():
    """A leaf's row equals the chain of its path, the other drafts taken out."""
    q, k, v, tables, lens, cu = _setup([(20, 6)], seed=1)
    parents = np.asarray([-1, 0, 0, 1, 2, 4], dtype=np.int32)
    out = ref.tree(q, k, v, tables, lens, cu, parents)[0]
    path = [0, 2, 4, 5]
    key, val = _dense(k, v, tables, 0, 26)
    pos = list(range(20)) + [20 + j for j in path]
    for h in range(4):
        s = key[pos, h // 2] @ q[5, h] / 8.0
        w = np.exp(s - s.max())
        np.testing.assert_allclose(out[5, h], (w / w.sum()) @ val[pos, h // 2], rtol=1e-10, atol=1e-13)


def test_reference_closed_forms():
    q, k, v, tables, lens, cu = _setup([(0, 3), (9, 2)], seed=2)
    parents = np.asarray([-1, -1, 0, -1, 0], dtype=np.int32)
    out = ref.tree(q, k, v, tables, lens, cu, parents)[0]
    _, val = _dense(k, v, tables, 0, 3)
    np.testing.assert_allclose(out[0], val[0].repeat(2, 0))  # a root without context: its own value
    np.testing.assert_allclose(out[1], val[1].repeat(2, 0))
    out = ref.tree(0 * q, k, v, tables, lens, cu, parents)[0]
    _, val = _dense(k, v, tables, 1, 11)
    np.testing.assert_allclose(out[4], val.mean(0).repeat(2, 0), atol=1e-12)
    np.testing.assert_allclose(out[3], val[:10].mean(0).repeat(2, 0), atol=1e-12)


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    k = torch.zeros((4, 2, 8, 16, 8), dtype=torch.bfloat16)
    v = torch.zeros((4, 2, 64, 16), dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        vlp.paged_attn_tree(torch.zeros((3, 4, 64), dtype=torch.bfloat16), k, v, i(1, 2), i(1), i(2))
