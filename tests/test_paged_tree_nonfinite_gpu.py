"""Values that are not finite, in sequences long enough that a walk over all
positions for each output would outlast the kernel's waits.

Many copies of one sequence share its pages, so that a CTA holds a row tile's
keys whole; the test build's waits end after 50 ms."""
import ctypes

import numpy as np
import pytest

from test_paged_tree_gpu import Case, _bits, _dev, _wide
from test_paged_tree_timeout import waitlib  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

COPIES = 456
BITS = {"bf16": (0x7FC0, 0x7F80, 0xFF80), "fp16": (0x7E00, 0x7C00, 0xFC00)}


def _poison(c, ctx, n, d, where):
    nan, inf, ninf = BITS[c.dtype]

    def put(pos, dim, bits, g=0):
        c.v[c.tables[0, pos // 16], g, dim, pos % 16] = bits

    if "draft" in where:
        put(ctx + n - 1, 3, nan)         # the last draft: seen by itself
        put(ctx, d - 1, inf)             # the first
    if "context" in where:
        put(17, 4, nan)
        put(ctx // 2 + 1, 8, inf)
        put(ctx // 2 + 200, 8, inf)
        put(ctx - 1, d - 2, ninf)
        put(33, d // 2, inf)
        put(ctx - 2, d // 2, ninf)       # both signs: NaN
    if "everywhere" in where:
        for dim in range(d):
            put((dim * 37) % ctx, dim, inf if dim % 3 else ninf)


@pytest.mark.parametrize("where", ["draft", "context", "draft context", "everywhere"])
@pytest.mark.parametrize("ctx,n,hq,hkv,d,dtype", [
    (24000, 3, 2, 1, 256, "bf16"), (30001, 5, 4, 1, 128, "bf16"), (30000, 40, 2, 1, 64, "fp16")])
def test_long_sequences_in_one_piece(waitlib, ctx, n, hq, hkv, d, dtype, where):  # noqa: F811
    import torch
    c = Case([(ctx, n)], hq, hkv, d, dtype, seed=71, behind=0)
    _poison(c, ctx, n, d, where)
    want = c.want()
    q, k, v = (_dev(x, dtype) for x in (np.tile(c.q, (COPIES, 1, 1)), c.k, c.v))
    ints = [_dev(x) for x in (np.tile(c.tables, (COPIES, 1)), np.tile(c.lens, COPIES),
                              np.arange(COPIES + 1, dtype=np.int32) * n, np.tile(c.parents, COPIES))]
    ws = torch.empty(waitlib.paged_attn_tree_workspace_size(d), dtype=torch.uint8, device="cuda")
    s = ctypes.c_void_p(int(torch.cuda.current_stream().cuda_stream))
    out = torch.full_like(q, 7.0)
    assert waitlib.paged_attn_tree(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), *(t.data_ptr() for t in ints), COPIES, COPIES * n,
        hq, hkv, d, 16, c.tables.shape[1], c.k.shape[0], 0.0, 1 if dtype == "fp16" else 0,
        out.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
    assert waitlib.attn_varlen_check(s) == 0
    got = _wide(_bits(out), dtype).reshape(COPIES, n, hq, d)
    assert not np.isfinite(want[0]).all() and (where == "everywhere" or np.isfinite(want[0]).any())
    for i in range(0, COPIES, 41):
        c.compare(got[i], want=want)
    for i in range(1, COPIES):  # the others have the same numbers in another order
        np.testing.assert_array_equal(np.isnan(got[i]), np.isnan(got[0]))
        np.testing.assert_array_equal(np.isinf(got[i]), np.isinf(got[0]))


EDGES = [[(45, 12), (0, 30), (3000, 8)], [(63, 2), (64, 3), (65, 9), (127, 1), (128, 4), (129, 70)],
         [(500, 256), (7, 200)], [(0, 1), (1, 1), (15, 17), (16, 16)]]


@pytest.mark.parametrize("rows", EDGES, ids=range(len(EDGES)))
@pytest.mark.parametrize("hq,hkv,d,dtype", [(4, 2, 64, "bf16"), (8, 1, 128, "fp16"),
                                            (2, 1, 256, "bf16"), (33, 3, 128, "bf16")])
def test_non_finite_values_anywhere(cuda_lib, rows, hq, hkv, d, dtype):
    """One value in forty tokens is not finite, in contexts and drafts, and the
    slots that no row sees are full of them."""
    c = Case(rows, hq, hkv, d, dtype, seed=72)
    rng = np.random.default_rng(73)
    bits = np.asarray(BITS[dtype], dtype=np.uint16)
    seen = np.zeros((c.v.shape[0], 16), dtype=bool)
    for i, size in enumerate(c.lens):
        for p in range(size):
            page, slot = c.tables[i, p // 16], p % 16
            seen[page, slot] = True
            if rng.random() < 1 / 40:
                c.v[page, rng.integers(hkv), rng.integers(d), slot] = rng.choice(bits)
    for page, slot in np.argwhere(~seen):
        c.v[page, :, :, slot] = rng.choice(bits, c.v[page, :, :, slot].shape)
    c.check(cuda_lib)


def test_a_draft_page_that_is_not_there(cuda_lib):
    """Bad ids beside non-finite values: what is there is summed."""
    c = Case([(400, 40), (30, 20)], 8, 2, 128, "bf16", seed=74)
    nan, inf, _ = BITS["bf16"]
    c.v[c.tables[0, 3], :, 5, 2] = inf
    c.v[c.tables[0, 25], :, 6, 4] = inf      # a draft
    c.v[c.tables[1, 0], :, 7, 9] = nan
    c.tables[0, 26], c.tables[0, 7], c.tables[1, 2] = -1, c.k.shape[0], 10 ** 9
    out = c.launch(cuda_lib)
    with pytest.raises(cuda_lib.AttnVarlenError) as e:
        cuda_lib.check()
    assert e.value.code == -11
    c.compare(_wide(_bits(out), "bf16"))
