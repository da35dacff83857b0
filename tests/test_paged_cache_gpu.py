"""The paged-cache operators on the GPU against the token-by-token reference,
bit for bit: every byte of the caches, tables, lengths and counts, so that
what a call must leave alone is compared as well."""
import numpy as np
import pytest

import paged_cache_ref as ref

pytestmark = pytest.mark.gpu

PAGE = ref.PAGE


def _t(a):
    import torch
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def _bf16(a):
    import torch
    return _t(a).view(torch.bfloat16)


def _bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _raises(vlp, *codes):
    """The check call reports one of the codes (none: it is silent)."""
    if not codes:
        vlp.check()
        return
    with pytest.raises(vlp.AttnVarlenError) as e:
        vlp.check()
    assert e.value.code in codes
    vlp.check()  # reported once


def _cu(counts, start=0):
    return (start + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)


# ---------------------------------------------------------------------- write
WRITE = [
    # (context, new) of each sequence; heads; head size; packed start
    ([(0, 1)], 1, 64, 0),
    ([(15, 1), (16, 1), (31, 2), (0, 0), (7, 1)], 3, 128, 0),
    ([(0, 16), (0, 32), (5, 11), (5, 27), (5, 28), (16, 16)], 8, 128, 3),
    ([(0, 333)], 16, 128, 0),
    ([(9, 100), (0, 0), (0, 47)], 4, 256, 2),
    ([(i % 40, (i * 7) % 37) for i in range(300)], 5, 64, 0),
    ([(3, 40)] * 3, 20, 128, 0),
    ([(100, 1)] * 700, 2, 128, 0),
    ([(3, 9000), (0, 1), (40, 17)], 2, 64, 0),  # one far longer than the others
    ([(i % 20, 1) for i in range(3000)], 3, 64, 0),
]


@pytest.mark.parametrize("rows,hkv,d,start", WRITE, ids=range(len(WRITE)))
@pytest.mark.parametrize("fused", [False, True])
def test_write(cuda_lib, rows, hkv, d, start, fused):
    rng = np.random.default_rng(11)
    lens = np.asarray([c + n for c, n in rows], dtype=np.int32)
    cu = _cu([n for _, n in rows], start)
    tables, blocks = ref.tables_for(rng, lens)
    k, v = ref.new_caches(rng, blocks, hkv, d)
    total = int(cu[-1]) + 4  # rows behind the last sequence
    kv = rng.integers(0, 1 << 16, (total, 2 * hkv + 3, d), dtype=np.uint16)
    key, value = kv[:, 1:1 + hkv], kv[:, 2 + hkv:2 + 2 * hkv]
    if fused:  # strided views of one projection
        t = _bf16(kv)
        tk, tv = t[:, 1:1 + hkv], t[:, 2 + hkv:2 + 2 * hkv]
    else:
        tk, tv = _bf16(key), _bf16(value)
    gk, gv = _bf16(k), _bf16(v)
    cuda_lib.paged_attn_cache_write(tk, tv, gk, gv, _t(tables), _t(lens), _t(cu))
    _raises(cuda_lib)
    assert not ref.write(key, value, k, v, tables, lens, cu)
    np.testing.assert_array_equal(_bits(gk), k)
    np.testing.assert_array_equal(_bits(gv), v)


def test_write_single_token_and_head_with_any_stride(cuda_lib):
    """The stride of a dimension of one says nothing about the layout."""
    rng = np.random.default_rng(14)
    lens = np.asarray([21], dtype=np.int32)
    tables, blocks = ref.tables_for(rng, lens)
    k, v = ref.new_caches(rng, blocks, 1, 64)
    x = rng.integers(0, 1 << 16, (1, 1, 64), dtype=np.uint16)
    t = _bf16(x).as_strided((1, 1, 64), (3, 5, 1))
    gk, gv = _bf16(k), _bf16(v)
    cuda_lib.paged_attn_cache_write(t, t, gk, gv, _t(tables), _t(lens), _t(_cu([1])))
    _raises(cuda_lib)
    assert not ref.write(x, x, k, v, tables, lens, _cu([1]))
    np.testing.assert_array_equal(_bits(gk), k)
    np.testing.assert_array_equal(_bits(gv), v)


def test_write_odd_calls(cuda_lib):
    """Slices that step backwards, lengths below the new tokens or negative,
    offsets past the packed rows: what has a place is written, no more."""
    rng = np.random.default_rng(12)
    cu = np.asarray([4, 10, 6, 9, 30, 29], dtype=np.int32)
    lens = np.asarray([20, 40, 2, 33, 17], dtype=np.int32)
    tables, blocks = ref.tables_for(rng, lens, width=3)
    k, v = ref.new_caches(rng, blocks, 2, 64)
    key = rng.integers(0, 1 << 16, (26, 2, 64), dtype=np.uint16)
    value = rng.integers(0, 1 << 16, (26, 2, 64), dtype=np.uint16)
    gk, gv = _bf16(k), _bf16(v)
    cuda_lib.paged_attn_cache_write(_bf16(key), _bf16(value), gk, gv, _t(tables), _t(lens), _t(cu))
    _raises(cuda_lib)
    assert not ref.write(key, value, k, v, tables, lens, cu)
    np.testing.assert_array_equal(_bits(gk), k)
    np.testing.assert_array_equal(_bits(gv), v)
    lens[:] = [-3, 0, -2 ** 31, 1, 0]
    cuda_lib.paged_attn_cache_write(_bf16(key), _bf16(value), gk, gv, _t(tables), _t(lens), _t(cu))
    _raises(cuda_lib)
    ref.write(key, value, k, v, tables, lens, cu)
    np.testing.assert_array_equal(_bits(gk), k)


def test_write_bad_pages(cuda_lib):
    """Bad page ids, and positions past the table, are skipped and reported."""
    rng = np.random.default_rng(13)
    lens = np.asarray([50, 70, 20], dtype=np.int32)
    cu = _cu([50, 50, 20])
    tables, blocks = ref.tables_for(rng, [50, 64, 20], width=4)
    tables[0, 1], tables[2, 0] = blocks, -1
    k, v = ref.new_caches(rng, blocks, 3, 128)
    key = rng.integers(0, 1 << 16, (120, 3, 128), dtype=np.uint16)
    gk, gv = _bf16(k), _bf16(v)
    cuda_lib.paged_attn_cache_write(_bf16(key), _bf16(key), gk, gv, _t(tables), _t(lens), _t(cu))
    _raises(cuda_lib, -11)
    assert ref.write(key, key, k, v, tables, lens, cu)
    np.testing.assert_array_equal(_bits(gk), k)
    np.testing.assert_array_equal(_bits(gv), v)


# --------------------------------------------------------------------- accept
def _accept_case(rng, counts, take_most, fill=99):
    n = len(counts)
    accepted = np.full((n, take_most), fill, dtype=np.int32)
    num = np.zeros(n, dtype=np.int32)
    for i, c in enumerate(counts):
        num[i] = rng.integers(0, min(c, take_most) + 1)
        accepted[i, :num[i]] = np.sort(rng.choice(c, num[i], replace=False)) if c else []
    return accepted, num


@pytest.mark.parametrize("hkv,d,counts,take", [
    (1, 64, [1, 0, 5], 1), (8, 128, [8] * 4, 4), (3, 128, [64, 1, 17, 33, 0, 40], 12),
    (5, 256, [30, 2], 30), (2, 64, [300, 256], 290), (4, 128, [7] * 260, 7)])
def test_accept(cuda_lib, hkv, d, counts, take):
    rng = np.random.default_rng(21)
    ctx = [int(rng.integers(0, 90)) for _ in counts]
    ctx[0] = 0
    lens = np.asarray([a + b for a, b in zip(ctx, counts)], dtype=np.int32)
    tables, blocks = ref.tables_for(rng, lens)
    accepted, num = _accept_case(rng, counts, take)
    k, v = ref.new_caches(rng, blocks, hkv, d)
    gk, gv = _bf16(k), _bf16(v)
    cu = _cu(counts, 2)
    out = cuda_lib.paged_attn_cache_accept(gk, gv, _t(tables), _t(lens), _t(cu), _t(accepted), _t(num))
    _raises(cuda_lib)
    new, bad, page = ref.accept(k, v, tables, lens, cu, accepted, num)
    assert not bad and not page
    np.testing.assert_array_equal(out.cpu().numpy(), new)
    np.testing.assert_array_equal(_bits(gk), k)
    np.testing.assert_array_equal(_bits(gv), v)


def test_accept_bad_lists(cuda_lib):
    """Lists out of order or out of range, counts out of range, lengths below
    the drafts: a row's acceptance ends before its first bad entry."""
    rng = np.random.default_rng(22)
    counts = [8] * 8
    lens = np.asarray([40, 41, 42, 43, 44, 5, 46, 8], dtype=np.int32)
    tables, blocks = ref.tables_for(rng, lens)
    accepted = np.asarray([[1, 3, 3, 5], [2, 1, 4, 5], [0, 2, 8, 9], [-1, 2, 3, 4], [1, 3, 5, 7],
                           [4, 5, 6, 7], [0, 1, 2, 3], [2 ** 31 - 1, 0, 0, 0]], dtype=np.int32)
    num = np.asarray([4, 4, 4, 4, 9, 4, -2, 2], dtype=np.int32)
    k, v = ref.new_caches(rng, blocks, 2, 64)
    gk, gv = _bf16(k), _bf16(v)
    cu = _cu(counts)
    out = cuda_lib.paged_attn_cache_accept(gk, gv, _t(tables), _t(lens), _t(cu), _t(accepted), _t(num))
    _raises(cuda_lib, -12)
    new, bad, page = ref.accept(k, v, tables, lens, cu, accepted, num)
    assert bad and not page
    np.testing.assert_array_equal(out.cpu().numpy(), new)
    np.testing.assert_array_equal(_bits(gk), k)
    np.testing.assert_array_equal(_bits(gv), v)


def test_accept_bad_pages(cuda_lib):
    rng = np.random.default_rng(23)
    counts = [30, 30]
    lens = np.asarray([60, 75], dtype=np.int32)
    tables, blocks = ref.tables_for(rng, lens, width=4)
    tables[0, 3] = blocks + 7
    accepted = np.asarray([[2, 20, 21, 29], [1, 9, 25, 28]], dtype=np.int32)
    num = np.asarray([4, 4], dtype=np.int32)
    k, v = ref.new_caches(rng, blocks, 2, 128)
    gk, gv = _bf16(k), _bf16(v)
    cu = _cu(counts)
    out = cuda_lib.paged_attn_cache_accept(gk, gv, _t(tables), _t(lens), _t(cu), _t(accepted), _t(num))
    _raises(cuda_lib, -11)
    new, bad, page = ref.accept(k, v, tables, lens, cu, accepted, num)
    assert page and not bad
    np.testing.assert_array_equal(out.cpu().numpy(), new)
    np.testing.assert_array_equal(_bits(gk), k)
    np.testing.assert_array_equal(_bits(gv), v)


# -------------------------------------------------------------- fork and free
def _pool(rng, rows, lens, blocks_more, hkv=2, d=64):
    width = max(2, max(-(-n // PAGE) for n in lens) + 1)
    all_lens = np.asarray(list(lens) + [0] * (rows - len(lens)), dtype=np.int32)
    tables, blocks = ref.tables_for(rng, all_lens, width=width, spare=blocks_more)
    refs = np.zeros(blocks, dtype=np.int32)
    for i, n in enumerate(all_lens):
        refs[tables[i, :-(-n // PAGE)]] += 1
    k, v = ref.new_caches(rng, blocks, hkv, d)
    return k, v, tables, all_lens, refs


def _same(got, want):
    for g, w in zip(got, want):
        np.testing.assert_array_equal(_bits(g) if w.dtype == np.uint16 else g.cpu().numpy(), w)


def _fork(vlp, state, src, dst, codes=()):
    k, v, tables, lens, refs = state
    dev = [_bf16(k), _bf16(v), _t(tables), _t(lens), _t(refs)]
    vlp.paged_attn_cache_fork(*dev, _t(np.asarray(src, np.int32)), _t(np.asarray(dst, np.int32)))
    _raises(vlp, *codes)
    bad, dry = ref.fork(k, v, tables, lens, refs, src, dst)
    _same(dev, state)
    return bad, dry


@pytest.mark.parametrize("hkv,d", [(2, 64), (8, 128), (1, 256), (3, 128)])
def test_fork(cuda_lib, hkv, d):
    rng = np.random.default_rng(31)
    state = _pool(rng, 12, [40, 48, 1, 0, 16, 17], 9, hkv, d)
    assert _fork(cuda_lib, state, [0, 0, 1, 5, 3, 2], [6, 7, 8, 9, 10, 11]) == (False, False)


def test_fork_many_rows_and_pages(cuda_lib):
    """More forks than the plan's threads, and free pages past its first sweep."""
    rng = np.random.default_rng(32)
    lens = [int(x) for x in rng.integers(1, 60, 1500)]
    state = _pool(rng, 3000, lens, 1600)
    k, v, tables, all_lens, refs = state
    hold = np.flatnonzero(refs == 0)[:100]
    refs[hold] = 1  # held by no row
    assert _fork(cuda_lib, state, [int(x) for x in rng.integers(0, 1500, 1400)],
                 [int(x) for x in 1500 + rng.permutation(1500)[:1400]]) == (False, False)


def test_fork_refusals(cuda_lib):
    """Rows out of range, rows that hold tokens, a row that is a source, one
    named twice (the first counts), and a pool without a free page."""
    rng = np.random.default_rng(33)
    state = _pool(rng, 10, [40, 33, 20], 4)
    assert _fork(cuda_lib, state, [0, 1, 2, 3, 0, 10, 1, -1, 4], [5, 5, 1, 3, 6, 7, 10, 8, 9],
                 (-14,)) == (True, False)
    state = _pool(rng, 8, [40, 33, 16], 2)
    assert _fork(cuda_lib, state, [0, 2, 1, 0, 2], [3, 4, 5, 6, 7], (-13,)) == (False, True)


def test_fork_long_row_and_bad_pages(cuda_lib):
    """A length past the table has no partial page; bad ids are not counted."""
    rng = np.random.default_rng(34)
    state = _pool(rng, 4, [40, 33], 3)
    k, v, tables, lens, refs = state
    lens[0] = tables.shape[1] * PAGE + 5
    tables[0, :] = tables[0, 0]
    assert _fork(cuda_lib, state, [0], [2]) == (False, False)
    dev = [_bf16(k), _bf16(v), _t(tables), _t(lens), _t(refs)]
    dev[2][1, 0], dev[2][1, 2] = -5, 10 ** 6
    cuda_lib.paged_attn_cache_fork(*dev, _t(np.asarray([1], np.int32)), _t(np.asarray([3], np.int32)))
    _raises(cuda_lib, -11)
    _same(dev[:2], (k, v))


@pytest.mark.parametrize("rows", [0, 3])
def test_nothing_to_fork_or_free(cuda_lib, rows):
    rng = np.random.default_rng(31)
    k, v = ref.new_caches(rng, 4, 2, 64)
    gk, gv, none = _bf16(k), _bf16(v), _t(np.zeros(0, dtype=np.int32))
    tables, lens = np.zeros((rows, 2), dtype=np.int32), np.zeros(rows, dtype=np.int32)
    refs = _t(np.ones(4, dtype=np.int32))
    cuda_lib.paged_attn_cache_fork(gk, gv, _t(tables), _t(lens), refs, none, none)
    cuda_lib.paged_attn_cache_free(_t(tables), _t(lens), refs, none)
    _raises(cuda_lib)
    np.testing.assert_array_equal(_bits(gk), k)
    assert (refs.cpu().numpy() == 1).all()


def test_free(cuda_lib):
    rng = np.random.default_rng(35)
    k, v, tables, lens, refs = _pool(rng, 9, [40, 48, 1, 0, 16, 300], 3)
    refs[tables[1, :3]] += 2
    rows = [1, 5, 1, 3, 2]  # one twice, one empty
    dev = [_t(tables), _t(lens), _t(refs)]
    cuda_lib.paged_attn_cache_free(*dev, _t(np.asarray(rows, np.int32)))
    _raises(cuda_lib)
    assert not ref.free(tables, lens, refs, rows)
    _same(dev, (tables, lens, refs))


def test_free_refusals(cuda_lib):
    rng = np.random.default_rng(36)
    k, v, tables, lens, refs = _pool(rng, 4, [40, 48], 3)
    refs[tables[0, 1]] = 0
    dev = [_t(tables), _t(lens), _t(refs)]
    rows = [0, 4, -1, 1]
    cuda_lib.paged_attn_cache_free(*dev, _t(np.asarray(rows, np.int32)))
    _raises(cuda_lib, -14)
    assert ref.free(tables, lens, refs, rows)
    _same(dev, (tables, lens, refs))


def test_fork_then_free_gives_the_pool_back(cuda_lib):
    rng = np.random.default_rng(37)
    state = _pool(rng, 8, [100, 37], 9)
    before = [a.copy() for a in state]
    assert _fork(cuda_lib, state, [0, 1, 1], [4, 5, 6]) == (False, False)
    k, v, tables, lens, refs = state
    dev = [_t(tables), _t(lens), _t(refs)]
    cuda_lib.paged_attn_cache_free(*dev, _t(np.asarray([4, 5, 6], np.int32)))
    _raises(cuda_lib)
    np.testing.assert_array_equal(dev[1].cpu().numpy(), before[3])
    np.testing.assert_array_equal(dev[2].cpu().numpy(), before[4])


# -------------------------------------------------------------------- compact
@pytest.mark.parametrize("blocks,used,hkv,d", [
    (1, 1, 2, 64), (1, 0, 2, 64), (7, 7, 2, 64), (64, 30, 2, 128), (300, 1, 1, 64), (300, 299, 3, 128),
    (4096, 2000, 1, 64), (4096, 4096, 1, 64), (5000, 4093, 1, 64), (9001, 4100, 1, 64),
    (16384, 9000, 1, 64), (16385, 16384, 1, 64), (33000, 20000, 1, 64), (100, 50, 8, 256)])
@pytest.mark.parametrize("place", [False, True])
def test_compact(cuda_lib, blocks, used, hkv, d, place):
    rng = np.random.default_rng(41)
    ids = rng.permutation(blocks)[:used]
    rows, width = 5, max(2, -(-used // 4) + 1)
    tables = np.full((rows, width), -1, dtype=np.int32)
    lens = np.zeros(rows, dtype=np.int32)
    for i in range(4):  # row 4 stays empty
        mine = ids[i * used // 4:(i + 1) * used // 4]
        tables[i, :len(mine)] = mine
        lens[i] = max(0, len(mine) * PAGE - i)
    refs = np.zeros(blocks, dtype=np.int32)
    refs[ids] = rng.integers(1, 5, used)
    k, v = ref.new_caches(rng, blocks, hkv, d)
    dev = [_bf16(k), _bf16(v), _t(tables), _t(lens), _t(refs)]
    got = cuda_lib.paged_attn_cache_compact(*dev, out=(dev[2], dev[4]) if place else None)
    _raises(cuda_lib)
    if not place:
        _same((dev[2], dev[4]), (tables, refs))  # the inputs keep their values
    want = ref.compact(k, v, tables, lens, refs)
    _same((dev[0], dev[1], *got), (k, v, *want))
    assert (np.flatnonzero(want[1] > 0) == np.arange(used)).all()


def test_compact_reports_bad_entries(cuda_lib):
    rng = np.random.default_rng(42)
    k, v, tables, lens, refs = _pool(rng, 3, [40, 33], 6)
    tables[1, 1] = 10 ** 6
    dev = [_bf16(k), _bf16(v), _t(tables), _t(lens), _t(refs)]
    got = cuda_lib.paged_attn_cache_compact(*dev)
    _raises(cuda_lib, -11)
    assert got[0][1, 1].item() == 10 ** 6


# ---------------------------------------------------------- streams and graphs
def test_calls_on_another_stream(cuda_lib):
    """Workspaces belong to the stream of the call."""
    import torch
    rng = np.random.default_rng(43)
    state = _pool(rng, 8, [100, 37], 9)
    k, v, tables, lens, refs = state
    dev = [_bf16(k), _bf16(v), _t(tables), _t(lens), _t(refs)]
    src, dst = _t(np.asarray([0, 1], np.int32)), _t(np.asarray([4, 5], np.int32))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    cuda_lib.paged_attn_cache_fork(*dev, src, dst, stream=side)
    got = cuda_lib.paged_attn_cache_compact(*dev, stream=side)
    side.synchronize()
    _raises(cuda_lib)
    ref.fork(k, v, tables, lens, refs, [0, 1], [4, 5])
    want = ref.compact(k, v, tables, lens, refs)
    _same((dev[0], dev[1], *got), (k, v, *want))


def test_captured_and_replayed(cuda_lib):
    """A beam step, captured once and replayed: free, fork, compact in place."""
    import torch
    rng = np.random.default_rng(44)
    state = _pool(rng, 8, [100, 37], 9)
    k, v, tables, lens, refs = state
    dev = [_bf16(k), _bf16(v), _t(tables), _t(lens), _t(refs)]
    src, dst = _t(np.asarray([0, 1, 1], np.int32)), _t(np.asarray([4, 5, 6], np.int32))

    def step():
        cuda_lib.paged_attn_cache_free(*dev[2:], dst)
        cuda_lib.paged_attn_cache_fork(*dev, src, dst)
        cuda_lib.paged_attn_cache_compact(*dev, out=(dev[2], dev[4]))

    def want():
        ref.free(tables, lens, refs, [4, 5, 6])
        ref.fork(k, v, tables, lens, refs, [0, 1, 1], [4, 5, 6])
        tables[:], refs[:] = ref.compact(k, v, tables, lens, refs)

    step()
    want()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
        want()
    torch.cuda.synchronize()
    _raises(cuda_lib)
    _same(dev, state)
