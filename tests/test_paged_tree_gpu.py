"""Tree attention over a paged cache against the float64 reference: every head
layout and size, one token to many tiles of keys, trees, chains and single
tokens, rows that see nothing, NaN and infinities where a row does not look."""
import numpy as np
import pytest

import paged_cache_ref as cref
import paged_tree_ref as ref
from workloads import bf16_bits_to_f64, f16_bits_to_f64, round_to_bf16_bits, round_to_f16_bits

pytestmark = pytest.mark.gpu


def _dev(a, dtype=None):
    import torch
    a = np.ascontiguousarray(a)
    if dtype:
        return torch.from_numpy(a.view(np.int16)).view(
            torch.bfloat16 if dtype == "bf16" else torch.float16).cuda()
    return torch.from_numpy(a).cuda()


def _bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _wide(bits, dtype):
    return (bf16_bits_to_f64 if dtype == "bf16" else f16_bits_to_f64)(bits)


def _round(x, dtype):
    return (round_to_bf16_bits if dtype == "bf16" else round_to_f16_bits)(x.astype(np.float32))


class Case:
    """rows: (context, drafts) of each sequence; tree: "tree", "chain" or None."""

    def __init__(self, rows, hq, hkv, d, dtype="bf16", tree="tree", seed=0, width=None, start=0,
                 behind=3, spread=1.0):
        rng = np.random.default_rng(seed)
        self.dtype = dtype
        self.lens = np.asarray([c + n for c, n in rows], dtype=np.int32)
        counts = [n for _, n in rows]
        self.cu = (start + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
        self.total = int(self.cu[-1]) + behind
        self.tables, blocks = cref.tables_for(rng, self.lens, width=width, fill=0)
        x = lambda *s: _round(rng.standard_normal(s) * spread, dtype)  # noqa: E731
        self.q = x(self.total, hq, d)
        self.k = x(blocks, hkv, d // 8, 16, 8)
        self.v = _round(rng.standard_normal((blocks, hkv, d, 16)), dtype)
        self.parents = None
        if tree:
            self.parents = np.full(self.total, -1, dtype=np.int32)
            for i, n in enumerate(counts):
                for j in range(n):
                    self.parents[self.cu[i] + j] = j - 1 if tree == "chain" else \
                        max(-1, j - 1 - int(rng.integers(0, 4)))

    def launch(self, vlp, **kw):
        import torch
        out = torch.full(self.q.shape, 7.0, device="cuda",
                         dtype=torch.bfloat16 if self.dtype == "bf16" else torch.float16)
        return vlp.paged_attn_tree(
            _dev(self.q, self.dtype), _dev(self.k, self.dtype), _dev(self.v, self.dtype),
            _dev(self.tables), _dev(self.lens), _dev(self.cu),
            _dev(self.parents) if self.parents is not None else None, out=out, **kw)

    def run(self, vlp, **kw):
        out = self.launch(vlp, **kw)
        vlp.check()
        return _bits(out)

    def want(self, scale=None):
        w = lambda a: _wide(a, self.dtype)  # noqa: E731
        return ref.tree(w(self.q), w(self.k), w(self.v), self.tables, self.lens, self.cu,
                        self.parents, scale, fill=7.0)

    def check(self, vlp, **kw):
        got = _wide(self.run(vlp, **kw), self.dtype)
        self.compare(got, **kw)
        return got

    def compare(self, got, scale=None, want=None):
        out, absv, sumv, top = want or self.want(scale)
        b = ref.bound(out, absv, sumv, top, self.dtype, self.q.shape[2])
        fine = np.isfinite(out)
        np.testing.assert_array_equal(np.isnan(got), np.isnan(out))
        np.testing.assert_array_equal(got[np.isinf(out)], out[np.isinf(out)])
        with np.errstate(invalid="ignore"):
            over = (np.abs(got - out) > b) & fine
        assert not over.any(), (int(over.sum()), np.argwhere(over)[:4].tolist(),
                                float((np.abs(got - out)[over] / b[over]).max()))


HEADS = [(16, 16), (16, 2), (3, 3), (32, 4), (40, 8), (4, 1), (64, 8), (1, 1), (129, 1), (26, 2)]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16"), (128, "bf16"), (256, "bf16"),
                                     (256, "fp16"), (64, "fp16")])
def test_heads(cuda_lib, hq, hkv, d, dtype):
    Case([(45, 7), (130, 1), (0, 3)], hq, hkv, d, dtype, seed=hq + d).check(cuda_lib)


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 47, 63, 64, 65, 111, 112, 127, 128, 129, 241,
                                 255, 256, 257, 300, 511, 640])
@pytest.mark.parametrize("d", [128, 256])
def test_context_edges(cuda_lib, ctx, d):
    Case([(ctx, 5), (ctx, 1), (ctx, 16)], 8, 2, d, seed=ctx).check(cuda_lib)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 256])
@pytest.mark.parametrize("tree", ["tree", "chain", None])
def test_draft_counts(cuda_lib, n, tree):
    Case([(37, n), (150, n)], 4, 2, 64, tree=tree, seed=n).check(cuda_lib)


def test_chain_is_the_same_as_no_parents(cuda_lib):
    a = Case([(100, 40), (7, 9)], 8, 2, 128, tree="chain", seed=3)
    b = a.run(cuda_lib)
    a.parents = None
    np.testing.assert_array_equal(a.run(cuda_lib), b)


def test_one_token_is_the_decode(cuda_lib):
    """n = 1 is paged_attn_decode's operation: both meet the bound."""
    c = Case([(n, 1) for n in (0, 1, 63, 64, 500, 31)], 16, 4, 128, tree=None, behind=0, seed=4)
    c.check(cuda_lib)
    dec = cuda_lib.paged_attn_decode(_dev(c.q, "bf16"), _dev(c.k, "bf16"), _dev(c.v, "bf16"),
                                     _dev(c.tables), _dev(c.lens))
    c.compare(_wide(_bits(dec), "bf16"))


def test_many_sequences(cuda_lib):
    """More sequences than CTAs, empty ones and rows before the first among them."""
    rows = [((i * 29) % 200, (i * 5) % 7) for i in range(700)]
    Case(rows, 4, 2, 64, seed=5, start=3).check(cuda_lib)


def test_few_long_sequences(cuda_lib):
    """The keys of a sequence are split over many CTAs, and joined."""
    Case([(5000, 6), (40, 2), (2500, 33)], 8, 2, 128, seed=6).check(cuda_lib)
    Case([(9000, 3)], 2, 1, 64, "fp16", seed=7).check(cuda_lib)
    Case([(3100, 9)], 4, 1, 256, seed=8).check(cuda_lib)


# one sequence by itself: its row tiles are split over 2 to about 70 CTAs, and
# their parts joined by one to eight groups of warps
PARTS = [250, 700, 1300, 2600, 6000, 21000]


@pytest.mark.parametrize("ctx", PARTS)
@pytest.mark.parametrize("hq,hkv,d,dtype,n", [(3, 1, 64, "bf16", 3), (8, 1, 128, "fp16", 5),
                                              (10, 2, 128, "bf16", 33), (8, 1, 256, "bf16", 20)])
def test_parts_of_one_long_sequence(cuda_lib, ctx, hq, hkv, d, dtype, n):
    c = Case([(ctx, n)], hq, hkv, d, dtype, seed=32)
    c.compare(_wide(c.run(cuda_lib), dtype), want=_dense(c))


@pytest.mark.parametrize("hq,hkv,d,dtype", [(4, 1, 64, "fp16"), (8, 1, 128, "bf16"),
                                            (4, 1, 256, "bf16")])
def test_nonfinite_context_in_one_of_many_parts(cuda_lib, hq, hkv, d, dtype):
    c = Case([(6000, 3), (9, 2)], hq, hkv, d, dtype, seed=33)
    nan, inf = (0x7FC0, 0x7F80) if dtype == "bf16" else (0x7E00, 0x7C00)
    c.v[c.tables[0, 100], 0, 4, 3] = nan
    c.v[c.tables[0, 200], 0, 7, 9] = inf
    c.v[c.tables[0, 300], 0, d - 1, 15] = inf
    got = c.check(cuda_lib)[:3]
    assert np.isnan(got[:, :, 4]).all() and np.isposinf(got[:, :, [7, d - 1]]).all()
    assert np.isfinite(np.delete(got, [4, 7, d - 1], axis=2)).all()


def _dense(c, scale=None):
    """ref.tree on the GPU, a (sequence, KV head) at a time, for finite inputs."""
    import torch
    total, hq, d = c.q.shape
    hkv = c.k.shape[1]
    grp = hq // hkv
    scale = scale or d ** -0.5
    q, k, v = (_dev(x, c.dtype).double() for x in (c.q, c.k, c.v))
    out = torch.full((total, hq, d), 7.0, dtype=torch.float64, device="cuda")
    absv, sumv = torch.zeros_like(out), torch.zeros_like(out)
    top = torch.zeros((total, hq), dtype=torch.float64, device="cuda")
    for i in range(len(c.lens)):
        lo, n, sees = ref.visible(c.lens, c.cu, c.parents, c.tables, c.k.shape[0], i, total)
        size = int(c.lens[i])
        mask = np.zeros((n, size), dtype=bool)
        for j in range(n):
            mask[j, sees[j]] = True
        mask = torch.from_numpy(mask).cuda().repeat_interleave(grp, 0)
        pages = torch.from_numpy(c.tables[i, :-(-size // 16)]).long().cuda()
        for g in range(hkv):
            key = k[pages, g].permute(0, 2, 1, 3).reshape(-1, d)[:size]
            val = v[pages, g].permute(0, 2, 1).reshape(-1, d)[:size]
            rows = q[lo:lo + n, g * grp:(g + 1) * grp].reshape(-1, d)
            w = torch.softmax((scale * rows @ key.T).masked_fill(~mask, float("-inf")), dim=1)
            at = (slice(lo, lo + n), slice(g * grp, (g + 1) * grp))
            out[at] = (w @ val).view(n, grp, d)
            absv[at] = (w @ val.abs()).view(n, grp, d)
            sumv[at] = (mask.double() @ val.abs()).view(n, grp, d)
            top[at] = ((scale * rows.abs() @ key.abs().T) * mask).amax(1).view(n, grp)
    return tuple(t.cpu().numpy() for t in (out, absv, sumv, top))


LONG = [
    # every CTA walks dozens of key tiles: rings and phases wrap, page ids come
    # in several reads, row tiles of 1 to 128 and of several times 128 rows
    ([(8000, 2)] * 8, 8, 8, 128, "bf16"),
    ([(8000, 12)] * 8, 32, 8, 128, "bf16"),
    ([(8000, 16)] * 4, 64, 8, 128, "fp16"),
    ([(5000 + 333 * i, 1 + 7 * i) for i in range(9)], 40, 8, 128, "bf16"),
    ([(5000 + 333 * i, 1 + 7 * i) for i in range(9)], 16, 4, 64, "fp16"),
    ([(5000 + 333 * i, 1 + 7 * i) for i in range(9)], 16, 4, 256, "bf16"),
    ([(3000, 3)] * 16, 16, 16, 256, "fp16"),
    ([(100, 3)] * 300, 16, 16, 128, "bf16"),
    ([(20, 1)] * 600, 8, 8, 64, "bf16"),
]


@pytest.mark.parametrize("rows,hq,hkv,d,dtype", LONG, ids=range(len(LONG)))
def test_long_walks(cuda_lib, rows, hq, hkv, d, dtype):
    c = Case(rows, hq, hkv, d, dtype, seed=30)
    want = _dense(c)
    for _ in range(20):  # queued one behind the other
        out = c.launch(cuda_lib)
    cuda_lib.check()
    got = _wide(_bits(out), dtype)
    c.compare(got, want=want)


def test_dense_reference_agrees(cuda_lib):
    c = Case([(45, 7), (130, 1), (0, 3)], 8, 2, 64, seed=31)
    for a, b in zip(_dense(c), c.want()):
        np.testing.assert_allclose(a, b, rtol=1e-9, atol=1e-12)


def test_rising_scores(cuda_lib):
    """Scores that rise along the context raise the running maximum in every tile."""
    c = Case([(1500, 4)] * 30, 4, 4, 128, seed=9, spread=0.5)
    k = _wide(c.k, "bf16")
    for i in range(30):
        for p in range(1500):
            k[c.tables[i, p // 16], :, :, p % 16, :] *= 1 + p / 100
    c.k = _round(k, "bf16")
    c.compare(_wide(c.run(cuda_lib), "bf16"), want=_dense(c))


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
def test_garbage_where_no_row_looks(cuda_lib, d, dtype):
    """Unused pages, and slots behind the last token, hold NaN and infinities."""
    c = Case([(45, 7), (130, 1), (0, 3), (128, 0), (250, 9)], 8, 2, d, dtype, seed=10)
    bad = np.asarray([0x7FC0, 0x7F80, 0xFF80] if dtype == "bf16" else [0x7E00, 0x7C00, 0xFC00],
                     dtype=np.uint16)
    rng = np.random.default_rng(1)
    used = np.zeros((c.k.shape[0], 16), dtype=bool)
    for i, n in enumerate(c.lens):
        for p in range(n):
            used[c.tables[i, p // 16], p % 16] = True
    for page, slot in np.argwhere(~used):
        c.k[page, :, :, slot] = rng.choice(bad, c.k[page, :, :, slot].shape)
        c.v[page, :, :, slot] = rng.choice(bad, c.v[page, :, :, slot].shape)
    assert np.isfinite(c.check(cuda_lib)).all()


@pytest.mark.parametrize("d,dtype,hq,hkv", [(128, "bf16", 4, 2), (256, "fp16", 2, 1),
                                            (64, "fp16", 8, 1)])
def test_nonfinite_drafts_stay_in_their_branch(cuda_lib, d, dtype, hq, hkv):
    """NaN and infinities in a draft reach the rows that see it and no other."""
    c = Case([(45, 12), (0, 30), (3000, 8)], hq, hkv, d, dtype, seed=11)
    nan, inf, ninf = (0x7FC0, 0x7F80, 0xFF80) if dtype == "bf16" else (0x7E00, 0x7C00, 0xFC00)
    for i, j, dim, x in [(0, 3, 5, nan), (0, 7, 2, inf), (0, 8, 2, ninf), (1, 20, 0, inf),
                         (1, 29, d - 1, nan), (2, 4, 9, ninf), (2, 7, 9, inf)]:
        p = int(c.lens[i] - (c.cu[i + 1] - c.cu[i])) + j
        c.v[c.tables[i, p // 16], :, dim, p % 16] = x
    for i, j in [(0, 10), (1, 28), (2, 6)]:  # a key of NaN: the rows that see it are NaN
        p = int(c.lens[i] - (c.cu[i + 1] - c.cu[i])) + j
        c.k[c.tables[i, p // 16], :, 0, p % 16, :] = nan
    got = c.check(cuda_lib)
    assert np.isnan(got).any() and np.isinf(got).any() and np.isfinite(got).any()


def test_nonfinite_context_reaches_every_row(cuda_lib):
    c = Case([(45, 6), (300, 3)], 4, 2, 128, seed=12)
    c.v[c.tables[0, 1], :, 4, 3] = 0x7FC0
    c.v[c.tables[1, 9], :, 7, 3] = 0x7F80
    got = c.check(cuda_lib)
    assert np.isnan(got[:6, :, 4]).all() and np.isinf(got[6:9, :, 7]).all()


def test_scale(cuda_lib):
    Case([(70, 5)], 4, 2, 64, seed=13).check(cuda_lib, scale=0.37)


@pytest.mark.parametrize("scale", [0.0, -1.0, 1e-46, 2.0 ** 127, float("inf"), float("nan")])
def test_scales_that_32_bits_do_not_hold_are_refused(cuda_lib, scale):
    with pytest.raises(ValueError, match="scale"):
        Case([(7, 2)], 2, 1, 64, seed=15).check(cuda_lib, scale=scale)


def test_lengths_below_the_drafts(cuda_lib):
    """Fewer tokens than drafts: those at negative positions do not exist, and
    a row that sees nothing is zero.  Negative lengths are empty."""
    c = Case([(10, 8), (20, 8), (30, 4), (0, 3)], 4, 2, 64, seed=14)
    c.lens[:] = [5, 0, -7, 3]
    got = c.check(cuda_lib)
    assert (got[8:20] == 0).all()


def test_slices_that_step_backwards(cuda_lib):
    c = Case([(60, 8), (50, 8), (40, 8), (33, 5)], 4, 2, 64, seed=15)
    c.parents[:] = -1
    c.cu[:] = [10, 14, 6, 10, 4]  # sequences 1 and 3 are empty
    c.lens[:] = [68, 40, 45, 38]
    c.check(cuda_lib)
    c.cu[:] = [-2, 5, 9, 20, 60]  # the first starts before the rows, the last ends past them
    c.check(cuda_lib)


def test_past_the_table(cuda_lib):
    """Tokens past the table's width do not exist."""
    c = Case([(60, 8), (50, 3)], 4, 2, 64, width=3, seed=16)
    c.check(cuda_lib)


def test_bad_pages_and_parents(cuda_lib):
    from variable_length_prefill_gb300 import AttnVarlenError
    c = Case([(300, 8), (50, 8), (5, 9)], 4, 2, 128, seed=17)
    c.tables[0, 3], c.tables[0, 18], c.tables[2, 0] = -1, 10 ** 6, c.k.shape[0]
    got = _wide(_bits(c.launch(cuda_lib)), "bf16")
    with pytest.raises(AttnVarlenError) as e:
        cuda_lib.check()
    assert e.value.code == -11
    c.compare(got)
    c = Case([(300, 8), (50, 8), (5, 9)], 4, 2, 128, seed=17)
    c.parents[[2, 9, 20]] = [2, -2, 10 ** 9]
    got = _wide(_bits(c.launch(cuda_lib)), "bf16")
    with pytest.raises(AttnVarlenError) as e:
        cuda_lib.check()
    assert e.value.code == -12
    c.compare(got)
    cuda_lib.check()


def test_too_many_drafts(cuda_lib):
    from variable_length_prefill_gb300 import AttnVarlenError
    c = Case([(30, 257), (20, 3)], 2, 1, 64, seed=18)
    got = _wide(_bits(c.launch(cuda_lib)), "bf16")
    with pytest.raises(AttnVarlenError) as e:
        cuda_lib.check()
    assert e.value.code == -12
    c.compare(got)
    assert (got[:257] == 0).all()


def test_deterministic(cuda_lib):
    c = Case([(5000, 6), (40, 2), (2500, 33)], 8, 2, 128, seed=6)
    np.testing.assert_array_equal(c.run(cuda_lib), c.run(cuda_lib))


def test_two_streams_at_once(cuda_lib):
    """Calls share no workspace: two streams give what each gives alone."""
    import torch
    cases = [Case([(3000, 6)], 8, 2, 128, seed=19), Case([(2500, 9), (70, 2)], 8, 2, 128, seed=20)]
    alone = [c.run(cuda_lib) for c in cases]
    args = [[_dev(c.q, "bf16"), _dev(c.k, "bf16"), _dev(c.v, "bf16"), _dev(c.tables), _dev(c.lens),
             _dev(c.cu), _dev(c.parents)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [cuda_lib.paged_attn_tree(*a, stream=s) for a, s in zip(args, streams)]
        for s in streams:
            s.synchronize()
        for c, g, want in zip(cases, got, alone):
            np.testing.assert_array_equal(_bits(g)[:c.total - 3], want[:c.total - 3])
    cuda_lib.check()


def test_captured_step_of_drafting(cuda_lib):
    """A verification step as a server runs it, captured and replayed: write
    the drafts, attend, move the accepted path up, and go on from there."""
    import torch
    rng = np.random.default_rng(23)
    lens0, n, hq, hkv, d = [50, 0, 127], 8, 8, 2, 128
    s = len(lens0)
    lens = np.asarray([x + n for x in lens0], dtype=np.int32)
    tables, blocks = cref.tables_for(rng, [x + 40 for x in lens], fill=0)
    cu = np.arange(s + 1, dtype=np.int32) * n
    x = lambda *sh: _round(rng.standard_normal(sh), "bf16")  # noqa: E731
    k, v = x(blocks, hkv, d // 8, 16, 8), x(blocks, hkv, d, 16)
    parents = np.tile(np.asarray([-1, 0, 0, 1, 1, 2, 4, 4], dtype=np.int32), s)
    accepted = np.asarray([[0, 1, 4, 7], [0, 2, 5, 5], [1, 1, 1, 1]], dtype=np.int32)
    num = np.asarray([4, 3, 1], dtype=np.int32)
    gk, gv, gt, gcu, gp = _dev(k, "bf16"), _dev(v, "bf16"), _dev(tables), _dev(cu), _dev(parents)
    glen, ga, gn = _dev(lens), _dev(accepted), _dev(num)
    gq, gkey, gval = (torch.zeros((s * n, h, d), dtype=torch.bfloat16, device="cuda")
                      for h in (hq, hkv, hkv))
    gout = torch.empty_like(gq)

    def step():
        cuda_lib.paged_attn_cache_write(gkey, gval, gk, gv, gt, glen, gcu)
        cuda_lib.paged_attn_tree(gq, gk, gv, gt, glen, gcu, gp, out=gout)
        new = cuda_lib.paged_attn_cache_accept(gk, gv, gt, glen, gcu, ga, gn)
        glen.copy_(new + n)  # room for the next drafts

    graph = None
    for turn in range(4):
        q, key, val = x(s * n, hq, d), x(s * n, hkv, d), x(s * n, hkv, d)
        for g, a in ((gq, q), (gkey, key), (gval, val)):
            g.copy_(_dev(a, "bf16"))
        if turn == 1:
            keep = [t.clone() for t in (gk, gv, glen)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for t, o in zip((gk, gv, glen), keep):
                t.copy_(o)
        graph.replay() if graph else step()
        cuda_lib.check()
        cref.write(key, val, k, v, tables, lens, cu)
        w = bf16_bits_to_f64
        out, absv, sumv, top = ref.tree(w(q), w(k), w(v), tables, lens, cu, parents)
        got = w(_bits(gout))
        assert (np.abs(got - out) <= ref.bound(out, absv, sumv, top, "bf16", d)).all()
        new, bad, page = cref.accept(k, v, tables, lens, cu, accepted, num)
        assert not bad and not page
        lens = (new + n).astype(np.int32)
        np.testing.assert_array_equal(glen.cpu().numpy(), lens)
        np.testing.assert_array_equal(_bits(gk), k)
        np.testing.assert_array_equal(_bits(gv), v)
