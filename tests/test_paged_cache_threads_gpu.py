"""Calls of several threads on one stream: each acts as if it were alone, in some
order, though some are more than one launch."""
import threading

import numpy as np
import pytest

import paged_cache_ref as ref
from test_paged_cache_gpu import _bf16, _pool, _t

pytestmark = pytest.mark.gpu


def _both(*calls):
    """The calls at once, a thread each, on the current stream."""
    import torch
    stream, gate, wrong = torch.cuda.current_stream(), threading.Barrier(len(calls)), []

    def work(call):
        try:
            gate.wait()
            call(stream)
        except BaseException as e:  # noqa: BLE001  (told to the test)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_forks_never_share_a_fresh_page(cuda_lib):
    rng = np.random.default_rng(55)
    k, v, tables, lens, refs = _pool(rng, 6, [20, 37], 12)
    dev = [_bf16(k), _bf16(v), _t(tables), _t(lens), _t(refs)]
    src, one, two = (_t(np.asarray(x, np.int32)) for x in ([0, 1], [2, 3], [4, 5]))
    both = _t(np.asarray([2, 3, 4, 5], np.int32))
    for _ in range(400):
        _both(lambda s: cuda_lib.paged_attn_cache_fork(*dev, src, one, stream=s),
              lambda s: cuda_lib.paged_attn_cache_fork(*dev, src, two, stream=s))
        cuda_lib.check()
        t, r = dev[2].cpu().numpy(), dev[4].cpu().numpy()
        last = [t[2, 1], t[3, 2], t[4, 1], t[5, 2]]
        assert len(set(last)) == 4 and (r[last] == 1).all(), (last, r.tolist())
        cuda_lib.paged_attn_cache_free(*dev[2:], both)
    cuda_lib.check()
    assert (dev[4].cpu().numpy() == refs).all()


def test_forks_and_compactions(cuda_lib):
    """Whatever the order, every row holds its tokens and counts its pages."""
    rng = np.random.default_rng(56)
    state = _pool(rng, 4, [20, 37], 40)
    k, v, tables, lens, refs = state
    dev = [_bf16(k), _bf16(v), _t(tables), _t(lens), _t(refs)]
    src, dst = _t(np.asarray([0, 1], np.int32)), _t(np.asarray([2, 3], np.int32))

    def tokens(row, n):
        at = np.arange(n)
        page = dev[2].cpu().numpy()[row, at // 16]
        kk, vv = (x.view(__import__("torch").int16).cpu().numpy().view(np.uint16) for x in dev[:2])
        return kk[page, :, :, at % 16], vv[page, :, :, at % 16]

    want = [tokens(0, 20), tokens(1, 37)]
    for _ in range(150):
        _both(lambda s: cuda_lib.paged_attn_cache_fork(*dev, src, dst, stream=s),
              lambda s: cuda_lib.paged_attn_cache_compact(*dev, out=(dev[2], dev[4]), stream=s))
        cuda_lib.check()
        for row, n, w in [(0, 20, 0), (2, 20, 0), (1, 37, 1), (3, 37, 1)]:
            for a, b in zip(tokens(row, n), want[w]):
                np.testing.assert_array_equal(a, b)
        count = np.zeros_like(refs)
        t = dev[2].cpu().numpy()
        for row, pages in enumerate([2, 3, 2, 3]):
            np.add.at(count, t[row, :pages], 1)
        np.testing.assert_array_equal(dev[4].cpu().numpy(), count)
        _both(lambda s: cuda_lib.paged_attn_cache_free(*dev[2:], dst, stream=s),
              lambda s: cuda_lib.paged_attn_cache_compact(*dev, out=(dev[2], dev[4]), stream=s))
        cuda_lib.check()
