"""Attention rows that one key decides, for scores so large that a softmax is a choice."""
import numpy as np

import paged_q8_ref as ref


def winners(q, cache, tables, lens, cu, kind, scale, fold=0.0):
    """(out, decided): the value of the key with the largest score, and whether its lead is sure.

    A score is off by (d + 8) 2^-23 of the sum of its products' magnitudes (sums in 32 bits, which tensor
    cores may cut), by 4 roundings of 2^-24 of itself and by `fold` of itself, for what is told apart no further;
    a lead of 400 more than twice that leaves the others no weight, whatever the size of their values."""
    k, v, ks, vs = cache
    total, hq, d = q.shape
    group = hq // v.shape[1]
    out, decided = np.zeros(q.shape), np.zeros((total, hq), dtype=bool)
    for i, lo, n, size in ref.slices(cu, lens, total):
        key, value, good = ref.dense(k, v, ks, vs, tables, i, size, kind)
        for j in range(n):
            seen = np.nonzero(good[:max(size - n + j + 1, 0)])[0]
            for h in range(hq if seen.size else 0):
                a, x = key[seen, h // group], q[lo + j, h]
                to_log2 = scale * np.log2(np.e)
                s = a @ x * to_log2
                off = (d + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(x)).max() * to_log2 + (4 * 2.0 ** -24 + fold) * np.abs(s).max()
                best = int(s.argmax())
                rest = np.delete(s, best)
                decided[lo + j, h] = not rest.size or s[best] - rest.max() > 2 * off + 400
                out[lo + j, h] = value[seen[best], h // group]
    return out, decided


def check_winners(got, want, decided, half, least):
    """The weight is rounded to fp16 (2^-11), the exponentials to 2^-22 each, the result once."""
    assert np.isfinite(got).all()
    bound = (half * (1 + 2.0 ** -10) + 2.0 ** -11 + 2.0 ** -20) * np.abs(want) + least
    off = (np.abs(got - want) / bound)[decided]
    assert off.size and off.max() <= 1.0, off.max()
