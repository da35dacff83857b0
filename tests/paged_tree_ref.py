"""Tree attention over a paged cache in float64, a row at a time, and the
error bound that the kernel's arithmetic implies."""
import numpy as np

PAGE = 16


def visible(lens, cu, parents, tables, blocks, i, total):
    """(packed start, drafts, positions each draft sees) of sequence i."""
    lo, hi = max(int(cu[i]), 0), min(int(cu[i + 1]), total)
    n = max(hi - lo, 0)
    size = max(int(lens[i]), 0)
    base = size - n
    size = min(size, tables.shape[1] * PAGE)
    sees = []
    for j in range(n):
        mine = set()
        if n <= 256:
            mine |= set(range(max(0, min(base, size))))
            a = j
            while a >= 0:
                mine.add(base + a)
                up = a - 1 if parents is None else int(parents[lo + a])
                a = up if -1 <= up < a else -1
        sees.append([p for p in sorted(mine)
                     if 0 <= p < size and 0 <= tables[i, p // PAGE] < blocks])
    return lo, n, sees


def tree(q, k, v, tables, lens, cu, parents, scale=None, fill=np.nan):
    """q, k, v float64 (values of the 16-bit inputs); returns (out, bound_w,
    bound_s): out [total, Hq, D], sum of w |value|, and per row the largest
    scale * sum |q key| over the keys it sees, for the error bound."""
    total, hq, d = q.shape
    blocks, hkv = k.shape[:2]
    scale = scale or d ** -0.5
    out = np.full((total, hq, d), fill)
    absv = np.zeros((total, hq, d))
    sumv = np.zeros((total, hq, d))
    top = np.zeros((total, hq))
    for i in range(len(lens)):
        lo, n, sees = visible(lens, cu, parents, tables, blocks, i, total)
        for j in range(n):
            pos = np.asarray(sees[j], dtype=np.int64)
            pages, slots = (tables[i, pos // PAGE], pos % PAGE) if len(pos) else ([], [])
            for h in range(hq):
                if not len(pos):
                    out[lo + j, h] = 0.0
                    continue
                g = h // (hq // hkv)
                key = k[pages, g, :, slots, :].reshape(len(pos), d)
                val = v[pages, g, :, slots]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (key @ q[lo + j, h])
                    w = np.exp(s - s.max())
                    w = w / w.sum()
                    out[lo + j, h] = w @ val
                    absv[lo + j, h] = w @ np.abs(val)
                    sumv[lo + j, h] = np.abs(val).sum(0)
                    top[lo + j, h] = scale * (np.abs(key) @ np.abs(q[lo + j, h])).max()
    return out, absv, sumv, top


def bound(out, absv, sumv, top, dtype, d):
    """Largest error of an output element.

    u = eps / 2 of the type is the relative error of one rounding.  Weights are
    rounded once (u sum w |v|; fp16 weights below 2^-14, against a row maximum
    of at least 1, are off by at most 2^-25 instead, so 2^-25 sum |v| more) and
    so is the output (u |o|).  A score in fp32 is off by at most (d + 2) 2^-24
    scale sum |q k| for the products' sum and the scaling, and the base-2
    exponential and its argument by 2^-22 relative plus 2^-23 of the argument
    (|argument| <= 2 top / ln 2): a weight's relative error e bounds the
    output's by 2 e sum w |v| (numerator and normalisation).  Sums of up to 2^17
    weights and products, in fp32 in any order, are off by at most 2^-24 each
    step; pairwise over tiles of 128 and then tile by tile that is (128 + 1024)
    2^-24 sum w |v| at most.
    """
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    t = top[..., None]
    e = (d + 2) * 2.0 ** -24 * t + 2.0 ** -22 + 2.0 ** -23 * 3.0 * t
    b = u * (absv * (1 + u) + np.abs(out)) + (2 * e + 2 * 1152 * 2.0 ** -24) * absv
    if dtype != "bf16":
        b = b + 2.0 ** -25 * sumv + 2.0 ** -25  # the last: an output below 2^-14
    return b * 1.0001 + 1e-30
