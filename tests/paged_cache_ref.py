"""What the paged-cache operators compute, written out one token and one page
at a time on host arrays.  Cache elements are 16-bit patterns, so comparisons
are exact whatever value they stand for (NaN patterns among them)."""
import numpy as np

PAGE = 16


def new_caches(rng, blocks, hkv, d):
    k = rng.integers(0, 1 << 16, (blocks, hkv, d // 8, PAGE, 8), dtype=np.uint16)
    v = rng.integers(0, 1 << 16, (blocks, hkv, d, PAGE), dtype=np.uint16)
    return k, v


def tables_for(rng, lens, width=None, spare=5, fill=-1):
    """Shuffled distinct pages for rows of `lens` tokens, other entries `fill`."""
    pages = [max(0, -(-n // PAGE)) for n in lens]
    width = width or max(1, max(pages, default=1))
    blocks = sum(pages) + spare
    ids = rng.permutation(blocks)
    t = np.full((len(lens), width), fill, dtype=np.int32)
    at = 0
    for i, n in enumerate(pages):
        n = min(n, width)
        t[i, :n] = ids[at:at + n]
        at += n
    return t, blocks


def put(k, v, page, slot, key, value):
    """key, value [Hkv, D] into one slot."""
    k[page, :, :, slot, :] = key.reshape(k.shape[1], k.shape[2], 8)
    v[page, :, :, slot] = value


def write(key, value, k, v, tables, lens, cu):
    """In place; returns whether a bad page or position was met."""
    bad = False
    for i in range(len(lens)):
        lo, hi = max(int(cu[i]), 0), min(int(cu[i + 1]), key.shape[0])
        n, size = max(hi - lo, 0), max(int(lens[i]), 0)
        for j in range(n):
            p = size - n + j
            if p < 0:
                continue
            if p >= tables.shape[1] * PAGE or not 0 <= tables[i, p // PAGE] < k.shape[0]:
                bad = True
                continue
            put(k, v, tables[i, p // PAGE], p % PAGE, key[lo + j], value[lo + j])
    return bad


def accept(k, v, tables, lens, cu, accepted, num):
    """In place; returns (new lengths, draft error, page error)."""
    out, bad, page = [], False, False
    k0, v0 = k.copy(), v.copy()
    for i in range(len(lens)):
        n, size = max(int(cu[i + 1]) - max(int(cu[i]), 0), 0), max(int(lens[i]), 0)
        base = size - n
        take = max(0, min(int(num[i]), accepted.shape[1], n))
        bad |= take != num[i]
        for m in range(take):
            a = int(accepted[i, m])
            if not (a > (int(accepted[i, m - 1]) if m else -1) and m <= a < n):
                take, bad = m, True
                break
        for m in range(take):
            src, dst = base + int(accepted[i, m]), base + m
            if dst < 0 or src == dst:
                continue
            if src >= tables.shape[1] * PAGE:
                page = True
                continue
            a, b = int(tables[i, src // PAGE]), int(tables[i, dst // PAGE])
            if not (0 <= a < k.shape[0] and 0 <= b < k.shape[0]):
                page = True
                continue
            k[b, :, :, dst % PAGE] = k0[a, :, :, src % PAGE]
            v[b, :, :, dst % PAGE] = v0[a, :, :, src % PAGE]
        out.append(max(base + take, 0))
    return np.asarray(out, dtype=np.int32), bad, page


def free(tables, lens, refs, rows):
    """In place; returns whether a row or a count was bad."""
    bad = False
    for r in rows:
        if not 0 <= r < len(lens):
            bad = True
            continue
        for b in tables[r, :min(-(-int(lens[r]) // PAGE), tables.shape[1])] if lens[r] > 0 else []:
            if refs[b] <= 0:
                bad = True
            else:
                refs[b] -= 1
        lens[r] = 0
    return bad


def fork(k, v, tables, lens, refs, src, dst):
    """In place; returns (row error, out of pages)."""
    rows = len(lens)
    bad = dry = False
    named, t0, l0 = set(), tables.copy(), lens.copy()
    good = [0 <= a < rows and 0 <= b < rows for a, b in zip(src, dst)]
    sources = {a for a, g in zip(src, good) if g}
    holes = iter([b for b in range(len(refs)) if refs[b] <= 0])
    for a, b, g in zip(src, dst, good):
        if not g or b in named or b in sources or l0[b] > 0:
            bad = True
            if g:
                named.add(b)
            continue
        named.add(b)
        n = max(int(l0[a]), 0)
        full, rest = divmod(n, PAGE)
        full, rest = (full, rest) if full < tables.shape[1] else (tables.shape[1], 0)
        if rest:
            page = next(holes, None)
            if page is None:
                dry = True
                continue
            refs[page] = 1
            tables[b, full] = page
            k[page], v[page] = k[t0[a, full]], v[t0[a, full]]
        tables[b, :full] = t0[a, :full]
        for x in t0[a, :full]:
            refs[x] += 1
        lens[b] = n
    return bad, dry


def compact(k, v, tables, lens, refs):
    """Caches in place; returns (tables, refs) after the move."""
    used = int((refs > 0).sum())
    tables, refs = tables.copy(), refs.copy()
    now, top = {}, len(refs) - 1
    for b in range(used):
        if refs[b] <= 0:
            while refs[top] <= 0:
                top -= 1
            k[b], v[b], refs[b], refs[top], now[top] = k[top], v[top], refs[top], 0, b
    for r in range(len(lens)):
        for c in range(min(-(-max(int(lens[r]), 0) // PAGE), tables.shape[1])):
            tables[r, c] = now.get(int(tables[r, c]), tables[r, c])
    return tables, refs
