"""Writing behind tokens whose scale is above 2^127, the largest power of two: it becomes 2^127, and what its
codes cannot hold any more becomes the largest."""
import numpy as np
import pytest

import paged_q8_ref as ref
from test_paged_q8_gpu import back, batch, check_write, new_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_scales_above_the_largest_power_of_two(cuda_lib, kind):
    scales = [1.5 * 2.0 ** 127, np.finfo(np.float32).max, 2.0 ** 127, 1.25 * 2.0 ** 126]
    rng, lens, cu, tables, blocks = batch([(5, 4)] * 4, seed=140)
    cache = ref.new_cache(rng, blocks, 2, 64, kind)
    old = ref.decode(cache[1][tables[:, 0]], kind)  # values, as they lie
    for i, x in enumerate(scales):
        cache[2][tables[i, 0]] = cache[3][tables[i, 0]] = x
    rows = new_rows(rng, int(cu[-1]), 2, 64, "bf16")
    _, v, ks, vs = check_write(cuda_lib, rng, rows, rows, cache, tables, lens, cu, kind)
    most = ref.LARGEST[kind]
    for scale in (ks, vs):
        assert (scale.cpu().numpy()[tables[:, 0]] == 2.0 ** 127).all()
    got = ref.decode(back(v)[tables[:, 0]], kind)
    for i, x in enumerate(scales):
        mine = got[i][..., :5]
        if x == 2.0 ** 127:  # the scale stays, and so do the codes, -128 among them
            np.testing.assert_array_equal(mine, old[i][..., :5])
            continue
        want = old[i][..., :5] * (float(np.float32(x)) / 2.0 ** 127)
        cut = np.abs(want) > most
        assert (np.abs(mine[cut]) == most).all() and (cut.any() or x < 2.0 ** 127)
        np.testing.assert_array_equal(mine, ref.decode(ref.encode(np.clip(want, -most, most), kind), kind))
