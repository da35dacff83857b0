"""Tree attention with scores that 32 bits hardly hold, and the ends of the
range of its scale."""
import numpy as np
import pytest

from test_paged_tree_gpu import Case, _round, _wide

pytestmark = pytest.mark.gpu


def _one_hot_case(rows, hq, hkv, d, dtype, unit, seed):
    """Queries and keys of small whole numbers times `unit`: scores are exact in
    32 bits, and those of a row equal or far apart."""
    c = Case(rows, hq, hkv, d, dtype, seed=seed)
    rng = np.random.default_rng(seed)
    c.q = _round(rng.integers(-3, 4, c.q.shape) * unit, dtype)
    c.k = _round(rng.integers(-3, 4, c.k.shape) * unit, dtype)
    return c


@pytest.mark.parametrize("rows", [[(45, 7), (130, 1), (0, 3)], [(700, 20)], [(6000, 3), (9, 2)],
                                  [(300, 2)] * 200], ids=range(4))
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (16, 2, 128), (4, 1, 256), (129, 1, 128)])
@pytest.mark.parametrize("dtype,unit,scale", [
    ("bf16", 1.0, 2.0 ** 126),      # the largest scale: scores past 32 bits
    ("fp16", 1.0, 2.0 ** 126),
    ("fp16", 1.0, 2.0 ** 30),
    ("fp16", 8192.0, None),         # ordinary scale, scores up to 2^34
    ("bf16", 2.0 ** 40, None),      # up to 2^88
    ("bf16", 2.0 ** -40, 2.0 ** 120),
    ("fp16", 512.0, None),          # up to 2^24
    ("bf16", 64.0, None),           # up to 2^18
])
def test_large_scores(cuda_lib, rows, hq, hkv, d, dtype, unit, scale):
    """A row's largest score takes all the weight, keys that share it equal parts.

    Bound: the weights of the k keys that share a maximum are equal and all
    others 0.  They are rounded once, as the output is, and their sum and that of
    the values in 32 bits, in k steps each.
    """
    if dtype == "fp16" and unit > 1 and len(rows) == 200:
        pytest.skip("the same as the largest scale")
    c = _one_hot_case(rows, hq, hkv, d, dtype, unit, 63)
    kw = {} if scale is None else {"scale": scale}
    got = _wide(c.run(cuda_lib, **kw), dtype)
    out, absv, sumv, top = c.want(scale)
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    k = 64  # as many of the keys of small whole numbers hardly share a maximum
    b = u * (np.abs(out) + absv) * 1.01 + 2 * k * 2.0 ** -24 * absv
    b += 0 if dtype == "bf16" else 2.0 ** -25  # an output below 2^-14
    assert np.isfinite(got).all()
    over = np.abs(got - out) > b
    assert not over.any(), (int(over.sum()), np.argwhere(over)[:4].tolist())


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "fp16")])
def test_tiny_scale(cuda_lib, d, dtype):
    """The smallest scale: all weights are equal."""
    Case([(45, 7), (300, 2)], 4, 2, d, dtype, seed=64).check(cuda_lib, scale=2.0 ** -126)
