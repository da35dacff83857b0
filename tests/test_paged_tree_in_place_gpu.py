"""An output over the queries is refused: row tiles are finished while others
that were split still read theirs."""
import pytest

from test_paged_tree_gpu import Case, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [0, 1, -1])
def test_out_over_the_queries_is_refused(cuda_lib, shift):
    import torch
    c = Case([(40, 4), (50, 5)], 4, 2, 64, seed=92, behind=0)
    both = torch.empty((c.total + 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    q, out = both[max(0, -shift):][:c.total], both[max(0, shift):][:c.total]
    args = [_dev(c.k, "bf16"), _dev(c.v, "bf16"), _dev(c.tables), _dev(c.lens), _dev(c.cu),
            _dev(c.parents)]
    with pytest.raises(ValueError, match="overlap"):
        cuda_lib.paged_attn_tree(q, *args, out=out)
    apart = torch.empty((2 * c.total, 4, 64), dtype=torch.bfloat16, device="cuda")
    apart[:c.total] = _dev(c.q, "bf16")
    cuda_lib.paged_attn_tree(apart[:c.total], *args, out=apart[c.total:])
    cuda_lib.check()
