"""Prefix-shared decode where a CTA takes many short items one after another: the
queries of the next item follow the records of the last in the same shared memory."""
import pytest
import torch

from tests.test_gpu_prefix_attn import BF16, F32, Case, zp  # noqa: F401 (zp is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(32, 8, 128, 16, BF16), (16, 2, 128, 16, BF16), (32, 4, 64, 16, BF16), (32, 8, 128, 16, F32)],
                         ids=["g4", "g8", "d64", "f32"])
@pytest.mark.parametrize("scored", [False, True])
def test_many_items_per_cta(zp, heads, scored):  # noqa: F811
    """380 groups, one to three tiles each, some with more rows than one stream has: against the oracle, and the
    same bits every time."""
    sizes = [2 + (i % 7 == 0) * 3 + (i % 95 == 0) * 40 for i in range(380)]
    c = Case(zp, 201, heads, sizes, [1 + (5 * i) % 24 for i in range(380)], (1, 20), 3, 1)
    if scored:
        c.score_rows(202, 11)
    out, S = c.run(zp)
    c.check(out, S)
    for _ in range(8):
        out2, S2 = c.run(zp)
        assert torch.equal(out, out2) and (S is None or torch.equal(S, S2))
