"""bf16 outputs of the decode over a 4-bit cache within the bound that the roundings of its weights give (q4_fine.py):
sequences in one CTA, in clusters and cut over all, steps of one size and of many."""
import numpy as np
import pytest
import torch

from q4_fine import Fine
from test_gpu_q4_decode import zp  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = 4096  # table columns past every cluster: the units of all pairs are cut evenly
KINDS = ["near", "flat", "up", "down", "far"]


@pytest.mark.parametrize("extra", [1, WIDE])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,group", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64)])
def test_few_tokens(zp, d, group, kind, extra):  # noqa: F811
    c = Fine(zp, [1, 2, 10, 31, 32, 34, 64, 100], 8, 2, d, group, kind=kind, extra=extra, seed=d + group)
    c.check(c.run())


@pytest.mark.parametrize("h_q,h_kv", [(8, 8), (15, 3), (8, 1), (32, 8)])
@pytest.mark.parametrize("spread", [0.4, 40.0])
def test_heads(zp, h_q, h_kv, spread):  # noqa: F811
    c = Fine(zp, [50, 0, 7, 250], h_q, h_kv, 64, 32, seed=h_q, spread=spread)
    c.check(c.run())


@pytest.mark.parametrize("extra", [1, WIDE])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens", [[2600], [1024, 40], [700, 3, 0, 500], [64] * 100])
def test_splits(zp, lens, kind, extra):  # noqa: F811
    """Every token's weight over the cuts between warps, CTAs and clusters."""
    c = Fine(zp, lens, 4, 2, 64, 32, seed=len(lens), kind=kind, extra=extra)
    c.check(c.run())


def test_blocks_of_64(zp):  # noqa: F811
    c = Fine(zp, [90, 300, 33], 8, 2, 128, 32, b=64, seed=1)
    c.check(c.run())


def test_scored(zp):  # noqa: F811
    c = Fine(zp, [49, 321, 33], 16, 4, 128, 32, seed=2)
    S = torch.zeros(3, 4, c.table.shape[1] * 16, device="cuda")
    c.check(c.run(16, S))
    for s in range(3):
        _, _, prob, ptol = c.reference(s)
        L = int(c.lens[s])
        want = prob.reshape(4, 4, L).max(1) / 16
        assert (np.abs(S[s, :, :L].cpu().double().numpy() - want) <= (ptol.max() + 2.0 ** -18) * want).all()
