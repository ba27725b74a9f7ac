"""Prefix-shared decode at more of the layouts, block sizes and plans that it takes:
every head count and group size of the decode's limits, large blocks, plans that a
scheduler fills itself, batches without a token."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prefix_attn import BF16, DEV, F32, Case, _d, zp  # noqa: F401 (zp is a fixture)

pytestmark = pytest.mark.gpu

LAYOUTS = ([(h_kv * G, h_kv, d, 16, BF16) for h_kv in (1, 2, 4, 8) for G in (1, 2, 4, 8) for d in (64, 128)] +
           [(64, 16, 128, 16, BF16), (128, 16, 64, 16, BF16)] +
           [(h_kv * G, h_kv, d, 16, F32) for h_kv, d in ((2, 64), (4, 128), (8, 64), (16, 64)) for G in (4, 8)] +
           [(8, 2, 128, 128, BF16), (8, 1, 64, 256, BF16), (8, 2, 64, 128, F32), (32, 4, 128, 256, F32)])


@pytest.mark.parametrize("layout", LAYOUTS, ids=["%dq%dkv%d_b%d_%s" % (*x[:4], "bf16" if x[4] is BF16 else "f32") for x in LAYOUTS])
def test_layouts(zp, layout):  # noqa: F811
    b = layout[3]
    big = b > 64
    c = Case(zp, 501, layout, [5, 12, 2], [2, 3, 1] if big else [9, 17, 4], (1, 3 * b), 3, 1)
    c.score_rows(502, max(1, b // 3))
    c.check(*c.run(zp))


@pytest.mark.parametrize("layout", [(32, 8, 128, 16, BF16), (16, 4, 64, 16, BF16), (16, 4, 64, 16, F32)], ids=["d128", "d64", "f32"])
def test_a_plan_filled_by_the_caller(zp, layout):  # noqa: F811
    """Groups of one, more of them than the joining kernel scans itself, and groups that share less than they could."""
    c = Case(zp, 511, layout, [4, 6], [10, 30], (1, 60), 400, 2)
    c.score_rows(512, 16)
    groups = [([s], max(int(c.lens[s]) - 1, 0) // c.b) for s in np.nonzero(c.group == -1)[0]]  # each its own blocks
    groups += [(np.nonzero(c.group == 0)[0].tolist(), 3), (np.nonzero(c.group == 1)[0].tolist()[1:], 30)]
    groups = sorted((g for g in groups if g[1] > 0), key=lambda g: g[0][0])
    assert len(groups) > 256
    c.plan = zp.prefix_plan(c.B)
    pre, start, members, blocks = np.zeros(c.B), np.zeros(c.B + 1), np.full(c.B, -1), np.zeros(c.B)
    at = 0
    for i, (mem, p) in enumerate(groups):
        members[at:at + len(mem)] = mem
        blocks[i], pre[mem] = p, p * c.b
        at += len(mem)
        start[i + 1:] = at
    for name, v in (("prefix_lens", pre), ("group_start", start), ("members", members), ("group_blocks", blocks)):
        getattr(c.plan, name).copy_(_d(v))
    c.plan.n_groups.fill_(len(groups))
    c.check(*c.run(zp))


@pytest.mark.parametrize("layout", [(32, 8, 128, 16, BF16), (8, 2, 64, 16, F32)], ids=["bf16", "f32"])
def test_no_entry_has_a_token(zp, layout):  # noqa: F811
    """Every L is 0, with the plan of a step before: nothing is written."""
    c = Case(zp, 521, layout, [4, 9], [10, 3], (1, 60), 2)
    c.score_rows(522, 16)
    c.ld = torch.zeros_like(c.ld)
    out, S = c.run(zp)
    assert bool((out == 7.0).all()) and torch.equal(S, torch.from_numpy(c.S0).to(DEV))


@pytest.mark.parametrize("layout", [(32, 8, 128, 16, BF16), (8, 2, 64, 16, F32)], ids=["bf16", "f32"])
def test_one_sequence(zp, layout):  # noqa: F811
    """A batch of one, with a plan of one group of one, and one token behind the prefix."""
    c = Case(zp, 531, layout, [1], [50], (1, 1))
    c.score_rows(532, 16)
    c.rows[:] = 1
    c.plan.prefix_lens.fill_(50 * 16)
    c.plan.n_groups.fill_(1)
    c.plan.group_start.copy_(_d([0, 1]))
    c.plan.members.fill_(0)
    c.plan.group_blocks.fill_(50)
    c.check(*c.run(zp))
