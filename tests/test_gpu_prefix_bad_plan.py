"""Plans and tables that name what is not there, in prefix-shared decode: recorded, and
what the bad entry does not touch keeps its value."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prefix_attn import BF16, DEV, F32, HEADS, Case, _d, zp  # noqa: F401 (zp is a fixture)

pytestmark = pytest.mark.gpu


def _case(zp, heads, scored=True):  # noqa: F811
    c = Case(zp, 401, HEADS[heads], [6, 9, 3], [7, 12, 5], (1, 40), 3)
    if scored:
        c.score_rows(402, c.b)
    return c


def _call(zp, c):  # noqa: F811
    out, S = torch.full_like(c.qd, 7.0), torch.from_numpy(c.S0).to(DEV)
    zp.zp_prefix_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, c.plan, out, score_accum=S, window=c.window,
                             score_rows=_d(c.rows))
    torch.cuda.synchronize()
    return out, S, zp.zp_device_status()


@pytest.mark.parametrize("heads", ["qwen", "g8d64", "tiny32"])
@pytest.mark.parametrize("place", ["first", "second", "last"])
def test_the_other_members_of_a_bad_one(zp, heads, place):  # noqa: F811
    """A member outside the batch, wherever it stands in its group: every other entry keeps its bits."""
    c = _case(zp, heads)
    good, S_good, status = _call(zp, c)
    assert status == (0, 0)
    start = c.plan.group_start.tolist()
    g = 1  # neither the first group nor the last
    at = {"first": start[g], "second": start[g] + 1, "last": start[g + 1] - 1}[place]
    lost = int(c.plan.members[at])
    c.plan.members[at] = -3 if place == "last" else c.B + 7
    out, S, status = _call(zp, c)
    assert status == (7, 0x142)
    rest = torch.arange(c.B, device=DEV) != lost
    assert torch.equal(out[rest], good[rest])
    kept = torch.ones(S.shape[0], dtype=torch.bool)
    if c.rows[lost] >= 0:
        kept[int(c.rows[lost])] = False
    assert torch.equal(S[kept.to(DEV)], S_good[kept.to(DEV)])


@pytest.mark.parametrize("heads", ["qwen", "g8d64", "tiny32"])
def test_a_bad_shared_block_stays_in_its_group(zp, heads):  # noqa: F811
    """A block id outside the cache in one group's prefix: the entries outside that group keep their bits."""
    c = _case(zp, heads)
    good, S_good, _ = _call(zp, c)
    bad = np.nonzero(c.group == 1)[0]
    for s, block in zip(bad, [-1, c.n_total, 2 ** 31 - 1, -2 ** 31] * 3):
        c.td[int(s), 4] = block
    out, S, status = _call(zp, c)
    assert status == (7, 0x143)
    rest = np.setdiff1d(np.arange(c.B), bad)
    assert torch.equal(out[_d(rest).long()], good[_d(rest).long()])
    rows = np.setdiff1d(np.arange(S.shape[0]), c.rows[bad])
    assert torch.equal(S[_d(rows).long()], S_good[_d(rows).long()])


@pytest.mark.parametrize("h_q,h_kv,dtype", [(8, 8, F32), (8, 4, F32), (16, 16, BF16), (32, 16, BF16), (12, 4, BF16), (4, 1, F32)])
def test_head_layouts_that_are_refused(zp, h_q, h_kv, dtype):  # noqa: F811
    """The decode's limits: groups of 1 and 2 with bf16 caches of up to 8 kv heads only."""
    desc = zp.cache_desc(h_q, h_kv, 64, 16, 8, dtype)
    with pytest.raises(zp.ZPError) as e:
        zp.zp_prefix_decode_workspace_size(desc, 2, 4)
    assert e.value.status == 2
    q = torch.zeros(2, h_q, 64, dtype=dtype, device=DEV)
    K = torch.zeros(8, 16, h_kv, 64, dtype=dtype, device=DEV)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    with pytest.raises(zp.ZPError) as e:
        zp.zp_prefix_decode_attn(desc, q, K, K, _d(np.zeros((2, 4))), _d([3, 3]), zp.prefix_plan(2), torch.empty_like(q),
                                 workspace=ws)
    assert e.value.status == 2


@pytest.mark.parametrize("heads", ["qwen", "tiny32"])
def test_outputs_over_the_queries(zp, heads):  # noqa: F811
    """Unscored calls may write their outputs over q; scored ones are refused."""
    c = _case(zp, heads)
    S = torch.from_numpy(c.S0).to(DEV)
    good = torch.empty_like(c.qd)
    zp.zp_prefix_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, c.plan, good)
    with pytest.raises(zp.ZPError):
        zp.zp_prefix_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, c.plan, c.qd, score_accum=S, window=c.b, score_rows=_d(c.rows))
    zp.zp_prefix_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, c.plan, c.qd)
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0) and torch.equal(c.qd, good)
