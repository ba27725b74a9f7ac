"""Prefix-shared decode at the ends of the range of its values, against the decode of
every sequence alone: logits far from zero or of -infinity, NaN in queries and keys."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prefix_attn import DEV, HEADS, Case, _d, zp  # noqa: F401 (zp is a fixture)

pytestmark = pytest.mark.gpu
INF = float("inf")
BLOCKS = {"all": range(37), "first": range(24), "some": range(5, 37, 3)}  # of the third group's 37


def _case(zp, heads, seed=301):  # noqa: F811
    c = Case(zp, seed, HEADS[heads], [7, 3, 40], [20, 3, 37], (1, 50), 2)
    c.score_rows(seed + 1, c.b)
    return c


def _alone(zp, c):  # noqa: F811
    out = torch.full_like(c.qd, 7.0)
    S = torch.from_numpy(c.S0).to(DEV)
    zp.zp_paged_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, out, score_accum=S, window=c.window, score_rows=_d(c.rows))
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    return out, S


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("low", [-1e5, -1e9, -1e30, "min"])
@pytest.mark.parametrize("blocks", BLOCKS)
def test_logits_far_below(zp, heads, blocks, low):  # noqa: F811
    """Shared tokens whose logits are so low that they weigh nothing (a key channel set to the type's lowest
    value among them): the sequences' other tokens."""
    c = _case(zp, heads)
    c.qd[..., 0] = 1.0
    g2 = int(np.nonzero(c.group == 2)[0][0])
    c.Kd[_d(c.table[g2, list(BLOCKS[blocks])]).long(), :, :, 0] = torch.finfo(c.dtype).min if low == "min" else low
    out, S = c.run(zp)
    alone, S_alone = _alone(zp, c)
    # both within 2^-8 (sum p |v| + |out|) of the same value; |v| is below 6
    torch.testing.assert_close(out.float(), alone.float(), rtol=2.0 ** -7, atol=6 * 2.0 ** -7)
    torch.testing.assert_close(S, S_alone, rtol=1e-4, atol=1e-12)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("big", [2.0 ** 40, -2.0 ** 40, 2.0 ** 100, -2.0 ** 100])
def test_equal_logits_far_from_zero(zp, heads, big):  # noqa: F811
    """A key channel that drowns the others: every logit of a sequence is the same, its output the mean of its values."""
    c = _case(zp, heads)
    c.qd[..., 0] = 1.0
    c.Kd[..., 0] = big
    out, S = c.run(zp)
    V = c.V.double().numpy()
    G = c.h_q // c.h_kv
    for s in np.nonzero(c.lens > 0)[0]:
        L = int(c.lens[s])
        t = np.arange(L)
        v = V[c.table[s, t // c.b], t % c.b]
        want, absv = (np.repeat(x.mean(0), G, axis=0) for x in (v, np.abs(v)))
        # probabilities of equal logits are equal: sums of n terms, a reciprocal, and the output's half step
        tol = (2 * L + 8) * 2.0 ** -24 * absv + torch.finfo(c.dtype).eps / 2 * 1.01 * np.abs(want)
        assert (np.abs(out[int(s)].double().cpu().numpy() - want) <= tol).all()
    assert bool(torch.isfinite(S).all()) and float(S.max()) <= 1.0 + (c.b - 1)  # S0 < 1, one step's share of at most 1


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("which", ["first", "last"])
def test_a_bad_query_head_stays_alone(zp, heads, which):  # noqa: F811
    """NaN in one q head of a kv head: its own output is NaN, every other head keeps its bits."""
    c = _case(zp, heads)
    good, _ = c.run(zp)
    G = c.h_q // c.h_kv
    h = 0 if which == "first" else G - 1
    for s in np.nonzero(c.group >= 0)[0][::3]:
        c.qd[int(s), h] = float("nan")
    bad = torch.isnan(c.qd).any(-1)
    out, _ = c.run(zp)
    assert bool(torch.isnan(out[bad]).all())
    assert torch.equal(out[~bad], good[~bad])


@pytest.mark.parametrize("heads", HEADS)
def test_bad_keys_reach_their_readers(zp, heads):  # noqa: F811
    """NaN in the keys of one kv head, in a whole prefix and in one private token: NaN where the decode of every
    sequence alone has it, and the other heads keep their bits."""
    c = _case(zp, heads)
    good, _ = c.run(zp)
    g0 = np.nonzero(c.group == 0)[0]
    lone = int(np.nonzero(c.group == 2)[0][1])
    c.Kd[_d(c.table[g0[0], :20]).long(), :, 0] = float("nan")
    L = int(c.lens[lone])
    c.Kd[int(c.table[lone, (L - 1) // c.b]), (L - 1) % c.b, c.h_kv - 1] = float("nan")
    out, _ = c.run(zp)
    ref, _ = _alone(zp, c)
    nan = torch.isnan(ref.float())
    assert bool(nan.any()) and torch.equal(torch.isnan(out.float()), nan)
    assert torch.equal(out[~nan], good[~nan])


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("blocks", BLOCKS)
def test_logits_of_minus_infinity(zp, heads, blocks):  # noqa: F811
    """Shared tokens with a logit of -infinity, from the first tile on or in the middle of it, or all of them:
    the bits of the same call with logits so low that their weights are 0."""
    c = _case(zp, heads)
    c.qd[..., 0] = 1.0
    g2 = int(np.nonzero(c.group == 2)[0][0])
    at = _d(c.table[g2, list(BLOCKS[blocks])]).long()
    got = []
    for low in (-1e30, -INF):
        c.Kd[at, :, :, 0] = low
        got.append(c.run(zp))
    (out_low, S_low), (out, S) = got
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(S).all())
    assert torch.equal(out, out_low) and torch.equal(S, S_low)


@pytest.mark.parametrize("heads", HEADS)
def test_a_sequence_with_nothing_but_minus_infinity(zp, heads):  # noqa: F811
    """Every logit of a sequence -infinity: zeros, as the decode of the sequence alone gives; the others are not touched."""
    c = _case(zp, heads)
    c.qd[..., 0] = 1.0
    good, _ = c.run(zp)
    s = int(np.nonzero(c.group == 1)[0][1])
    c.qd[s] = 0.0
    c.qd[s, :, 0] = 1.0
    L, p = int(c.lens[s]), 3 * c.b
    for t in range(p, L):
        c.Kd[int(c.table[s, t // c.b]), t % c.b, :, 0] = -INF
    others = torch.arange(c.B, device=DEV) != s
    c.Kd[_d(c.table[s, :3]).long(), :, :, 0] = -INF
    mates = torch.from_numpy(np.nonzero(c.group == 1)[0]).to(DEV)
    others[mates] = False  # they lose the prefix
    out, _ = c.run(zp)
    alone, _ = _alone(zp, c)
    assert torch.equal(out[s], alone[s]) and not bool(out[s].any())
    assert torch.equal(out[others], good[others])
    torch.testing.assert_close(out[mates].float(), alone[mates].float(), rtol=2.0 ** -7, atol=6 * 2.0 ** -7)
