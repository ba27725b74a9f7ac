"""Decode over a 4-bit cache with few sequences: pairs that one CTA or a cluster of CTAs has, and the same
sequences in tables so wide that the units of all are cut evenly."""
import numpy as np
import pytest
import torch

from test_gpu_q4_decode import SHAPES, Case, _status, zp  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = 4096  # more columns than any cluster takes: 16 * 16 * 3 units of 32 tokens are 1536 blocks of 16


@pytest.mark.parametrize("extra", [0, 60, WIDE])
@pytest.mark.parametrize("dtype,h_q,h_kv,d,group,b", SHAPES)
def test_widths(zp, dtype, h_q, h_kv, d, group, b, extra):  # noqa: F811
    c = Case(zp, [33, 0, 1, 700], dtype, h_q, h_kv, d, group, b, seed=2, extra=extra)
    c.check(c.run())


@pytest.mark.parametrize("extra", [0, WIDE])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 31, 32, 33, 511, 512, 513, 1025, 2047, 4099, 9000])
def test_one_sequence(zp, dtype, L, extra):  # noqa: F811
    """Clusters of every size, with CTAs that have no unit, one warp each, and all warps."""
    c = Case(zp, [L], dtype, 8, 1, 128, 32, 16, seed=L, extra=extra)
    c.check(c.run())


@pytest.mark.parametrize("h_q,h_kv", [(8, 8), (16, 4), (16, 2)])
def test_long_and_short(zp, h_q, h_kv):  # noqa: F811
    c = Case(zp, [2500, 0, 40, 1], "bf16", h_q, h_kv, 64, 64, 16, seed=6)
    c.check(c.run())


def test_same_bits_again(zp):  # noqa: F811
    c = Case(zp, [1800, 5, 900], "bf16", 8, 2, 128, 32, 16, seed=3)
    want = c.run()
    for _ in range(5):
        assert torch.equal(c.run(), want)


@pytest.mark.parametrize("extra", [1, WIDE])
def test_bad_blocks_and_lengths(zp, extra):  # noqa: F811
    """Tokens of bad blocks weigh nothing, also where a whole CTA has no others; lengths are cut to the table."""
    c = Case(zp, [1500, 40, 0], "bf16", 8, 2, 128, 32, 16, seed=8, extra=extra)
    want = c.run()
    table = c.table.copy()
    c.table[1, :] = -1                     # nothing is left
    c.table[0, 40:60] = c.n_total          # tokens 640 to 959
    out = c.run()
    assert _status(zp) == (7, 0x159)
    assert (out[1] == 0).all() and (out[2] == 9.0).all()
    keep = c.table[0, :94]
    good = np.flatnonzero((keep >= 0) & (keep < c.n_total))
    short = Case(zp, [1500 - 320], "bf16", 8, 2, 128, 32, 16, seed=8)
    short.K, short.V, short.q, short.n_total, short.desc = c.K, c.V, c.q[:1], c.n_total, c.desc
    short.table = np.concatenate([keep[good], [-1]])[None].astype(np.int32)
    want0, tol, _, _ = short.reference(0)
    assert (np.abs(out[0].double().numpy() - want0) <= tol).all()
    c.table = table
    c.lens = np.array([1500, 40, -3])
    assert torch.equal(c.run(), want)
    assert _status(zp) == (7, 0x158)


def test_streams_and_graph(zp):  # noqa: F811
    """Captured and replayed with lengths that grow, beside calls on another stream."""
    c = Case(zp, [1200, 300], "bf16", 8, 2, 128, 32, 16, seed=9)
    args = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (c.K, c.V, c.table)]
    q, lens = c.q.cuda(), torch.tensor([1200, 300], dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(q), torch.empty_like(q)
    n = zp.zp_q4_decode_workspace_size(c.desc, 2, c.table.shape[1], scored=False)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    zp.zp_q4_decode_attn(c.desc, q, *args, lens, a, workspace=ws[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zp.zp_q4_decode_attn(c.desc, q, *args, lens, a, workspace=ws[0])
    for l0, l1 in ((1200, 300), (1, 0), (513, 299), (1200, 17)):
        lens.copy_(torch.tensor([l0, l1], dtype=torch.int32))
        a.fill_(9.0)
        b.fill_(9.0)
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            graph.replay()
            zp.zp_q4_decode_attn(c.desc, q, *args, lens, b, workspace=ws[1], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
        c.lens = np.array([l0, l1])
        c.check(a.cpu())



@pytest.mark.parametrize("extra", [0, 60, WIDE])
@pytest.mark.parametrize("dtype,h_q,h_kv,d,group,b", SHAPES)
@pytest.mark.parametrize("window", [4, 0])
def test_score(zp, dtype, h_q, h_kv, d, group, b, window, extra):  # noqa: F811
    """Written on the first step of the window, added on the others, left alone without a row, off the window and
    behind the newest token."""
    w = window or b
    lens = np.array([b - w + 1, 12 * b, 2 * b - w, 8 * b])
    c = Case(zp, lens, dtype, h_q, h_kv, d, group, b, seed=w, extra=extra)
    rows = np.array([3, 1, 2, -1], dtype=np.int32)
    S0 = np.random.default_rng(1).uniform(0.5, 1.0, size=(4, h_kv, c.table.shape[1] * b)).astype(np.float32)
    S = torch.from_numpy(S0).cuda()
    c.check(c.run(w, S, torch.from_numpy(rows).cuda()))
    got, want, tol = S.cpu().numpy().astype(np.float64), S0.astype(np.float64), np.zeros(S0.shape)
    for s, L in enumerate(lens):
        P = int(L) - 1
        if rows[s] < 0 or P % b < b - w:
            continue
        _, _, prob, ptol = c.reference(s)
        new = prob.reshape(h_kv, -1, L).max(1) / w
        rel = ptol.reshape(h_kv, -1).max(1)[:, None] + 2.0 ** -21
        old = np.where((P % b == b - w) | (np.arange(L) == P), 0.0, want[rows[s], :, :L])
        want[rows[s], :, :L] = old + new
        tol[rows[s], :, :L] = rel * new + 2.0 ** -24 * (old + new) * (old > 0)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [16, 512, 1040, 2048, 9008])
def test_score_of_one(zp, dtype, L):  # noqa: F811
    """Clusters of every size; the same scores from the even cut, to rounding."""
    S = []
    for extra in (0, WIDE):
        c = Case(zp, [L], dtype, 8, 1, 128, 32, 16, seed=L, extra=extra)
        S.append(torch.full((1, 1, c.table.shape[1] * 16), 7.0, device="cuda"))
        c.check(c.run(1, S[-1]))
        assert (S[-1][..., L:] == 7.0).all()
    _, _, prob, ptol = c.reference(0)
    for x in S:
        got = x[0, 0, :L].cpu().double().numpy()
        assert (np.abs(got - prob.max(0)) <= (ptol.max() + 2.0 ** -21) * prob.max(0)).all()
