"""Decode attention behind shared prefixes against the 64-bit oracle: outputs
and window scores of groups of many shapes, and the calls around them (stale
plans, captured graphs, streams, entries that are skipped)."""
import numpy as np
import pytest
import torch

from tests.prefix_util import attention_bounds, make_groups, plan_ref, window_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    return m


def _d(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Case:
    def __init__(self, zp, seed, heads, sizes, blocks, own, lone=0, zero=0, lens=None):
        self.h_q, self.h_kv, self.d, self.b, self.dtype = heads
        self.lens, self.table, self.group, self.n_total = make_groups(seed, sizes, blocks, own, self.b, lone, zero)
        if lens is not None:
            self.lens = np.asarray(lens(self.lens), np.int32)
        g = torch.Generator().manual_seed(seed)
        self.B = len(self.lens)
        mk = lambda *s: torch.randn(*s, generator=g).to(self.dtype)  # noqa: E731
        self.K, self.V = mk(self.n_total, self.b, self.h_kv, self.d), mk(self.n_total, self.b, self.h_kv, self.d)
        self.q = mk(self.B, self.h_q, self.d)
        self.desc = zp.cache_desc(self.h_q, self.h_kv, self.d, self.b, self.n_total, self.dtype)
        self.Kd, self.Vd, self.qd, self.td, self.ld = (self.K.to(DEV), self.V.to(DEV), self.q.to(DEV), _d(self.table),
                                                       _d(self.lens))
        self.plan = zp.prefix_plan(self.B)
        zp.zp_prefix_plan(self.desc, self.td, self.ld, self.plan)
        self.S0 = None

    def score_rows(self, seed, window):
        rng = np.random.default_rng(seed)
        self.rows = rng.permutation(self.B + 2)[:self.B]
        self.rows[rng.random(self.B) < 0.15] = -1
        self.S0 = rng.random((self.B + 2, self.h_kv, self.table.shape[1] * self.b)).astype(np.float32)
        self.window = window

    def run(self, zp, **kw):
        out = torch.full_like(self.qd, 7.0)
        S = None
        if self.S0 is not None:
            S = torch.from_numpy(self.S0).to(DEV)
            kw.update(score_accum=S, window=self.window, score_rows=_d(self.rows))
        zp.zp_prefix_decode_attn(self.desc, self.qd, self.Kd, self.Vd, self.td, self.ld, self.plan, out, **kw)
        torch.cuda.synchronize()
        assert zp.zp_device_status() == (0, 0)
        return out, S

    def check(self, out, S=None):
        f = lambda t: t.float().numpy()  # noqa: E731
        table = np.maximum(self.table, 0)
        live = np.nonzero(self.lens > 0)[0]
        ref, tol, probs, rel = attention_bounds(f(self.q)[live], f(self.K), f(self.V), table[live], self.lens[live],
                                                self.dtype == BF16)
        got = out.float().cpu().numpy().astype(np.float64)
        assert (got[self.lens == 0] == 7.0).all()  # skipped entries keep their rows
        bad = np.abs(got[live] - ref) - tol
        assert (bad <= 0).all(), "off by %g of %g" % ((bad + tol).max(), tol[np.unravel_index(bad.argmax(), bad.shape)])
        if S is not None:
            want = window_ref(probs, self.lens[live], None, self.S0.astype(np.float64), self.rows[live], self.h_kv,
                              self.b, self.window)
            # the probability's bound, and the half steps of the product by 1/w and of the sum with the row
            np.testing.assert_allclose(S.cpu().numpy(), want, rtol=rel + 2.0 ** -22, atol=1e-30)


HEADS = {
    "qwen": (32, 8, 128, 16, BF16), "g8": (16, 2, 128, 16, BF16), "g8d64": (32, 4, 64, 32, BF16), "g4d64": (16, 4, 64, 64, BF16),
    "g2": (8, 4, 128, 16, BF16), "g1": (8, 8, 64, 16, BF16), "one_head": (4, 1, 128, 16, BF16), "wide": (64, 16, 64, 16, BF16),
    "tiny32": (8, 2, 64, 16, F32), "qwen32": (32, 8, 128, 16, F32), "g8_32": (16, 2, 128, 32, F32)}

GROUPS = [
    # sizes, prefix blocks, private tokens, lone, zero
    ("pair", [2], [1], (1, 1), 0, 0),
    ("one_group", [5], [9], (1, 40), 0, 0),
    ("mixed", [3, 17, 2], [21, 3, 40], (1, 70), 3, 2),
    ("wide_group", [70], [13], (1, 33), 1, 0),
    ("none", [], [], (1, 60), 5, 1),
]


@pytest.mark.parametrize("shape", GROUPS, ids=[g[0] for g in GROUPS])
@pytest.mark.parametrize("heads", HEADS)
def test_matches_oracle(zp, heads, shape):
    _, sizes, blocks, own, lone, zero = shape
    c = Case(zp, 11 + len(sizes), HEADS[heads], sizes, blocks, own, lone, zero)
    c.check(*c.run(zp))


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("heads,sizes,blocks", [
    ("wide", [66, 2, 3], [257, 70, 1]),  # few CTAs per head: two items of many tiles, and starts that a cut falls into
    ("qwen", [65, 9], [129, 64]),
    ("g8d64", [33, 40], [35, 150]),
    ("qwen32", [17, 5], [40, 70]),
])
def test_long_items(zp, heads, sizes, blocks, scored):
    """Prefixes of many tiles in several row tiles: CTAs that end one item and begin another."""
    c = Case(zp, 23, HEADS[heads], sizes, blocks, (1, 40), 1, 0)
    if scored:
        c.score_rows(3, HEADS[heads][3])
    c.check(*c.run(zp))


@pytest.mark.parametrize("window", [1, 5, 16])
@pytest.mark.parametrize("heads", HEADS)
def test_scored(zp, heads, window):
    """Every phase of the window: off it, its first row (written), later rows (added); entries without a row."""
    b = HEADS[heads][3]
    c = Case(zp, 5, HEADS[heads], [6, 9], [9, 12], (1, 3 * b), 4, 1,
             lens=lambda n: np.where((n > 0) & (np.arange(len(n)) % 3 == 0), (n // b) * b + b - window + 1, n))
    c.lens = np.minimum(c.lens, (c.table >= 0).sum(1) * b).astype(np.int32)
    c.ld = _d(c.lens)
    zp.zp_prefix_plan(c.desc, c.td, c.ld, c.plan)
    c.score_rows(3, window)
    c.check(*c.run(zp))


@pytest.mark.parametrize("heads", ["qwen", "g8d64", "tiny32"])
def test_long_prefix_few_rows(zp, heads):
    """A prefix far longer than the batch: every CTA takes a piece of it and the pieces are joined."""
    c = Case(zp, 21, HEADS[heads], [3], [400], (1, 200))
    c.score_rows(22, c.b)
    c.check(*c.run(zp))


@pytest.mark.parametrize("heads", ["qwen", "qwen32"])
def test_many_groups(zp, heads):
    c = Case(zp, 23, HEADS[heads], [2] * 60 + [7, 40], [1 + i % 9 for i in range(62)], (1, 40), 10, 3)
    c.score_rows(24, 7)
    c.check(*c.run(zp))


def test_large_logits(zp):
    """Logits far from zero (a row maximum that keeps rising, attention sinks): no overflow, no lost tail."""
    c = Case(zp, 31, HEADS["qwen"], [9], [40], (1, 60))
    K = c.K.float()
    first = c.table[int(c.plan.members[0])]
    for i in range(40):
        K[first[i]] *= 0.05 * (i + 1)
    K[first[0], 0] *= 200
    c.K = K.to(BF16)
    c.Kd = c.K.to(DEV)
    c.score_rows(32, 16)
    c.check(*c.run(zp))


def test_equals_the_decode_without_sharing(zp):
    c = Case(zp, 41, HEADS["qwen"], [30, 4], [33, 70], (1, 300), 6, 2)
    c.score_rows(42, 16)
    out, S = c.run(zp)
    S2 = torch.from_numpy(c.S0).to(DEV)
    out2 = torch.full_like(c.qd, 7.0)
    zp.zp_paged_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, out2, score_accum=S2, window=16, score_rows=_d(c.rows))
    torch.cuda.synchronize()
    # both within 2^-8 (sum p |v| + |out|) of the same value; |v| is below 6
    torch.testing.assert_close(out.float(), out2.float(), rtol=2.0 ** -7, atol=6 * 2.0 ** -7)
    torch.testing.assert_close(S, S2, rtol=1e-4, atol=1e-12)


def test_a_plan_serves_while_sequences_grow(zp):
    """The plan of step 0 used for later steps, one with a member that restarted below its prefix, one that stops."""
    c = Case(zp, 51, HEADS["qwen"], [6, 3], [5, 8], (20, 40), 2)
    c.lens = c.lens - 3
    c.lens[np.nonzero(c.group == 0)[0][2]] = 30   # inside its group's prefix: decoded alone
    c.lens[np.nonzero(c.group == 1)[0][1]] = 0    # no token this step
    for _ in range(3):
        c.ld = _d(c.lens)
        c.check(*c.run(zp))
        c.lens = np.where(c.lens > 0, c.lens + 1, 0).astype(np.int32)


def test_empty_batch_and_empty_plan(zp):
    c = Case(zp, 61, HEADS["qwen"], [4], [6], (1, 40))
    c.plan = zp.prefix_plan(c.B)  # no groups: the plain decode
    c.check(*c.run(zp))
    e = zp.prefix_plan(0)
    zp.zp_prefix_decode_attn(c.desc, c.qd[:0], c.Kd, c.Vd, c.td[:0], c.ld[:0], e, torch.empty_like(c.qd[:0]))


def test_same_bits_again_and_on_another_stream(zp):
    c = Case(zp, 71, HEADS["qwen"], [37], [60], (1, 400), 3)
    c.score_rows(72, 16)
    out, S = c.run(zp)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for stream in (None, st):
        out2, S2 = c.run(zp, stream=stream)
        assert torch.equal(out, out2) and torch.equal(S, S2)


def test_two_captured_graphs_with_their_own_workspaces(zp):
    cs = [Case(zp, 81 + i, HEADS["qwen"], [12, 5], [20 + i, 9], (1, 100), 2) for i in range(2)]
    outs, graphs, spaces = [], [], []  # the workspaces outlive the graphs that name them
    for c in cs:
        ws = torch.empty(zp.zp_prefix_decode_workspace_size(c.desc, c.B, c.td.shape[1]), dtype=torch.uint8, device=DEV)
        out = torch.full_like(c.qd, 7.0)

        def step(c=c, out=out, ws=ws):
            zp.zp_prefix_plan(c.desc, c.td, c.ld, c.plan)
            zp.zp_prefix_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, c.plan, out, workspace=ws)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        outs.append(out)
        graphs.append(g)
        spaces.append(ws)
    for out in outs:
        out.fill_(7.0)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    for c, out in zip(cs, outs):
        c.check(out)


def test_bad_members_and_blocks_are_recorded(zp):
    c = Case(zp, 91, HEADS["qwen"], [4], [6], (1, 40), 3)
    good, _ = c.run(zp)
    c.plan.members[1] = c.B + 5
    out = torch.full_like(c.qd, 7.0)
    zp.zp_prefix_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, c.plan, out)
    assert zp.zp_device_status() == (7, 0x142)
    lone = torch.from_numpy(np.nonzero(c.group < 0)[0]).to(DEV)
    assert torch.equal(out[lone], good[lone])
    zp.zp_prefix_plan(c.desc, c.td, c.ld, c.plan)
    for s in np.nonzero(c.group == 0)[0]:
        c.td[int(s), 2] = c.n_total + 1
    zp.zp_prefix_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, c.plan, out)
    assert zp.zp_device_status() == (7, 0x143)
    assert torch.equal(out[lone], good[lone]) and bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("heads", ["qwen", "g8d64", "tiny32", "wide"])
def test_rows_outside_the_sequences_do_not_matter(zp, heads):
    """NaN and infinities in every cache row that holds no token (unused blocks, the rest of last blocks)."""
    c = Case(zp, 101, HEADS[heads], [5, 3], [3, 9], (1, 90), 2, 1)
    used = np.zeros((c.n_total, c.b), bool)
    for s, L in enumerate(c.lens):
        t = np.arange(int(L))
        used[c.table[s, t // c.b], t % c.b] = True
    clean = (c.K.clone(), c.V.clone())
    bad = torch.from_numpy(~used)
    c.K[bad] = float("nan")
    c.V[bad] = float("inf")
    c.Kd, c.Vd = c.K.to(DEV), c.V.to(DEV)
    c.score_rows(102, c.b)
    out, S = c.run(zp)
    c.K, c.V = clean
    c.check(out, S)


def test_blocks_far_into_a_large_cache(zp):
    """Byte offsets beyond 32 bits: the sequences' blocks are the last of a 4.9 GB layer."""
    c = Case(zp, 111, HEADS["qwen"], [6], [20], (1, 60), 2)
    far = 150000
    K = torch.zeros(far, c.b, c.h_kv, c.d, dtype=BF16, device=DEV)
    V = torch.zeros_like(K)
    off = far - c.n_total
    K[off:], V[off:] = c.Kd, c.Vd
    c.score_rows(112, 16)
    td = torch.where(c.td >= 0, c.td + off, c.td)
    desc = zp.cache_desc(c.h_q, c.h_kv, c.d, c.b, far, BF16)
    out = torch.full_like(c.qd, 7.0)
    S = torch.from_numpy(c.S0).to(DEV)
    zp.zp_prefix_plan(desc, td, c.ld, c.plan)
    zp.zp_prefix_decode_attn(desc, c.qd, K, V, td, c.ld, c.plan, out, score_accum=S, window=16, score_rows=_d(c.rows))
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    near, S2 = c.run(zp)
    assert torch.equal(out, near) and torch.equal(S, S2)  # the same work on the same values
    c.check(out, S)


def test_full_batch(zp):
    """The largest batch: 4096 entries, groups and lone entries, some without a token."""
    c = Case(zp, 121, (4, 1, 64, 16, BF16), [1500, 700, 2] + [3] * 400, [3, 2, 5] + [1] * 400, (1, 20), 600, 94)
    assert c.B == 4096
    c.check(*c.run(zp))


@pytest.mark.parametrize("heads", [(8, 2, 128, 16, BF16), (8, 2, 64, 16, F32)], ids=["bf16", "f32"])
def test_scored_batch_beyond_512(zp, heads):
    """More entries than the joining kernel scans itself: the split is read from the workspace."""
    c = Case(zp, 131, heads, [300, 250, 40], [9, 3, 20], (1, 60), 20, 5)
    c.score_rows(132, 11)
    c.check(*c.run(zp))


@pytest.mark.parametrize("heads", HEADS)
def test_what_the_workspace_held_does_not_matter(zp, heads):
    """Records that a call leaves unwritten (streams and CTAs without tiles) are not used: a workspace of NaN."""
    for sizes, blocks in (([3], [30]), ([40, 7], [9, 70])):
        c = Case(zp, 141, HEADS[heads], sizes, blocks, (1, 120), 2, 1)
        c.score_rows(142, c.b)
        n = zp.zp_prefix_decode_workspace_size(c.desc, c.B, c.td.shape[1])
        out, S = c.run(zp, workspace=torch.zeros(n, dtype=torch.uint8, device=DEV))
        out2, S2 = c.run(zp, workspace=torch.full((n,), 255, dtype=torch.uint8, device=DEV))
        assert torch.equal(out, out2) and torch.equal(S, S2)
        c.check(out, S)


def test_captured_without_a_workspace(zp):
    """Captured calls that take their own workspaces, replayed between eager calls and allocations; two on two streams."""
    cs = [Case(zp, 151 + i, HEADS["qwen"], [12, 5], [20 + i, 9], (1, 100), 2) for i in range(2)]
    outs, graphs = [], []
    for c in cs:
        c.run(zp)
        out = torch.full_like(c.qd, 7.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):
                zp.zp_prefix_decode_attn(c.desc, c.qd, c.Kd, c.Vd, c.td, c.ld, c.plan, out)
        outs.append(out)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for out in outs:
            out.fill_(7.0)
        torch.cuda.synchronize()
        for g, st, c in zip(graphs, streams, cs):
            with torch.cuda.stream(st):
                g.replay()
        junk = [torch.full((1 << 24,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
        eager, _ = cs[0].run(zp)
        torch.cuda.synchronize()
        del junk
        cs[0].check(eager)
        for c, out in zip(cs, outs):
            c.check(out)
    assert zp.zp_device_status() == (0, 0)
