"""Decode attention over a 4-bit cache against the definition in 64 bits."""
import ctypes
import math

import numpy as np
import pytest
import torch

import q4_util as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    m.lib.zp_device_status(None, None, 1)
    yield m
    assert _status(m) == (0, 0)


def _status(zp):
    code, detail = ctypes.c_int32(), ctypes.c_int32()
    zp._check(zp.lib.zp_device_status(ctypes.byref(code), ctypes.byref(detail), 1))
    return code.value, detail.value


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Sequences of given lengths in scattered blocks; every row behind a sequence's last token, and every
    block of none, holds NaN."""

    def __init__(self, zp, lens, dtype="bf16", h_q=32, h_kv=8, d=128, group=32, b=16, seed=0, extra=1, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.zp, self.dtype, self.h_q, self.h_kv, self.d, self.group, self.b = zp, dtype, h_q, h_kv, d, group, b
        self.lens = np.asarray(lens)
        B = self.B = len(lens)
        stride = max(1, -(-int(self.lens.max()) // b)) + extra
        n_blocks = -(-self.lens // b)
        self.n_total = int(n_blocks.sum()) + 3
        ids = rng.permutation(self.n_total)
        self.table = np.full((B, stride), -1, dtype=np.int32)
        at = 0
        for s in range(B):
            self.table[s, :n_blocks[s]] = ids[at:at + n_blocks[s]]
            at += n_blocks[s]
        t = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.desc = zp.cache_desc(h_q, h_kv, d, b, self.n_total, t)
        self.q = (torch.from_numpy(rng.standard_normal((B, h_q, d)).astype(np.float32)) * q_scale).to(t)
        self.K = q4.random_cache(rng, self.n_total, h_kv, d, group, b)
        self.V = q4.random_cache(rng, self.n_total, h_kv, d, group, b)
        nan = np.full(d // group, 0x7FC07FC0, np.uint32).view(np.uint8)
        for cache in (self.K, self.V):
            rows = cache[..., 8 * d:].reshape(self.n_total, h_kv, b // 16, 16, len(nan))
            live = np.zeros((self.n_total, b), bool)
            for s in range(B):
                p = np.arange(self.lens[s])
                live[self.table[s, p // b], p % b] = True
            rows[~live.reshape(self.n_total, 1, b // 16, 16).repeat(h_kv, 1)] = nan
            cache[..., 8 * d:] = rows.reshape(self.n_total, h_kv, b // 16, -1)

    def run(self, window=0, S=None, rows=None, workspace=None):
        zp = self.zp
        out = torch.full_like(self.q, 9.0).cuda()
        extra = {} if S is None else dict(score_accum=S, window=window, score_rows=rows)
        zp.zp_q4_decode_attn(self.desc, self.q.cuda(), _dev(self.K), _dev(self.V), _dev(self.table),
                             _dev(self.lens.astype(np.int32)), out, group=self.group, workspace=workspace, **extra)
        torch.cuda.synchronize()
        return out.cpu()

    def reference(self, s):
        """Output [h_q][d], its bound, probabilities [h_q][L] and theirs (relative) of sequence s."""
        L, G, b = int(self.lens[s]), self.h_q // self.h_kv, self.b
        p = np.arange(L)
        slots = self.table[s, p // b].astype(np.int64) * b + p % b
        kc = q4.get_rows(self.K, slots, self.d, self.group, b)
        vc = q4.get_rows(self.V, slots, self.d, self.group, b)
        k, v = q4.values(*kc, self.group), q4.values(*vc, self.group)
        # the size of what is added up for a value: |lo| + code * step
        v_abs = q4.values(vc[0], vc[1], np.abs(vc[2]), self.group)
        k_abs = q4.values(kc[0], kc[1], np.abs(kc[2]), self.group)
        q = self.q[s].double().numpy()
        out, tol = np.empty((self.h_q, self.d)), np.empty((self.h_q, self.d))
        prob, ptol = np.empty((self.h_q, L)), np.empty(self.h_q)
        for h in range(self.h_q):
            x = k[:, h // G] @ q[h] / math.sqrt(self.d)
            size = (k_abs[:, h // G] @ np.abs(q[h]) / math.sqrt(self.d)).max()
            e = np.exp(x - x.max())
            prob[h] = e / e.sum()
            out[h] = prob[h] @ v[:, h // G]
            a = prob[h] @ v_abs[:, h // G]
            # fp32: every logit is d products and a few more steps, each off by 2^-24 of the sum of the
            # magnitudes.
            dx = (self.d + 16) * 2.0 ** -24 * size
            ptol[h] = 2 * dx + 2.0 ** -20 + L * 2.0 ** -24
            # bf16: the probability and its product with the step are each rounded (2^-8), then the output
            r = 2 * 2.0 ** -8 if self.dtype == "bf16" else 0
            tol[h] = (2 * r + 2 * ptol[h] + L * 2.0 ** -23) * a + (2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -23) * np.abs(out[h])
        return out, tol, prob, ptol

    def check(self, out):
        for s in range(self.B):
            got = out[s].double().numpy()
            if self.lens[s] == 0:
                assert (got == 9.0).all()
                continue
            want, tol, _, _ = self.reference(s)
            assert (np.abs(got - want) <= tol).all(), (s, float((np.abs(got - want) / tol).max()))


SHAPES = [("bf16", 32, 8, 128, 32, 16), ("f32", 32, 8, 128, 32, 16), ("bf16", 8, 8, 128, 64, 16), ("bf16", 8, 1, 128, 128, 32),
          ("f32", 8, 2, 64, 32, 16), ("bf16", 32, 4, 64, 64, 48), ("bf16", 15, 3, 64, 32, 64), ("f32", 10, 5, 128, 128, 16),
          ("f32", 21, 3, 64, 64, 32), ("bf16", 16, 16, 64, 32, 16)]


@pytest.mark.parametrize("dtype,h_q,h_kv,d,group,b", SHAPES)
def test_decode(zp, dtype, h_q, h_kv, d, group, b):
    c = Case(zp, [1, 0, 2, 15, 16, 17, 0, 31, 33, 200, 64, 1, 95, 500], dtype, h_q, h_kv, d, group, b)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[3000], [0, 0, 1], [5000, 3, 0, 2000], [1] * 300, [17] * 41 + [900]])
def test_splits(zp, dtype, lens):
    """One long sequence over many ranges, many short ones in one, and both."""
    c = Case(zp, lens, dtype, 8, 2, 64, 32, 16, seed=len(lens))
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_peaked(zp, dtype):
    """Large queries: one token holds nearly all the weight, and the running maximum moves often."""
    c = Case(zp, [700, 33, 2000], dtype, 32, 8, 128, 32, 16, seed=4, q_scale=6.0)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["spread", "late", "flat", "tiny", "huge", "groups"])
def test_step_sizes(zp, dtype, kind):
    """Steps of very different sizes: among all tokens, larger ones from some token on, flat groups (the
    smallest step) here and there, all tiny, all huge, and groups of sizes of their own."""
    rng = np.random.default_rng(7)
    c = Case(zp, [300, 1, 45, 1000], dtype, 32, 8, 128, 32, 16, seed=3)
    for cache in (c.V, c.K):
        word = np.ascontiguousarray(cache[..., 8 * 128:]).view(np.uint32).reshape(c.n_total, 8, 1, 16, 4)
        live = word != 0x7FC07FC0
        step = q4.bf16_value(word & 0xFFFF).copy()
        lo = q4.bf16_value(word >> 16).copy()
        if kind == "spread":
            f = np.exp2(rng.integers(-40, 6, size=step.shape))
        elif kind == "late":
            late = np.zeros((c.n_total, 16), bool)
            for s in range(c.B):
                p = np.arange(c.lens[s] // 2, c.lens[s])
                late[c.table[s, p // 16], p % 16] = True
            f = np.where(late[:, None, None, :, None], 64.0, 1.0) * np.ones(step.shape)
        elif kind == "flat":
            f = np.where(rng.random(step.shape) < 0.02, 0.0, 1.0)
        elif kind == "groups":
            f = np.exp2(np.array([-30.0, 0.0, 9.0, -100.0])) * np.ones(step.shape)
        else:
            f = np.full(step.shape, 2.0 ** -110 if kind == "tiny" else 2.0 ** 90)
        if cache is c.K:   # keys: sizes that leave the logits within reach
            f = np.where(f > 4, 4.0, f)
        step = np.maximum(step * f, 2.0 ** -126).astype(np.float32)
        lo = (lo * f).astype(np.float32)
        new = (q4.bf16_bits(step, True).astype(np.uint32) | q4.bf16_bits(lo, False).astype(np.uint32) << 16)
        cache[..., 8 * 128:] = np.where(live, new, word).astype(np.uint32).reshape(c.n_total, 8, 1, 64).view(np.uint8)
    c.check(c.run())


def test_batch_limit(zp):
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 20, size=4096)
    c = Case(zp, lens, "bf16", 4, 1, 64, 64, 16, seed=5)
    c.check(c.run())


@pytest.mark.parametrize("dtype,h_q,h_kv,d,group,b", SHAPES)
@pytest.mark.parametrize("window", [1, 4, 0])
def test_score(zp, dtype, h_q, h_kv, d, group, b, window):
    """Scores written on the first step of the window, added on the others, left alone off the window, without
    a row and behind the newest token; a slot map with more rows than entries."""
    w = window or b
    lens = np.array([b - w + 1, b, 3 * b, 2 * b - w + 1, 5 * b - w + 2 if w > 1 else b, 2 * b - w, 7 * b, 0, 40 * b])
    c = Case(zp, lens, dtype, h_q, h_kv, d, group, b, seed=w)
    rows = np.array([3, 1, -1, 0, 7, 5, 2, 4, 9], dtype=np.int32)
    rng = np.random.default_rng(1)
    S0 = rng.uniform(0.5, 1.0, size=(11, h_kv, c.table.shape[1] * b)).astype(np.float32)
    S = _dev(S0)
    c.check(c.run(w, S, _dev(rows)))
    got, want, tol = S.cpu().numpy().astype(np.float64), S0.astype(np.float64), np.zeros_like(S0, dtype=np.float64)
    for s, L in enumerate(lens):
        P = int(L) - 1
        if rows[s] < 0 or L == 0 or P % b < b - w:
            continue
        _, _, prob, ptol = c.reference(s)
        new = prob.reshape(h_kv, -1, L).max(1) / w
        rel = ptol.reshape(h_kv, -1).max(1)[:, None] + 2.0 ** -21
        old = np.where((P % b == b - w) | (np.arange(L) == P), 0.0, want[rows[s], :, :L])
        want[rows[s], :, :L] = old + new
        tol[rows[s], :, :L] = rel * new + 2.0 ** -24 * (old + new) * (old > 0)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


def test_score_without_map(zp):
    c = Case(zp, [16, 48, 30], "bf16", 32, 8, 128, 32, 16)
    S = torch.zeros(3, 8, c.table.shape[1] * 16, device="cuda")
    c.check(c.run(4, S))
    got = S.cpu().numpy()
    for s, L in ((0, 16), (1, 48), (2, 30)):  # query positions 15, 47 and 29: 15, 15 and 13 in their blocks, from 12 on
        _, _, prob, ptol = c.reference(s)
        new = prob.reshape(8, 4, L).max(1) / 4
        assert (np.abs(got[s, :, :L] - new) <= (ptol.max() + 2.0 ** -21) * new).all()
        assert not got[s, :, L:].any()


def test_same_bits_again(zp):
    """Any content of the workspace, and the same bits on every call."""
    c = Case(zp, [2000, 7, 900, 0, 64], "bf16", 32, 8, 128, 32, 16)
    n = zp.zp_q4_decode_workspace_size(c.desc, c.B, c.table.shape[1])
    outs, scores = [], []
    for fill in (0, 255, 127):
        S = torch.zeros(c.B, 8, c.table.shape[1] * 16, device="cuda")
        outs.append(c.run(16, S, None, torch.full((n,), fill, dtype=torch.uint8, device="cuda")))
        scores.append(S.cpu())
    for o, s in zip(outs[1:], scores[1:]):
        assert torch.equal(o, outs[0]) and torch.equal(s, scores[0])


def test_not_finite_query(zp):
    """A NaN in one query row reaches that row alone."""
    c = Case(zp, [40, 300], "bf16", 32, 8, 128, 32, 16)
    c.q[1, 5, 3] = float("nan")
    out = c.run()
    assert bool(torch.isnan(out[1, 5]).all())
    out[1, 5] = 0
    c.q[1, 5, 3] = 0
    for s in range(2):
        want, tol, _, _ = c.reference(s)
        ok = np.abs(out[s].double().numpy() - want) <= tol
        ok[5] |= s == 1
        assert ok.all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_not_finite_cache(zp, dtype):
    """A group of a key that reads as NaN makes its kv head's outputs NaN, a group of a value the
    dimensions of the group; other heads and sequences are as without it."""
    c = Case(zp, [40, 90], dtype, 8, 2, 128, 32, 16, seed=9)
    word = np.array([0x7FC07FC0], np.uint32).view(np.uint8)
    clean = [c.reference(s) for s in range(2)]
    slot = int(c.table[0, 1]) * 16 + 5                          # token 21 of sequence 0
    at = 8 * 128 + (slot % 16) * 16
    c.V[slot // 16, 0, 0, at + 8:at + 12] = word                 # head 0, group 2
    slot = int(c.table[1, 4]) * 16 + 1
    at = 8 * 128 + (slot % 16) * 16
    c.K[slot // 16, 1, 0, at:at + 4] = word                      # sequence 1, head 1, group 0
    out = c.run().double().numpy()
    nan = np.isnan(out)
    want = np.zeros_like(nan)
    want[0, :4, 64:96] = True
    want[1, 4:] = True
    assert np.array_equal(nan, want)
    for s in range(2):
        ref, tol, _, _ = clean[s]
        assert (np.abs(out[s] - ref) <= tol)[~want[s]].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-30, 1e-4, 300.0, 1e30])
def test_query_sizes(zp, dtype, scale):
    """Queries far from one: tiny ones give the mean of the values, huge ones the value of one token."""
    c = Case(zp, [77, 300], dtype, 8, 2, 64, 32, 16, seed=2, q_scale=scale)
    if scale < 100:
        c.check(c.run())
        return
    out = c.run().double().numpy()
    for s in range(2):
        want, tol, prob, _ = c.reference(s)
        sure = prob.max(1) == 1.0  # no other token within 2^-53 of the heaviest
        assert sure.any() and (np.abs(out[s] - want) <= tol)[sure].all()


def test_two_streams_at_once(zp):
    """Calls on two streams, each with memory of its own, while the other runs."""
    cases = [Case(zp, [900, 31, 2000], "bf16", 32, 8, 128, 32, 16, seed=i) for i in range(2)]
    want = [c.run() for c in cases]
    data = [(c.q.cuda(), _dev(c.K), _dev(c.V), _dev(c.table), _dev(c.lens.astype(np.int32)), torch.zeros_like(c.q).cuda())
            for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, d, st in zip(cases, data, streams):
            with torch.cuda.stream(st):
                zp.zp_q4_decode_attn(c.desc, *d)
    torch.cuda.synchronize()
    for d, w in zip(data, want):
        assert torch.equal(d[5].cpu(), w)


def test_graphs_share_a_workspace(zp):
    """Two captured graphs with one workspace, replayed one after the other in any order."""
    cases = [Case(zp, [700, 31], "bf16", 32, 8, 128, 32, 16, seed=1), Case(zp, [48, 160, 16], "f32", 8, 2, 64, 64, 16, seed=2)]
    S = [torch.zeros(c.B, c.h_kv, c.table.shape[1] * 16, device="cuda") for c in cases]
    want = [c.run(16, s) for c, s in zip(cases, S)]
    score = [s.clone() for s in S]
    n = max(zp.zp_q4_decode_workspace_size(c.desc, c.B, c.table.shape[1], c.group) for c in cases)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for c, s in zip(cases, S):
        d = (c.q.cuda(), _dev(c.K), _dev(c.V), _dev(c.table), _dev(c.lens.astype(np.int32)), torch.zeros_like(c.q).cuda())
        outs.append(d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            zp.zp_q4_decode_attn(c.desc, *d, group=c.group, score_accum=s, window=16, workspace=ws)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0, 0):
        S[i].zero_()
        outs[i][5].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i][5].cpu(), want[i]) and torch.equal(S[i], score[i])


def test_bad_blocks_and_lengths(zp):
    c = Case(zp, [50, 70, 33], "bf16", 32, 8, 128, 32, 16)
    good = c.table.copy()
    for bad in (-1, c.n_total):
        c.table = good.copy()
        c.table[1, 2] = bad
        out = c.run()
        assert _status(zp) == (7, 0x159)
        for s in (0, 2):
            want, tol, _, _ = c.reference(s)
            assert (np.abs(out[s].double().numpy() - want) <= tol).all()
        assert bool(torch.isfinite(out[1].float()).all())
    c.table = good
    c.lens = np.array([50, -3, 33])
    out = c.run()
    assert _status(zp) == (7, 0x158)
    assert bool((out[1] == 9.0).all())
    c.lens = np.array([50, 0, 33])
    c.check(out)
    rows = _dev(np.array([0, 1, 5], dtype=np.int32))
    S = torch.zeros(2, 8, c.table.shape[1] * 16, device="cuda")
    c.lens = np.array([48, 0, 32])
    c.check(c.run(16, S, rows))
    assert _status(zp) == (7, 0x15a)
    assert bool(S[0].any()) and not bool(S[1].any())


def test_streams_and_graph(zp):
    """On another stream with a workspace of its own, and captured and replayed with new lengths."""
    c = Case(zp, [600, 31, 90], "bf16", 32, 8, 128, 32, 16)
    want = c.run()
    q, K, V, table, lens = c.q.cuda(), _dev(c.K), _dev(c.V), _dev(c.table), _dev(c.lens.astype(np.int32))
    ws = torch.empty(zp.zp_q4_decode_workspace_size(c.desc, 3, c.table.shape[1]), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        zp.zp_q4_decode_attn(c.desc, q, K, V, table, lens, out)
    st.synchronize()
    assert torch.equal(out.cpu(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zp.zp_q4_decode_attn(c.desc, q, K, V, table, lens, out, workspace=ws)
    for now in ([600, 31, 90], [17, 1, 64], [600, 31, 90]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        d = Case(zp, [600, 31, 90], "bf16", 32, 8, 128, 32, 16)
        d.lens = np.array(now)
        d.check(out.cpu())


def test_chain(zp):
    """A prompt written, tokens appended, attended to with the score, the best kept and moved, and attended to
    again: against the same steps on the values read back."""
    rng = np.random.default_rng(6)
    h_q, h_kv, d, b, group, n_total, N = 32, 8, 128, 16, 32, 40, 12
    desc = zp.cache_desc(h_q, h_kv, d, b, n_total, torch.bfloat16)
    K, V = zp.zp_q4_cache(desc, group)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    i32 = lambda a: _dev(np.asarray(a, np.int32))  # noqa: E731
    B, prompt = 2, [N * b - 16, N * b - 30]
    table = np.full((B, N + 1), -1, np.int32)
    table[:, :N] = rng.permutation(n_total)[:B * N].reshape(B, N)
    slots = np.concatenate([table[s, np.arange(n) // b] * b + np.arange(n) % b for s, n in enumerate(prompt)])
    k, v = bf(len(slots), h_kv, d), bf(len(slots), h_kv, d)
    zp.zp_q4_write_kv(desc, k, v, i32(slots), K, V, group=group)
    S = torch.zeros(B, h_kv, (N + 1) * b, device="cuda")
    out = torch.zeros(B, h_q, d, dtype=torch.bfloat16, device="cuda")
    for step in range(16):
        lens = i32([n + step + 1 for n in prompt])
        zp.zp_q4_append_kv(desc, bf(B, h_kv, d), bf(B, h_kv, d), K, V, i32(table), lens, group=group)
        q = bf(B, h_q, d)
        zp.zp_q4_decode_attn(desc, q, K, V, i32(table), lens, out, score_accum=S, window=b, group=group)
    L, keep_n = N * b, (N - 1) * b                     # sequence 0 has filled its budget
    scores = torch.zeros(1, h_kv, L, device="cuda")
    F = torch.zeros(n_total, b, h_kv, device="cuda")
    first = torch.ones(1, dtype=torch.uint8, device="cuda")
    prm = zp.score_params(window=b, use_similarity=False)
    kc = torch.zeros(n_total, b, h_kv, d, dtype=torch.bfloat16, device="cuda")   # (not read without the redundancy)
    zp.zp_score_tokens(desc, prm, kc, i32(table[:1]), i32([L]), first, S, F, scores)
    keep = torch.empty(1, h_kv, keep_n, dtype=torch.int32, device="cuda")
    zp.zp_select_topk(scores, i32([L]), keep_n, keep)
    before = q4.get_rows(K.cpu().numpy(), table[0, np.arange(L) // b] * b + np.arange(L) % b, d, group, b)
    zp.zp_q4_compact_pages(desc, K, V, i32(table[:1]), i32(table[:1, :N - 1]), i32([L]), keep, global_F=F, scores=S,
                           rows=i32([0]), group=group)
    after = q4.get_rows(K.cpu().numpy(), table[0, np.arange(keep_n) // b] * b + np.arange(keep_n) % b, d, group, b)
    kept = keep[0].cpu().numpy()
    for h in range(h_kv):
        assert (np.diff(kept[h]) > 0).all() and set(range(L - b, L)) <= set(kept[h])
        for x, y in zip(before, after):
            assert np.array_equal(x[kept[h], h], y[:, h])
    zp.zp_q4_decode_attn(desc, q, K, V, i32(table), i32([keep_n, prompt[1] + 16]), out, group=group)
    c = Case(zp, [keep_n, prompt[1] + 16], "bf16", h_q, h_kv, d, group, b)
    c.q, c.K, c.V, c.table = q.cpu(), K.cpu().numpy(), V.cpu().numpy(), table
    c.check(out.cpu())
