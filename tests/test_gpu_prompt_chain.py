"""The shared-prompt operators together, as a serving step uses them: tables and
slots from request lengths, prompt rows written through them, groups found in
the tables, prefix-shared decode with the window score, eviction.

* A batch behind two prompts, prefilled and decoded step by step with every
  table entry dealt on the device, against the 64-bit oracle each step; the last
  step's scores go into the compression and its keep sets are the oracle's.
* The decode loop and the serving loop with prefix_decode, against the oracle
  loop (prompts shared, compressed by reference, then diverging).
"""
import numpy as np
import pytest
import torch

import oracle
import zp_inputs
from oracle import pipeline
from tests.gpu_util import TOL_OUT, gather_slots, keep_sets_match
from tests.oracle_loop import OracleLoop
from tests.prefix_util import attention_bounds, window_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    return m


def _d(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_decode_and_eviction(zp, dtype):
    h_q, h_kv, d, b, w, layers = 16, 4, 64, 16, 16, 2
    rng = np.random.default_rng(9)
    shared, n_total, stride = [6, 3], 300, 20
    group = np.array([0, 1, 0, 0, 1, 0, 0, 1])
    B = len(group)
    ids = rng.permutation(n_total).astype(np.int32)
    heads = [ids[:6], ids[6:9]]
    fresh = ids[9:]
    table = np.full((B, stride), -1, np.int32)
    for s in range(B):
        table[s, :shared[group[s]]] = heads[group[s]]
    desc = zp.cache_desc(h_q, h_kv, d, b, n_total, dtype)
    K = torch.zeros(layers, n_total, b, h_kv, d, dtype=dtype, device=DEV)
    V = torch.zeros_like(K)
    mk = lambda *s, seed: zp_inputs.normal(s, seed, "bf16" if dtype == torch.bfloat16 else "f32")  # noqa: E731

    # prefill: the first member of each group writes the prompt, the others what follows it
    pre = np.array([shared[g] * b for g in group])
    first = np.array([s == int(np.nonzero(group == group[s])[0][0]) for s in range(B)])
    lens = pre + rng.integers(1, 50, size=B)
    start = np.where(first, 0, pre)
    tables = [_d(table), _d(table)]
    room = int((lens - start).sum()) + 5
    slots, cu, used = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (room, B + 1, 1))
    zp.zp_build_slots(desc, tables[0], _d(start), _d(lens), slots, cu, fresh=_d(fresh), table_out=tables[1], n_used=used)
    dealt = int(used)
    kn, vn = mk(layers, room, h_kv, d, seed=1), mk(layers, room, h_kv, d, seed=2)
    zp.zp_write_kv(desc, kn.to(DEV), vn.to(DEV), slots, K, V)
    # decode steps: one block table behind the other, the append through the slot map
    S = torch.zeros(layers, B, h_kv, stride * b, device=DEV)
    S_ref = np.zeros((layers, B, h_kv, stride * b))
    plan = zp.prefix_plan(B)
    ws = torch.empty(zp.zp_prefix_decode_workspace_size(desc, B, stride), dtype=torch.uint8, device=DEV)
    steps = 2 * b + 3
    for step in range(steps):
        new = lens + 1
        if step == steps - 1:  # end on full blocks, where the eviction is triggered
            break
        src, dst = tables[1], tables[0]
        step_slots = torch.empty(B, dtype=torch.int32, device=DEV)
        zp.zp_build_slots(desc, src, _d(lens), _d(new), step_slots, cu, fresh=_d(fresh[dealt:]), table_out=dst, n_used=used)
        dealt += int(used)
        tables.reverse()
        lens = new
        table_h = tables[1].cpu().numpy()
        kn, vn = mk(layers, B, h_kv, d, seed=100 + step), mk(layers, B, h_kv, d, seed=200 + step)
        zp.zp_write_kv(desc, kn.to(DEV), vn.to(DEV), step_slots, K, V)
        if step % 5 == 0:
            zp.zp_prefix_plan(desc, tables[1], _d(lens), plan, min_blocks=2)
            assert sorted(plan.prefix_lens.tolist()) == sorted(pre.tolist())
        q = mk(layers, B, h_q, d, seed=300 + step)
        out = torch.empty(layers, B, h_q, d, dtype=dtype, device=DEV)
        for l in range(layers):
            zp.zp_prefix_decode_attn(desc, q[l].to(DEV), K[l], V[l], tables[1], _d(lens), plan, out[l], score_accum=S[l],
                                     window=w, workspace=ws)
        torch.cuda.synchronize()
        assert zp.zp_device_status() == (0, 0)
        Kh, Vh = K.float().cpu().numpy(), V.float().cpu().numpy()
        for l in range(layers):
            ref, tol, probs, rel = attention_bounds(q[l].float().numpy(), Kh[l], Vh[l], np.maximum(table_h, 0),
                                                    lens.astype(np.int32), dtype == torch.bfloat16)
            assert (np.abs(out[l].float().cpu().numpy() - ref) <= tol).all()
            window_ref(probs, lens, None, S_ref[l], np.arange(B), h_kv, b, w)
            # each of up to w accumulated terms has the probability's bound
            np.testing.assert_allclose(S[l].cpu().numpy(), S_ref[l], rtol=rel + w * 2.0 ** -23, atol=1e-30)
    # eviction of the sequences as they stand, keep sets against the oracle
    k = 4 * b
    keep = torch.empty(B, h_kv, k, dtype=torch.int32, device=DEV)
    prm = zp.score_params(window=w)
    F = torch.zeros(n_total, b, h_kv, device=DEV)
    scores = torch.zeros(B, h_kv, stride * b, device=DEV)
    S_now = S[1].double().cpu().numpy()
    zp.zp_score_tokens(desc, prm, K[1], tables[1], _d(lens), torch.ones(B, dtype=torch.uint8, device=DEV), S[1], F, scores)
    zp.zp_select_topk(scores, _d(lens), k, keep)
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    for s in range(B):
        L = int(lens[s])
        fs = pipeline.final_scores(S_now[s, :, :L], Kh[1], np.zeros((n_total, b, h_kv)), table_h[s], L, b, True,
                                   pipeline.ScoreParams(window=w))
        for h in range(h_kv):
            keep_sets_match(keep[s, h].cpu().numpy(), oracle.topk_keep(fs[h], k)[0], fs[h], k, L)


@pytest.mark.parametrize("async_compress", [False, True])
def test_decode_loop_with_shared_prompts(zp, async_compress):
    """The decode loop with prefix_decode against the oracle loop on private copies of the shared blocks."""
    from compressed_paged_kv_zp_gb300.engine import DecodeLoop
    layers, B, stride, N_max, P, b = 2, 7, 14, 6, 4, 16
    h_q, h_kv, d = 16, 4, 64
    rng = np.random.default_rng(31)
    lens0 = (P * b + rng.integers(1, 30, size=B)).astype(np.int32)
    n_total = 150
    tables = np.full((B, stride), -1, np.int32)
    ids = rng.permutation(n_total).astype(np.int32)
    at = P
    for s in range(B):
        nb = -(-int(lens0[s]) // b)
        tables[s, :P] = ids[:P]
        tables[s, P:nb] = ids[at:at + nb - P]
        at += nb - P
    loop = DecodeLoop(h_q, h_kv, d, b, n_total, N_max, stride, layers=layers, async_compress=async_compress,
                      prefix_decode=True, prefix_min_blocks=1)
    loop.add_sequences(lens0, tables)
    assert not loop.use_rho
    loop.K.copy_(zp_inputs.normal(tuple(loop.K.shape), 7, "bf16").cuda())
    loop.V.copy_(zp_inputs.normal(tuple(loop.V.shape), 8, "bf16").cuda())
    Kh, Vh = loop.K.float().cpu().numpy(), loop.V.float().cpu().numpy()
    nb0 = [-(-int(n) // b) for n in lens0]
    cfg = dict(h_q=h_q, h_kv=h_kv, d=d, b=b, N_max=N_max, w=b)
    ora = OracleLoop.mirror(cfg, [Kh[:, tables[s, :nb0[s]]] for s in range(B)], [Vh[:, tables[s, :nb0[s]]] for s in range(B)],
                            lens0, stride, spare=200)
    compressed, grouped = 0, 0
    for step in range(60):
        q = zp_inputs.normal((layers, B, h_q, d), 1000 + step, "bf16")
        kn = zp_inputs.normal((layers, B, h_kv, d), 2000 + step, "bf16")
        vn = zp_inputs.normal((layers, B, h_kv, d), 3000 + step, "bf16")
        if async_compress:
            loop.drain()
        trig = loop.step(q.cuda(), kn.cuda(), vn.cuda())
        torch.cuda.synchronize()
        grouped += int(loop.plan.n_groups)
        out_ref, trig_ref = ora.step(q.float().numpy(), kn.float().numpy(), vn.float().numpy())
        assert sorted(int(x) for x in trig) == trig_ref
        np.testing.assert_allclose(loop.out.float().cpu().numpy(), out_ref, **TOL_OUT["bf16"])
        if trig:
            seqs, keep = loop.last_keep
            keep = keep.cpu().numpy()
            for i, s in enumerate(seqs):
                ora.compress(int(s), keep[:, i])
                compressed += 1
            loop.drain()
            torch.cuda.synchronize()
            assert np.array_equal(loop.lens, ora.lens)
    assert zp.zp_device_status() == (0, 0)
    assert compressed >= B and 0 < grouped < 60  # shared at first, private after the compressions
    assert int(loop.plan.n_groups) == 0


def test_serving_loop_prefix_decode_matches_the_plain_decode(zp):
    """The same trace with and without prefix_decode: every step's inputs are drawn alike as long as the schedules
    agree, which they do (they do not depend on values), and the outputs agree to rounding until a near-tie in a
    keep set could part them."""
    from compressed_paged_kv_zp_gb300.serve import ServeLoop, synthetic_trace
    from compressed_paged_kv_zp_gb300.sched import HYBRID
    trace = synthetic_trace(24, 83, prompt=(120, 300), output=(30, 90), prefix_groups=2, prefix_len=112)
    loops = []
    for flag in (False, True):
        loop = ServeLoop(32, 8, 128, 16, 500, 64, 12, 64, layers=2, policy=HYBRID, prefix_sharing=True, max_running=24,
                         seed=84, prefix_decode=flag, prefix_min_blocks=2)
        for r in trace:
            loop.add_request(*r)
        loops.append(loop)
    steps = grouped = 0
    while True:
        c = loops[0].sched.counts()
        if c["waiting"] == 0 and c["running"] == 0:
            break
        kinds = [loop.step() for loop in loops]
        assert kinds[0] == kinds[1]
        if kinds[0][0] == "decode":
            # |v| < 6: both outputs are within 2^-8 (sum p |v| + |out|) of the same value
            torch.testing.assert_close(loops[0].out.float(), loops[1].out.float(), rtol=2.0 ** -7, atol=6 * 2.0 ** -7)
            grouped += int(loops[1]._plan_buf[1, 0])
            steps += 1
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    assert steps > 50 and grouped > steps // 2
    assert loops[0].stats["compressions"] == 0  # no eviction in this trace: the caches stay alike
    assert torch.equal(loops[0].K, loops[1].K)
