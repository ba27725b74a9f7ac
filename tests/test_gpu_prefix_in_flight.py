"""Prefix-shared decode while compressions are in flight: members of a group sit out
of the batch with their tables as they were, among them the one whose table row names
the group's prefix, while the others go on; then they return with blocks of their own.

* The decode loop, its compressions held open for several steps: every active
  sequence's output and every keep set against the oracle, sequence by sequence.
* The serving loop on a trace with shared prompts that does compress.
"""
import numpy as np
import pytest
import torch

import zp_inputs
from tests.gpu_util import TOL_OUT
from tests.oracle_loop import OracleLoop

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    return m


class Held:
    """The end of a compression as the loop sees it: not before the test lets go of it."""

    def __init__(self, event):
        self.event, self.free = event, False

    def query(self):
        return self.free and self.event.query()

    def synchronize(self):
        self.event.synchronize()


@pytest.mark.parametrize("hold", [1, 5, 12])
def test_decode_loop_with_compressions_in_flight(zp, hold):
    from compressed_paged_kv_zp_gb300.engine import DecodeLoop
    layers, B, stride, N_max, P, b = 2, 7, 14, 6, 4, 16
    h_q, h_kv, d = 16, 4, 64
    rng = np.random.default_rng(41)
    # the first of the group triggers first, the others a few steps after one another
    lens0 = (P * b + np.array([27, 6, 21, 24, 3, 15, 18])).astype(np.int32)
    n_total = 150
    tables = np.full((B, stride), -1, np.int32)
    ids = rng.permutation(n_total).astype(np.int32)
    at = P
    for s in range(B):
        nb = -(-int(lens0[s]) // b)
        tables[s, :P] = ids[:P]
        tables[s, P:nb] = ids[at:at + nb - P]
        at += nb - P
    loop = DecodeLoop(h_q, h_kv, d, b, n_total, N_max, stride, layers=layers, async_compress=True, prefix_decode=True,
                      prefix_min_blocks=1)
    loop.add_sequences(lens0, tables)
    loop.K.copy_(zp_inputs.normal(tuple(loop.K.shape), 7, "bf16").cuda())
    loop.V.copy_(zp_inputs.normal(tuple(loop.V.shape), 8, "bf16").cuda())
    Kh, Vh = loop.K.float().cpu().numpy(), loop.V.float().cpu().numpy()
    cfg = dict(h_q=h_q, h_kv=h_kv, d=d, b=b, N_max=N_max, w=b)
    ora = []
    for s in range(B):
        nb = -(-int(lens0[s]) // b)
        ora.append(OracleLoop.mirror(cfg, [Kh[:, tables[s, :nb]]], [Vh[:, tables[s, :nb]]], lens0[s:s + 1], stride, spare=40))
    flight = {}  # sequence -> (step it triggered in, its end, keep sets)
    listed_absent, first_absent, grouped, compressed = 0, 0, 0, 0
    for step in range(60):
        q = zp_inputs.normal((layers, B, h_q, d), 1000 + step, "bf16")
        kn = zp_inputs.normal((layers, B, h_kv, d), 2000 + step, "bf16")
        vn = zp_inputs.normal((layers, B, h_kv, d), 3000 + step, "bf16")
        for s in [s for s, f in flight.items() if step - f[0] > hold]:
            began, end, keep = flight.pop(s)
            end.synchronize()  # (what query() answers is then settled)
            end.free = True
            ora[s].compress(0, keep.cpu().numpy())
            compressed += 1
        before = loop.out.clone()
        trig = loop.step(q.cuda(), kn.cuda(), vn.cuda())
        out = loop.out.float().cpu().numpy()
        for s in range(B):
            if s in flight:
                assert torch.equal(loop.out[:, s], before[:, s])  # sits out: its row stays
                continue
            one = lambda x: x[:, s:s + 1].float().numpy()  # noqa: E731
            ref, trig_ref = ora[s].step(one(q), one(kn), one(vn))
            np.testing.assert_allclose(out[:, s:s + 1], ref, **TOL_OUT["bf16"])
            assert (s in trig) == bool(trig_ref)
        n = int(loop.plan.group_start[int(loop.plan.n_groups)])
        members = loop.plan.members[:n].tolist()
        grouped += bool(members)
        listed_absent += any(s in flight for s in members)
        first_absent += bool(members) and members[0] in flight
        if trig:
            seqs, keep = loop.last_keep
            end, *rest = loop.pending[-1]
            loop.pending[-1] = (Held(end), *rest)
            for i, s in enumerate(seqs):
                flight[int(s)] = (step, loop.pending[-1][0], keep[:, i])
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    assert compressed >= B and grouped > 5
    # a plan went on naming members that sat out, the one with the prefix's row among them
    assert listed_absent > 0 and first_absent > 0


def test_serving_loop_with_shared_prompts_that_compresses(zp):
    from compressed_paged_kv_zp_gb300.sched import HYBRID
    from compressed_paged_kv_zp_gb300.serve import ServeLoop, synthetic_trace
    b, N_max, M, layers = 16, 12, 6, 2
    trace = synthetic_trace(14, 91, prompt=(100, 170), output=(60, 240), prefix_groups=2, prefix_len=96)
    loop = ServeLoop(32, 8, 128, b, 400, N_max, M, (170 + 240) // b + 2, layers=layers, policy=HYBRID, prefix_sharing=True,
                     max_running=14, seed=92, prefix_decode=True, prefix_min_blocks=2)
    for r in trace:
        loop.add_request(*r)
    watch, mirrors, swaps, checked, keeps, mixed = set(range(M)), {}, 0, 0, 0, 0
    for _ in range(100000):
        c = loop.sched.counts()
        if c["waiting"] == 0 and c["running"] == 0:
            break
        kind, fin = loop.step()
        ids = [int(x) for x in loop.last_step[1]]
        if kind == "prefill":
            for pos, i in enumerate(ids):
                if i in watch and i not in mirrors:
                    info, row = loop.sched.info(i), loop.last_step[3][pos]
                    blk = torch.from_numpy(row[row >= 0].astype(np.int64)).to(loop.dev)
                    cfg = dict(h_q=32, h_kv=8, d=128, b=b, N_max=N_max, w=loop.window)
                    mirrors[i] = OracleLoop.mirror(cfg, [loop.K.index_select(1, blk).float().cpu().numpy()],
                                                   [loop.V.index_select(1, blk).float().cpu().numpy()],
                                                   np.array([info["L"]]), loop.stride, spare=loop.stride + 4)
        elif kind == "decode":
            # groups in a step that a compressing request sits out of
            mixed += bool(loop.inflight) and int(loop._plan_buf[1, 0]) > 0
            q, kn, vn = loop.last_step[2]
            for pos, i in enumerate(ids):
                if i not in mirrors:
                    continue
                info = loop.sched.info(i)
                if info["preemptions"]:  # (it loses its cache: no longer mirrored)
                    del mirrors[i]
                    watch.discard(i)
                    continue
                one = lambda x: x[:, pos:pos + 1].float().cpu().numpy()  # noqa: E731
                ref, trig = mirrors[i].step(one(q), one(kn), one(vn))
                np.testing.assert_allclose(loop.out[:, pos:pos + 1].float().cpu().numpy(), ref, **TOL_OUT["bf16"])
                checked += 1
                if i in fin:
                    del mirrors[i]
                elif trig:
                    assert info["state"] == 2  # compressing
                    torch.cuda.synchronize()
                    kids, keep = loop.last_keep
                    swaps += mirrors[i].compress(0, keep[:, kids.index(i)].cpu().numpy())
                    keeps += 1
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    c = loop.sched.counts()
    assert c["finished"] == len(trace) and c["free_blocks"] == loop.n_total and c["free_slots"] == M
    assert checked > 200 and keeps >= 4 and loop.stats["compressions"] >= 8
    print(loop.stats, "mirrored steps", checked, "keep sets", keeps, "near-tie swaps", swaps, "mixed steps", mixed)
