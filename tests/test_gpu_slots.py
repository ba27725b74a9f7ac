"""Slot maps and block tables built from request lengths, prompt rows written
through them, and the prefix groups found in the tables: exact against plain
host code (whole numbers and copies)."""
import numpy as np
import pytest
import torch

from tests.prefix_util import make_groups, plan_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    return m


def _d(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _desc(zp, b, n_total):
    return zp.cache_desc(8, 2, 64, b, n_total, torch.bfloat16)


def slots_ref(table, old, new, fresh, b, max_tokens):
    out = table.copy()
    used = 0
    slots, pos, cu = [], [], [0]
    for s in range(len(old)):
        o, n = int(old[s]), int(new[s])
        for c in range(-(-o // b), -(-n // b)):
            if out[s, c] < 0:
                out[s, c] = fresh[used] if used < len(fresh) else -1
                used += 1
        for t in range(o, n):
            blk = int(out[s, t // b])
            slots.append(blk * b + t % b if blk >= 0 else -1)
            pos.append(t)
        cu.append(cu[-1] + n - o)
    pad = [-1] * (max_tokens - len(slots))
    return out, np.array(slots + pad, np.int32), np.array(pos + pad, np.int32), np.array(cu, np.int32), used


def slots_case(seed, B, b, old, grow, ahead=0.2):
    rng = np.random.default_rng(seed)
    o = rng.integers(old[0], old[1] + 1, size=B)
    n = o + rng.integers(grow[0], grow[1] + 1, size=B)
    have, want = -(-o // b), -(-n // b)
    stride = int(want.max() if B else 0) + 3
    total = int(want.sum()) + B + 8
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((B, stride), -1, np.int32)
    at = 0
    for s in range(B):
        table[s, :have[s]] = ids[at:at + have[s]]
        at += have[s]
        for c in range(have[s], want[s]):  # blocks held ahead, anywhere in the growth
            if rng.random() < ahead:
                table[s, c] = ids[at]
                at += 1
    return table, o, n, ids[at:], total


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,b,old,grow", [
    (1, 16, (0, 0), (1, 1)), (1, 16, (0, 0), (0, 0)), (3, 16, (15, 17), (0, 40)), (5, 32, (0, 100), (1, 1)),
    (17, 16, (0, 300), (0, 700)), (512, 16, (1, 200), (1, 1)), (4096, 16, (0, 40), (0, 5)), (2, 64, (0, 0), (30000, 40000)),
    (4095, 16, (0, 0), (1, 33)), (40, 16, (16, 16), (0, 0))])
def test_build_slots(zp, B, b, old, grow, in_place):
    table, o, n, fresh, total = slots_case(B * 131 + b, B, b, old, grow)
    room = int((n - o).sum()) + 37
    ref = slots_ref(table, o, n, fresh, b, room)
    td = _d(table)
    out = td if in_place else torch.full_like(td, -7)
    slots, pos = torch.full((room,), 99, dtype=torch.int32, device=DEV), torch.full((room,), 99, dtype=torch.int32, device=DEV)
    cu, used = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    zp.zp_build_slots(_desc(zp, b, total), td, _d(o), _d(n), slots, cu, fresh=_d(fresh),
                      table_out=None if in_place else out, positions=pos, n_used=used)
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    for got, want in zip((out, slots, pos, cu), ref[:4]):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert int(used) == ref[4]
    if not in_place:
        np.testing.assert_array_equal(td.cpu().numpy(), table)  # the input stays


def test_build_slots_without_sequences_and_optional_outputs(zp):
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    cu = torch.full((1,), 5, dtype=torch.int32, device=DEV)
    slots = torch.zeros(9, dtype=torch.int32, device=DEV)
    zp.zp_build_slots(_desc(zp, 16, 4), torch.empty(0, 3, dtype=torch.int32, device=DEV), e, e, slots, cu)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 9
    table, o, n, fresh, total = slots_case(3, 6, 16, (0, 60), (0, 60), ahead=0)
    cu = torch.empty(7, dtype=torch.int32, device=DEV)
    zp.zp_build_slots(_desc(zp, 16, total), _d(table), _d(o), _d(o), e, cu)  # nobody grows, no buffers
    assert cu.tolist() == [0] * 7 and zp.zp_device_status() == (0, 0)


def test_build_slots_records_what_it_cannot_do(zp):
    b, total = 16, 10
    desc = _desc(zp, b, total)
    table = np.full((3, 4), -1, np.int32)
    table[0, 0], table[1, 0], table[2, 0] = 3, 4, 99  # 99 is no block
    cu = torch.empty(4, dtype=torch.int32, device=DEV)

    def call(old, new, fresh, room):
        slots = torch.full((room,), 77, dtype=torch.int32, device=DEV)
        used = torch.empty(1, dtype=torch.int32, device=DEV)
        out = torch.empty(3, 4, dtype=torch.int32, device=DEV)
        zp.zp_build_slots(desc, _d(table), _d(old), _d(new), slots, cu, fresh=_d(fresh), table_out=out, n_used=used)
        return slots.tolist(), out.cpu().numpy(), int(used), zp.zp_device_status()

    # new below old, new beyond the row, old negative: no growth, the others go on
    s, t, used, st = call([5, 16, -1], [4, 17, 3], [7], 2)
    assert st == (7, 0x120) and s == [7 * b, -1] and t[1, 1] == 7 and used == 1
    s, t, used, st = call([5, 16, 0], [65, 16, 0], [7], 1)
    assert st == (7, 0x120) and s == [-1] and used == 0
    # two blocks needed, one given: the second sequence's entry and slots are -1
    s, t, used, st = call([16, 16, 0], [17, 18, 0], [7], 3)
    assert st == (7, 0x121) and s == [7 * b, -1, -1] and used == 2 and t[0, 1] == 7 and t[1, 1] == -1
    # a bad block under a new token
    s, t, used, st = call([5, 5, 5], [6, 5, 7], [], 3)
    assert st == (7, 0x122) and s == [3 * b + 5, -1, -1]
    # more tokens than room: the first ones are written
    s, t, used, st = call([5, 5, 0], [9, 9, 0], [], 6)
    assert st == (7, 0x123) and s == [53, 54, 55, 56, 69, 70]
    assert call([5, 5, 0], [6, 6, 0], [], 2)[3] == (0, 0)


def test_build_slots_in_a_graph(zp):
    """A captured step replayed on new lengths: the token buffer has the largest size, the rest is padding."""
    b, B = 16, 33
    table, o, n, fresh, total = slots_case(8, B, b, (1, 90), (1, 1))
    room = 64
    td, od, nd, fd = _d(table), _d(o), _d(n), _d(fresh)
    out, slots, cu = torch.empty_like(td), torch.empty(room, dtype=torch.int32, device=DEV), torch.empty(B + 1, dtype=torch.int32, device=DEV)
    desc = _desc(zp, b, total)
    zp.zp_build_slots(desc, td, od, nd, slots, cu, fresh=fd, table_out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zp.zp_build_slots(desc, td, od, nd, slots, cu, fresh=fd, table_out=out)
    for step in range(3):
        n2 = o + (np.arange(B) % (step + 1) == 0)
        nd.copy_(_d(n2))
        g.replay()
        torch.cuda.synchronize()
        ref = slots_ref(table, o, n2, fresh, b, room)
        for got, want in zip((out, slots, cu), (ref[0], ref[1], ref[3])):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert zp.zp_device_status() == (0, 0)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("n,layers,h_kv,d,b,dtype", [
    (1, 1, 1, 64, 16, torch.bfloat16), (1, 2, 8, 128, 16, torch.bfloat16), (37, 1, 2, 64, 16, torch.float32),
    (300, 3, 8, 128, 16, torch.bfloat16), (1025, 2, 3, 48, 7, torch.float32), (5000, 1, 8, 128, 32, torch.bfloat16)])
def test_write_kv(zp, n, layers, h_kv, d, b, dtype, fused):
    g = torch.Generator(device=DEV).manual_seed(n)
    n_total = -(-n // b) + 3
    K = torch.randn(layers, n_total, b, h_kv, d, generator=g, device=DEV).to(dtype)
    V = torch.randn(layers, n_total, b, h_kv, d, generator=g, device=DEV).to(dtype)
    if fused:
        x = torch.randn(layers, n, 5 + 2 * h_kv, d, generator=g, device=DEV).to(dtype)
        k, v = x[:, :, 5:5 + h_kv], x[:, :, 5 + h_kv:]
    else:
        k = torch.randn(layers, n, h_kv, d, generator=g, device=DEV).to(dtype)
        v = torch.randn(layers, n, h_kv, d, generator=g, device=DEV).to(dtype)
    rng = np.random.default_rng(n)
    at = rng.permutation(n_total * b)[:n]
    at[rng.random(n) < 0.2] = -1
    Kr, Vr = K.clone(), V.clone()
    keep = torch.from_numpy(np.nonzero(at >= 0)[0]).to(DEV)
    to = torch.from_numpy(at[at >= 0]).to(DEV)
    Kr.view(layers, -1, h_kv, d)[:, to] = k[:, keep]
    Vr.view(layers, -1, h_kv, d)[:, to] = v[:, keep]
    desc = zp.cache_desc(h_kv, h_kv, d, b, n_total, dtype)
    if layers == 1:
        zp.zp_write_kv(desc, k[0], v[0], _d(at), K[0], V[0])
    else:
        zp.zp_write_kv(desc, k, v, _d(at), K, V)
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    assert torch.equal(K, Kr) and torch.equal(V, Vr)


def test_write_kv_skips_and_records_a_slot_outside_the_cache(zp):
    desc = zp.cache_desc(2, 2, 64, 16, 3, torch.bfloat16)
    K = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    k = torch.ones(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    zp.zp_write_kv(desc, k, k, _d([0, 48, -5, 47]), K, V)
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (7, 0x130)
    hit = K.view(48, -1).sum(1).nonzero().flatten().tolist()
    assert hit == [0, 47] and torch.equal(K, V)


def test_write_kv_far_slots(zp):
    """Slots whose byte offset passes 32 bits (a 6.4 GB cache layer)."""
    h_kv, d, b, n_total = 8, 128, 16, 200000
    K = torch.zeros(n_total, b, h_kv, d, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    at = np.array([n_total * b - 1, 0, 2 ** 21 + 3, n_total * b - 17])
    k = torch.randn(4, h_kv, d, device=DEV).to(torch.bfloat16)
    zp.zp_write_kv(zp.cache_desc(32, h_kv, d, b, n_total, torch.bfloat16), k, -k, _d(at), K, V)
    got = K.view(-1, h_kv, d)[torch.from_numpy(at).to(DEV)]
    assert torch.equal(got, k) and torch.equal(V.view(-1, h_kv, d)[torch.from_numpy(at).to(DEV)], -k)
    assert int((K.view(-1, h_kv * d).abs().amax(1) > 0).sum()) == 4


# ----------------------------------------------------------------------------- groups
def _plan(zp, table, lens, b, total, min_blocks=1, min_members=2):
    B = len(lens)
    plan = zp.prefix_plan(B)
    for t in (plan.prefix_lens, plan.n_groups, plan.group_start, plan.members, plan.group_blocks):
        t.fill_(1234567)  # the call writes every entry
    zp.zp_prefix_plan(_desc(zp, b, total), _d(table), _d(lens), plan, min_blocks=min_blocks, min_members=min_members)
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    return plan


def _check_plan(plan, ref):
    for name, want in ref.items():
        np.testing.assert_array_equal(getattr(plan, name).cpu().numpy(), want, err_msg=name)


@pytest.mark.parametrize("seed,sizes,blocks,own,b,lone,zero", [
    (1, [4], [4], (1, 60), 16, 0, 0), (2, [3, 2, 9], [1, 130, 33], (1, 40), 16, 4, 2), (3, [1, 1, 2], [5, 6, 7], (1, 5), 32, 3, 0),
    (4, [256], [64], (1, 300), 16, 0, 5), (5, list(range(2, 60)), list(range(1, 59)), (1, 90), 16, 30, 10),
    (6, [2] * 1000, [3] * 1000, (1, 20), 16, 96, 0), (7, [4096], [2], (1, 17), 16, 0, 0), (8, [], [], (1, 50), 16, 7, 1),
    (9, [2], [600], (1, 1), 16, 0, 0)])
def test_prefix_plan(zp, seed, sizes, blocks, own, b, lone, zero):
    lens, table, group, total = make_groups(seed, sizes, blocks, own, b, lone, zero)
    for min_blocks, min_members in ((1, 2), (4, 3)):
        ref = plan_ref(table, lens, b, total, min_blocks, min_members)
        _check_plan(_plan(zp, table, lens, b, total, min_blocks, min_members), ref)


@pytest.mark.parametrize("seed", range(8))
def test_prefix_plan_where_requests_depart(zp, seed):
    """Members that leave the prompt early, prompts that extend one another, short leaders, bad ids in a row."""
    rng = np.random.default_rng(seed)
    b = 16
    lens, table, group, total = make_groups(seed, [40, 25, 12], [30, 17, 64], (1, 200), b, 6, 3)
    for s in range(len(lens)):
        nb = -(-int(lens[s]) // b)
        if rng.random() < 0.4 and nb > 2:
            c = int(rng.integers(1, nb))
            table[s, c:nb] = rng.integers(0, total, size=nb - c)  # another continuation
        if rng.random() < 0.1:
            lens[s] = int(rng.integers(0, 4 * b))                 # a request that has just begun
        if rng.random() < 0.1 and nb > 1:
            table[s, int(rng.integers(0, nb))] = rng.choice([-1, total, total + 5])
    ref = plan_ref(table, lens, b, total, 1, 2)
    _check_plan(_plan(zp, table, lens, b, total), ref)


def test_prefix_plan_of_an_empty_batch(zp):
    plan = _plan(zp, np.zeros((0, 4), np.int32), np.zeros(0, np.int32), 16, 4)
    assert plan.n_groups.tolist() == [0] and plan.group_start.tolist() == [0]
