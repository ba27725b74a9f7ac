"""Rows quantised into a 4-bit cache, read back and moved: the bytes, bit for bit,
against the plain form."""
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
    import ctypes
    code, detail = ctypes.c_int32(), ctypes.c_int32()
    zp._check(zp.lib.zp_device_status(ctypes.byref(code), ctypes.byref(detail), 1))
    return code.value, detail.value


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _rows(rng, shape, dtype):
    """Rows with the values that decide roundings: normal ones, ties, flat groups, far offsets, tiny and huge ones."""
    x = rng.standard_normal(shape).astype(np.float32)
    flat = x.reshape(-1, 32)
    kind = rng.integers(0, 8, size=len(flat))
    flat[kind == 1] = np.round(flat[kind == 1] * 8) / 4          # many exact ties
    flat[kind == 2] = flat[kind == 2][:, :1]                     # all equal
    flat[kind == 3] += 300.0
    flat[kind == 4] *= np.float32(1e-39)                         # subnormal
    flat[kind == 5] *= np.float32(1e37)
    flat[kind == 6] = np.where(rng.random(flat[kind == 6].shape) < 0.5, 0.0, -0.0)
    t = torch.from_numpy(x)
    return t.bfloat16() if dtype == "bf16" else t


def _ref_write(cache, rows, slots, group, b):
    code, word = q4.quantise(rows.float().numpy(), group)
    for i, s in enumerate(slots):
        if 0 <= s < cache.shape[0] * b:
            for h in range(cache.shape[1]):
                q4.put_row(cache, int(s), h, code[i, h], word[i, h], b)


SHAPES = [("bf16", 8, 128, 32, 16), ("bf16", 4, 128, 64, 32), ("bf16", 1, 128, 128, 48), ("bf16", 3, 64, 32, 16),
          ("f32", 8, 128, 32, 16), ("f32", 2, 64, 64, 64), ("f32", 5, 64, 32, 16)]


@pytest.mark.parametrize("dtype,h_kv,d,group,b", SHAPES)
@pytest.mark.parametrize("n,layers,fused", [(1, 1, False), (37, 1, True), (150, 3, True)])
def test_write_and_read(zp, dtype, h_kv, d, group, b, n, layers, fused):
    rng = np.random.default_rng(n * 7 + d + group)
    n_total = -(-n // b) + 3
    desc = zp.cache_desc(h_kv, h_kv, d, b, n_total, torch.bfloat16 if dtype == "bf16" else torch.float32)
    ref = np.stack([[q4.random_cache(rng, n_total, h_kv, d, group, b) for _ in range(layers)] for _ in range(2)])
    K, V = _dev(ref[0]), _dev(ref[1])
    slots = rng.permutation(n_total * b)[:n].astype(np.int32)
    slots[5::11] = -1
    if fused:
        wide = _rows(rng, (layers, n, 3 * h_kv, d), dtype)
        k, v = wide[:, :, :h_kv], wide[:, :, 2 * h_kv:]
        wide = wide.cuda()
        kd, vd = wide[:, :, :h_kv], wide[:, :, 2 * h_kv:]
    else:
        k, v = _rows(rng, (layers, n, h_kv, d), dtype), _rows(rng, (layers, n, h_kv, d), dtype)
        kd, vd = k.cuda(), v.cuda()
    zp.zp_q4_write_kv(desc, kd, vd, _dev(slots), K, V, group=group)
    for l in range(layers):
        _ref_write(ref[0][l], k[l], slots, group, b)
        _ref_write(ref[1][l], v[l], slots, group, b)
    assert np.array_equal(K.cpu().numpy(), ref[0]) and np.array_equal(V.cpu().numpy(), ref[1])

    # and back: every slot once and some twice, padding rows left as they were
    want = np.concatenate([rng.permutation(n_total * b), [0, -1, 3, -5, 0]]).astype(np.int32)
    out = torch.full((2, layers, len(want), h_kv + 1, d), 7.0, dtype=kd.dtype, device="cuda")
    zp.zp_q4_read_kv(desc, K, V, _dev(want), out[0, :, :, :h_kv], out[1, :, :, :h_kv], group=group)
    got = out.cpu()
    for i in range(2):
        for l in range(layers):
            val = q4.values(*q4.get_rows(ref[i][l], np.maximum(want, 0), d, group, b), group)
            val = torch.from_numpy(val).float()     # lo + c * step: one rounding to 32 bits, then one to the type
            val[want < 0] = 7.0
            assert torch.equal(got[i, l, :, :h_kv], val.to(got.dtype))
    assert bool((got[:, :, :, h_kv] == 7.0).all())


@pytest.mark.parametrize("dtype,h_kv,d,group", [("bf16", 40, 128, 32), ("bf16", 65, 64, 64), ("f32", 33, 128, 128)])
def test_many_heads(zp, dtype, h_kv, d, group):
    """Rows of more pieces than a CTA has threads, a multiple of those or not."""
    rng = np.random.default_rng(h_kv)
    desc = zp.cache_desc(h_kv, h_kv, d, 16, 2, torch.bfloat16 if dtype == "bf16" else torch.float32)
    ref = q4.random_cache(rng, 2, h_kv, d, group, 16)
    K, V = _dev(ref), _dev(ref)
    k = _rows(rng, (11, h_kv, d), dtype)
    slots = rng.permutation(32)[:11].astype(np.int32)
    zp.zp_q4_write_kv(desc, k.cuda(), k.cuda(), _dev(slots), K, V, group=group)
    _ref_write(ref, k, slots, group, 16)
    assert np.array_equal(K.cpu().numpy(), ref) and np.array_equal(V.cpu().numpy(), ref)
    out = torch.empty(2, 11, h_kv, d, dtype=k.dtype, device="cuda")
    zp.zp_q4_read_kv(desc, K, V, _dev(slots), out[0], out[1], group=group)
    want = torch.from_numpy(q4.values(*q4.get_rows(ref, slots, d, group, 16), group)).float().to(k.dtype)
    assert torch.equal(out[0].cpu(), want) and torch.equal(out[1].cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_on_16_bytes(zp, dtype):
    """Rows and layers that begin on 16 but not on 32 bytes, for both directions."""
    rng = np.random.default_rng(3)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    n, h_kv, d, layers, pad = 21, 3, 64, 2, 8 if dtype == "bf16" else 4
    desc = zp.cache_desc(h_kv, h_kv, d, 16, 3, t)
    ref = np.stack([q4.random_cache(rng, 3, h_kv, d, 32, 16) for _ in range(layers)])
    K, V = _dev(ref), _dev(ref)
    k = _rows(rng, (layers, n, h_kv, d), dtype)
    place = lambda: torch.zeros(pad + layers * n * (h_kv * d + pad), dtype=t, device="cuda").as_strided(  # noqa: E731
        (layers, n, h_kv, d), (n * (h_kv * d + pad), h_kv * d + pad, d, 1), pad)
    kd, vd = place(), place()
    kd.copy_(k)
    vd.copy_(k)
    assert kd.data_ptr() % 32 == 16
    slots = rng.permutation(48)[:n].astype(np.int32)
    zp.zp_q4_write_kv(desc, kd, vd, _dev(slots), K, V)
    for l in range(layers):
        _ref_write(ref[l], k[l], slots, 32, 16)
    assert np.array_equal(K.cpu().numpy(), ref) and np.array_equal(V.cpu().numpy(), ref)
    ko, vo = place(), place()
    zp.zp_q4_read_kv(desc, K, V, _dev(slots), ko, vo)
    for l in range(layers):
        want = torch.from_numpy(q4.values(*q4.get_rows(ref[l], slots, d, 32, 16), 32)).float().to(t)
        assert torch.equal(ko[l].cpu(), want) and torch.equal(vo[l].cpu(), want)


def test_far_blocks(zp):
    """A cache of more than 4 GB: its last blocks are written, read, moved and attended to."""
    h_q, h_kv, d, group, b = 8, 4, 128, 32, 16
    n_total = (1 << 32) // (h_kv * q4.tile_bytes(d, group)) + 40
    desc = zp.cache_desc(h_q, h_kv, d, b, n_total, torch.float32)
    K, V = zp.zp_q4_cache(desc, group)
    assert K.numel() > 1 << 32
    rng = np.random.default_rng(4)
    L = 100
    table = np.full((1, 9), -1, np.int32)
    table[0, :7] = n_total - 1 - rng.permutation(30)[:7]
    slots = (table[0, np.arange(L) // b].astype(np.int64) * b + np.arange(L) % b).astype(np.int32)
    k, v = _rows(rng, (L, h_kv, d), "f32"), torch.from_numpy(rng.standard_normal((L, h_kv, d)).astype(np.float32))
    k = torch.where(k.abs() < 10, k, 0.5)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    zp.zp_q4_write_kv(desc, k[:L - 1].cuda(), v[:L - 1].cuda(), _dev(slots[:L - 1]), K, V, group=group)
    zp.zp_q4_append_kv(desc, k[L - 1:].cuda(), v[L - 1:].cuda(), K, V, _dev(table), lens, group=group)
    want = []
    for x in (k, v):
        code, word = q4.quantise(x.numpy(), group)
        want.append(torch.from_numpy(q4.values(code, q4.bf16_value(word & 0xFFFF), q4.bf16_value(word >> 16), group)))
    ko, vo = torch.empty(L, h_kv, d, device="cuda"), torch.empty(L, h_kv, d, device="cuda")
    zp.zp_q4_read_kv(desc, K, V, _dev(slots), ko, vo, group=group)
    assert torch.equal(ko.cpu(), want[0].float()) and torch.equal(vo.cpu(), want[1].float())
    assert int(K[:64].max()) == 0 and int(V[:64].max()) == 0   # nothing where a 32-bit offset would have gone
    q = torch.randn(1, h_q, d, device="cuda")
    out = torch.empty_like(q)
    zp.zp_q4_decode_attn(desc, q, K, V, _dev(table), lens, out, group=group)
    x = torch.einsum("hgd,thd->hgt", q.cpu().double().view(h_kv, 2, d), want[0]) / d ** 0.5
    ref = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), want[1]).reshape(1, h_q, d)
    # logits of up to 64 in 32 bits (2^-24 of the 128 terms' magnitudes, at most 2^11 in all): 2^-13 in a weight
    assert (out.cpu().double() - ref).abs().max() < 2.0 ** -13 * want[1].abs().max()
    keep = torch.from_numpy(np.stack([np.sort(rng.permutation(L)[:40]) for _ in range(h_kv)])[None].astype(np.int32)).cuda()
    zp.zp_q4_compact_pages(desc, K, V, _dev(table), _dev(table[:, :3].copy()), lens, keep, group=group)
    zp.zp_q4_read_kv(desc, K, V, _dev(slots[:40]), ko[:40], vo[:40], group=group)
    for h in range(h_kv):
        at = keep[0, h].cpu().long()
        assert torch.equal(ko[:40, h].cpu(), want[0].float()[at, h]) and torch.equal(vo[:40, h].cpu(), want[1].float()[at, h])


def test_not_finite(zp):
    """A NaN, an infinity or a spread past the largest float takes its group, and no other."""
    d, group, b = 128, 32, 16
    for dtype in (torch.bfloat16, torch.float32):
        desc = zp.cache_desc(1, 1, d, b, 2, dtype)
        rng = np.random.default_rng(3)
        x = torch.from_numpy(rng.standard_normal((6, 1, d)).astype(np.float32))
        x[0, 0, 5], x[1, 0, 40], x[2, 0, 127] = float("nan"), float("inf"), -float("inf")
        x[3, 0, 64], x[3, 0, 65] = 3e38, -3e38
        x[4, 0, :32] = float("nan")
        x = x.to(dtype)
        K, V = zp.zp_q4_cache(desc, group)
        slots = torch.arange(6, dtype=torch.int32, device="cuda")
        zp.zp_q4_write_kv(desc, x.cuda(), x.cuda(), slots, K, V, group=group)
        ref = np.zeros(tuple(K.shape), np.uint8)
        _ref_write(ref, x, range(6), group, b)
        assert np.array_equal(K.cpu().numpy(), ref)
        out = torch.zeros(2, 6, 1, d, dtype=dtype, device="cuda")
        zp.zp_q4_read_kv(desc, K, V, slots, out[0], out[1], group=group)
        nan = torch.isnan(out[0, :, 0].cpu()).reshape(6, 4, 32)
        want = torch.zeros(6, 4, dtype=torch.bool)
        want[0, 0] = want[1, 1] = want[2, 3] = want[3, 2] = want[4, 0] = True
        assert torch.equal(nan.all(-1), want) and torch.equal(nan.any(-1), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_error_is_half_a_step(zp, dtype):
    rng = np.random.default_rng(11)
    x = rng.standard_normal((300, 4, 128)).astype(np.float32)
    x = (torch.from_numpy(x).bfloat16().float() if dtype == "bf16" else torch.from_numpy(x)).numpy()
    code, word = q4.quantise(x, 32)
    step = q4.bf16_value(word & 0xFFFF)
    err = np.abs(q4.values(code, step, q4.bf16_value(word >> 16), 32) - x).reshape(300, 4, 4, 32)
    # (fp32 rows: x - lo is rounded to 32 bits before it is divided)
    assert (err <= step[..., None] * 0.5 + (0 if dtype == "bf16" else 2.0 ** -22)).all()


@pytest.mark.parametrize("dtype,h_kv,d,group,b", SHAPES)
def test_append(zp, dtype, h_kv, d, group, b):
    rng = np.random.default_rng(d + group + h_kv)
    B, stride = 33, 5
    lens = rng.integers(1, stride * b + 1, size=B)
    lens[3] = 0
    lens[4], lens[5], lens[6] = 1, b, b + 1
    table = rng.permutation(B * stride).reshape(B, stride).astype(np.int32)
    desc = zp.cache_desc(2 * h_kv, h_kv, d, b, B * stride, torch.bfloat16 if dtype == "bf16" else torch.float32)
    ref = np.stack([q4.random_cache(rng, B * stride, h_kv, d, group, b) for _ in range(2)])
    K, V = _dev(ref[0]), _dev(ref[1])
    k, v = _rows(rng, (B, h_kv, d), dtype), _rows(rng, (B, h_kv, d), dtype)
    zp.zp_q4_append_kv(desc, k.cuda(), v.cuda(), K, V, _dev(table), _dev(lens.astype(np.int32)), group=group)
    slots = [int(table[s, (L - 1) // b]) * b + (L - 1) % b if L else -1 for s, L in enumerate(lens)]
    _ref_write(ref[0], k, slots, group, b)
    _ref_write(ref[1], v, slots, group, b)
    assert np.array_equal(K.cpu().numpy(), ref[0]) and np.array_equal(V.cpu().numpy(), ref[1])


@pytest.mark.parametrize("dtype,h_kv,d,group,b", SHAPES)
@pytest.mark.parametrize("L,k,in_place", [(40, 32, True), (200, 150, True), (200, 150, False), (4500, 4400, True), (90, 90, True)])
def test_compact(zp, dtype, h_kv, d, group, b, L, k, in_place):
    if L > 1000 and h_kv > 3:
        pytest.skip("the long case runs with few heads")
    rng = np.random.default_rng(L + k + d)
    n, layers = 3, 2
    stride, targets = -(-L // b) + 1, -(-k // b)
    lens = np.array([L, max(L - 3, k), L - 1])
    n_total = n * (stride + targets)
    ids = rng.permutation(n_total)
    table = ids[:n * stride].reshape(n, stride).astype(np.int32)
    dst = table[:, :targets].copy() if in_place else ids[n * stride:].reshape(n, targets).astype(np.int32)
    k_seq = np.array([k, k // 2, k], dtype=np.int32)
    keep = np.full((layers, n, h_kv, k), -1, dtype=np.int32)
    for l in range(layers):
        for i in range(n):
            for h in range(h_kv):
                m = min(k_seq[i], lens[i])
                keep[l, i, h, :m] = np.sort(rng.permutation(lens[i])[:m])
    ref = np.stack([[q4.random_cache(rng, n_total, h_kv, d, group, b) for _ in range(layers)] for _ in range(2)])
    K, V = _dev(ref[0]), _dev(ref[1])
    F = rng.random((layers, n_total, b, h_kv)).astype(np.float32)
    S = rng.random((layers, n + 2, h_kv, L + 5)).astype(np.float32)
    rows = np.array([4, 0, 2], dtype=np.int32)
    Fd = _dev(F)
    desc = zp.cache_desc(h_kv, h_kv, d, b, n_total, torch.bfloat16 if dtype == "bf16" else torch.float32)
    zp.zp_q4_compact_pages(desc, K, V, _dev(table), _dev(dst), _dev(lens.astype(np.int32)), _dev(keep), global_F=Fd,
                           scores=_dev(S), rows=_dev(rows), k_seq=_dev(k_seq), group=group)
    for l in range(layers):
        for x in range(2):
            old = ref[x][l].copy()
            for i in range(n):
                for h in range(h_kv):
                    m = min(k_seq[i], lens[i])
                    pos = keep[l, i, h, :m]
                    code, step, lo = q4.get_rows(old[:, h:h + 1], table[i, pos // b] * b + pos % b, d, group, b)
                    word = (step.view(np.uint32) >> 16) | lo.view(np.uint32)
                    for r in range(m):
                        slot = int(dst[i, r // b]) * b + r % b
                        q4.put_row(ref[x][l], slot, h, code[r, 0], word[r, 0], b)
                        if x == 0:
                            F[l, slot // b, slot % b, h] = S[l, rows[i], h, pos[r]]
    assert np.array_equal(K.cpu().numpy(), ref[0]) and np.array_equal(V.cpu().numpy(), ref[1])
    assert np.array_equal(Fd.cpu().numpy(), F)


def test_compact_under_budget(zp):
    """Sequences shorter than k (their keep lists padded with -1), budgets of 0 and sequences of no tokens."""
    rng = np.random.default_rng(12)
    h_kv, d, group, b, k = 2, 64, 32, 16, 40
    lens = np.array([25, 0, 64, 17], np.int32)
    k_seq = np.array([40, 40, 0, 16], np.int32)
    table = rng.permutation(40)[:20].reshape(4, 5).astype(np.int32)
    dst = np.setdiff1d(np.arange(60), table)[:12].reshape(4, 3).astype(np.int32)
    keep = np.full((4, h_kv, k), -1, np.int32)
    keep[0, :, :25] = np.arange(25)
    keep[3, 0, :16], keep[3, 1, :16] = np.arange(16), np.arange(1, 17)
    desc = zp.cache_desc(h_kv, h_kv, d, b, 60, torch.bfloat16)
    ref = q4.random_cache(rng, 60, h_kv, d, group, b)
    K, V = _dev(ref), _dev(ref)
    zp.zp_q4_compact_pages(desc, K, V, _dev(table), _dev(dst), _dev(lens), _dev(keep), k_seq=_dev(k_seq), group=group)
    old = ref.copy()
    for i, m in ((0, 25), (3, 16)):
        for h in range(h_kv):
            pos = keep[i, h, :m]
            code, step, lo = q4.get_rows(old[:, h:h + 1], table[i, pos // b] * b + pos % b, d, group, b)
            word = (step.view(np.uint32) >> 16) | lo.view(np.uint32)
            for r in range(m):
                q4.put_row(ref, int(dst[i, r // b]) * b + r % b, h, code[r, 0], word[r, 0], b)
    assert np.array_equal(K.cpu().numpy(), ref) and np.array_equal(V.cpu().numpy(), ref)


def test_bad_indices(zp):
    """Slots, lengths, blocks and positions out of range are recorded and skipped; their neighbours are served."""
    rng = np.random.default_rng(8)
    h_kv, d, group, b, n_total = 2, 64, 32, 16, 6
    desc = zp.cache_desc(4, h_kv, d, b, n_total, torch.float32)
    x = _rows(rng, (3, h_kv, d), "f32")
    start = q4.random_cache(rng, n_total, h_kv, d, group, b)

    def check(call, slots, detail):
        ref, K, V = start.copy(), _dev(start), _dev(start)
        call(K, V)
        assert _status(zp) == (7, detail)
        _ref_write(ref, x, slots, group, b)
        assert np.array_equal(K.cpu().numpy(), ref) and np.array_equal(V.cpu().numpy(), ref)

    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    xd = x.cuda()
    check(lambda K, V: zp.zp_q4_write_kv(desc, xd, xd, i(3, n_total * b, 7), K, V, group=group), (3, -1, 7), 0x150)
    table = i(1, 2, 3, -1, 5, n_total).view(3, 2)
    check(lambda K, V: zp.zp_q4_append_kv(desc, xd, xd, K, V, table, i(20, 33, 4), group=group), (2 * b + 3, -1, 5 * b + 3), 0x151)
    check(lambda K, V: zp.zp_q4_append_kv(desc, xd, xd, K, V, table, i(20, 20, 32), group=group), (2 * b + 3, -1, -1), 0x152)
    K, V = _dev(start), _dev(start)
    out = torch.full((2, 2, h_kv, d), 5.0, device="cuda")
    zp.zp_q4_read_kv(desc, K, V, i(n_total * b, 4), out[0], out[1], group=group)
    assert _status(zp) == (7, 0x153)
    val = torch.from_numpy(q4.values(*q4.get_rows(start, [4], d, group, b), group)).float()[0]
    assert bool((out[0, 0] == 5.0).all()) and torch.equal(out[0, 1].cpu(), val)
    for table, dst, detail in ((i(1, n_total).view(1, 2), i(4).view(1, 1), 0x154), (i(1, 2).view(1, 2), i(-1).view(1, 1), 0x155)):
        K, V = _dev(start), _dev(start)
        keep = i(0, 17, 1, 18).view(1, h_kv, 2)
        zp.zp_q4_compact_pages(desc, K, V, table, dst, i(32), keep, group=group)
        assert _status(zp) == (7, detail)
        ref = start.copy()
        if detail == 0x154:  # the ranks whose source is inside the cache moved
            for h in range(h_kv):
                code, step, lo = q4.get_rows(start[:, h:h + 1], [b + h], d, group, b)
                q4.put_row(ref, 4 * b, h, code[0, 0], ((step.view(np.uint32) >> 16) | lo.view(np.uint32))[0, 0], b)
        assert np.array_equal(K.cpu().numpy(), ref)
