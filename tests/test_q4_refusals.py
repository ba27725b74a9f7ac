"""Refused calls of the 4-bit cache: documented statuses before any device work, the binding's
checks, and the plain form's own properties (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import q4_util as q4


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    return m


P = ctypes.c_void_p(4096)  # never dereferenced: every call below fails its argument checks


def _at(n):
    return ctypes.c_void_p(4096 + n)


def _desc(zp, **kw):
    a = dict(h_q=32, h_kv=8, head_dim=128, block_size=16, n_total_blocks=100, dtype=torch.bfloat16)
    a.update(kw)
    return ctypes.byref(zp.cache_desc(**a))


SHAPE = (dict(head_dim=96), dict(head_dim=256), dict(block_size=8), dict(block_size=24), dict(h_kv=3), dict(h_q=512, h_kv=512),
         dict(n_total_blocks=1 << 28))


def _common(zp, call):
    for kw in SHAPE:
        assert call(desc=_desc(zp, **kw)) == 2, kw
    assert call(desc=_desc(zp, dtype=7)) == 3
    for group in (0, 16, 48, 256, -32):
        assert call(group=group) == 2
    assert call(desc=_desc(zp, head_dim=64), group=128) == 2
    assert zp.lib.zp_q4_tile_bytes(_desc(zp), 48) == 0


def test_tile_bytes(zp):
    for d in (64, 128):
        for group in (32, 64, 128):
            if group <= d:
                assert zp.zp_q4_tile_bytes(zp.cache_desc(8, 2, d, 32, 4, torch.float32), group) == q4.tile_bytes(d, group)
    with pytest.raises(zp.ZPError):
        zp.zp_q4_tile_bytes(zp.cache_desc(8, 2, 64, 32, 4, torch.float32), 128)


@pytest.mark.parametrize("name", ["zp_q4_write_kv", "zp_q4_read_kv"])
def test_rows(zp, name):
    def call(desc=None, group=32, k=P, v=P, ts=1024, nl=0, slots=P, n=3, K=P, V=P, ls=0, layers=1):
        desc = desc or _desc(zp)
        if name == "zp_q4_write_kv":
            return zp.lib.zp_q4_write_kv(desc, group, k, v, ts, nl, slots, n, K, V, ls, layers, None)
        return zp.lib.zp_q4_read_kv(desc, group, K, V, ls, slots, n, k, v, ts, nl, layers, None)

    _common(zp, call)
    layer = 100 * 8 * 1280
    for kw in (dict(n=-1), dict(layers=-1), dict(k=None), dict(v=None), dict(slots=None), dict(K=None), dict(V=None),
               dict(ts=1023), dict(ts=1028), dict(k=_at(8)), dict(V=_at(8)), dict(layers=2, nl=4096, ls=layer - 16),
               dict(layers=2, nl=-8, ls=layer), dict(layers=2, nl=4, ls=layer), dict(layers=2, nl=4096, ls=layer + 8)):
        assert call(**kw) == 1, kw
    assert call(layers=65536, nl=4096, ls=layer) == 2 and call(n=(1 << 30) + 1) == 2
    assert call(n=0, k=None) == 0 and call(layers=0, k=None) == 0


def test_append(zp):
    def call(desc=None, group=32, k=P, v=P, K=P, V=P, table=P, stride=4, lens=P, B=2):
        return zp.lib.zp_q4_append_kv(desc or _desc(zp), group, k, v, K, V, table, stride, lens, B, None)

    _common(zp, call)
    for kw in (dict(B=-1), dict(stride=0), dict(k=None), dict(v=None), dict(K=None), dict(V=None), dict(table=None),
               dict(lens=None), dict(k=_at(8)), dict(K=_at(4))):
        assert call(**kw) == 1, kw
    assert call(B=0, k=None) == 0


def test_decode(zp):
    O = _at(1 << 20)

    def call(desc=None, group=32, q=P, k=P, v=P, table=P, stride=4, lens=P, B=2, out=O, S=None, rows=None, nr=0, w=0, ws=P):
        return zp.lib.zp_q4_decode_attn(desc or _desc(zp), group, q, k, v, table, stride, lens, B, out, S, rows, nr, w, ws,
                                        1 << 40, None)

    _common(zp, call)
    for kw in (dict(B=-1), dict(stride=-1), dict(stride=0), dict(q=None), dict(k=None), dict(v=None), dict(table=None),
               dict(lens=None), dict(out=None), dict(ws=None), dict(S=P, w=0), dict(S=P, w=17), dict(S=P, w=4, rows=P, nr=0),
               dict(q=_at(8)), dict(k=_at(8)), dict(S=_at(4), w=4), dict(ws=_at(4)), dict(out=_at(2)),
               dict(out=P), dict(out=_at(2 * 32 * 128 * 2 - 16)), dict(q=_at(16), out=P)):
        assert call(**kw) == 1, kw
    assert call(B=0, q=None) == 0


def test_compact(zp):
    rows = zp.ScoreRows(4096, 100, 0, None)

    def call(desc=None, group=32, K=P, V=P, ls=0, layers=1, F=None, S=None, src=P, stride=4, dst=P, ts=4, lens=P, keep=P, k=8, n=2):
        return zp.lib.zp_q4_compact_pages(desc or _desc(zp), group, K, V, ls, layers, F, 0, S, src, stride, dst, ts, lens, keep, k,
                                          None, n, None)

    _common(zp, call)
    for kw in (dict(n=-1), dict(k=-1), dict(layers=-1), dict(stride=0), dict(ts=0), dict(K=None), dict(V=None), dict(src=None),
               dict(dst=None), dict(lens=None), dict(keep=None), dict(F=P), dict(F=P, S=ctypes.byref(zp.ScoreRows(None, 1, 0, None))),
               dict(F=P, S=ctypes.byref(zp.ScoreRows(4096, 0, 0, None))), dict(K=_at(8)), dict(layers=2, ls=16)):
        assert call(**kw) == 1, kw
    assert call(k=65) == 4
    assert call(n=65536) == 2 and call(desc=_desc(zp, n_total_blocks=1 << 25)) == 2
    assert call(n=0, K=None) == 0 and call(k=0, K=None) == 0
    assert rows.stride == 100


def test_binding_checks(zp):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    desc = zp.cache_desc(32, 8, 128, 16, 10, torch.bfloat16)
    K, V = zp.zp_q4_cache(desc, device="cpu")
    assert K.shape == (10, 8, 1, 1280) and zp.zp_q4_cache(desc, 64, 3, device="cpu")[1].shape == (3, 10, 8, 1, 1152)
    x = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    q = torch.zeros(3, 32, 128, dtype=torch.bfloat16)
    for bad in (K[:9], K.to(torch.int8), K[..., :1152], K[None]):
        with pytest.raises(ValueError):
            zp.zp_q4_append_kv(desc, x, x, bad, V, i(3, 4), i(3))
        with pytest.raises(ValueError):
            zp.zp_q4_decode_attn(desc, q, bad, V, i(3, 4), i(3), q)
        with pytest.raises(ValueError):
            zp.zp_q4_write_kv(desc, x, x, i(3), bad, V)
    for rows in (x[:2], x.float(), x):                        # (the last: not on a GPU)
        with pytest.raises(ValueError):
            zp.zp_q4_write_kv(desc, rows, rows, i(3), K, V)
        with pytest.raises(ValueError):
            zp.zp_q4_read_kv(desc, K, V, i(3), rows, rows)
    for keep, F, S in ((i(3, 7, 5), None, None), (i(3, 8, 5), torch.zeros(10, 16, 7), None),
                       (i(3, 8, 5), torch.zeros(10, 16, 8), None), (i(3, 8, 5), None, None)):
        with pytest.raises(ValueError):
            zp.zp_q4_compact_pages(desc, K, V, i(3, 4), i(3, 1), i(3), keep, global_F=F, scores=S)


@pytest.mark.parametrize("d,group", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64)])
def test_plain_form(d, group):
    """The plain form's bytes give back what was put in, and no value is further than half a step."""
    rng = np.random.default_rng(d + group)
    x = rng.standard_normal((40, 2, d)).astype(np.float32)
    code, word = q4.quantise(x, group)
    cache = q4.random_cache(rng, 3, 2, d, group, 16)
    slots = rng.permutation(48)[:40]
    for i, s in enumerate(slots):
        for h in range(2):
            q4.put_row(cache, int(s), h, code[i, h], word[i, h], 16)
    got, step, lo = q4.get_rows(cache, slots, d, group, 16)
    assert np.array_equal(got, code)
    err = np.abs(q4.values(got, step, lo, group) - x).reshape(40, 2, -1, group)
    assert (err <= step[..., None] * 0.5 + 2.0 ** -22).all()


def test_compact_ranks(zp):
    """Ranks are counted in 32 bits, a few rounds ahead."""
    args = (_desc(zp), 32, P, P, 0, 1, None, 0, None, P, 4, P, 1 << 30, P, P)
    assert zp.lib.zp_q4_compact_pages(*args, (1 << 30) + 1, None, 1, None) == 2


def test_read_into_one_layer(zp):
    """Outputs of several layers that lie on one another are refused; the same rows stored into several layers are not."""
    size = 100 * 8 * 1280
    args = (_desc(zp), 32, P, P, size, P, 4, P, P, 1024)
    assert zp.lib.zp_q4_read_kv(*args, 0, 2, None) == 1
    assert zp.lib.zp_q4_read_kv(*args, 1016, 2, None) == 1
