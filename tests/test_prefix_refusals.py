"""Refused calls of the shared-prompt operators: documented statuses before any
device work, and the binding's checks (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    return m


P = ctypes.c_void_p(4096)  # never dereferenced: every call below fails its argument checks


def _desc(zp, **kw):
    a = dict(h_q=32, h_kv=8, head_dim=128, block_size=16, n_total_blocks=100, dtype=torch.bfloat16)
    a.update(kw)
    return ctypes.byref(zp.cache_desc(**a))


def test_build_slots(zp):
    def call(desc=None, table=P, out=P, stride=4, old=P, new=P, B=2, fresh=None, nf=0, slots=P, n=8, cu=P):
        return zp.lib.zp_build_slots(desc or _desc(zp), table, out, stride, old, new, B, fresh, nf, slots, None, n, cu, None, None)

    assert call(desc=_desc(zp, h_kv=3)) == 2
    assert call(desc=_desc(zp, dtype=9)) == 3
    for kw in (dict(B=-1), dict(stride=0), dict(nf=-1), dict(n=-1), dict(table=None), dict(out=None), dict(old=None),
               dict(new=None), dict(cu=None), dict(slots=None), dict(nf=3), dict(out=ctypes.c_void_p(4096 + 16))):
        assert call(**kw) == 1, kw
    assert call(B=4097) == 2
    assert call(desc=_desc(zp, n_total_blocks=1 << 28)) == 2   # slots beyond 32 bits
    assert call(B=4096, stride=1 << 16) == 2                   # tokens beyond 32 bits


def test_write_kv(zp):
    def call(desc=None, k=P, v=P, ts=1024, nl=0, slots=P, n=3, K=P, V=P, ls=0, layers=1):
        return zp.lib.zp_write_kv(desc or _desc(zp), k, v, ts, nl, slots, n, K, V, ls, layers, None)

    assert call(desc=_desc(zp, head_dim=20)) == 2
    for kw in (dict(n=-1), dict(layers=-1), dict(k=None), dict(v=None), dict(slots=None), dict(K=None), dict(V=None),
               dict(ts=1023), dict(ts=1028), dict(k=ctypes.c_void_p(4104)), dict(layers=2, nl=4096, ls=1024),
               dict(layers=2, nl=-8, ls=1 << 21), dict(layers=2, nl=4, ls=1 << 21)):
        assert call(**kw) == 1, kw
    assert call(layers=65536, nl=4096, ls=1 << 21) == 2
    assert call(n=0, k=None) == 0 and call(layers=0, k=None) == 0


def _groups(zp, **kw):
    a = dict(prefix_lens=4096, n_groups=4096, group_start=4096, members=4096, group_blocks=4096)
    a.update(kw)
    return ctypes.byref(zp._PrefixGroups(*a.values()))


def test_prefix_plan(zp):
    def call(desc=None, table=P, stride=4, lens=P, B=2, mb=1, mm=2, plan=None):
        return zp.lib.zp_prefix_plan(desc or _desc(zp), table, stride, lens, B, mb, mm, plan or _groups(zp), None)

    assert call(desc=_desc(zp, block_size=0)) == 2
    for kw in (dict(B=-1), dict(stride=0), dict(mb=0), dict(mm=1), dict(table=None), dict(lens=None),
               *(dict(plan=_groups(zp, **{k: None})) for k in ("prefix_lens", "n_groups", "group_start", "members", "group_blocks"))):
        assert call(**kw) == 1, kw
    assert call(B=4097) == 2 and call(stride=1 << 20) == 2


def test_prefix_decode(zp):
    def call(desc=None, q=P, k=P, v=P, table=P, stride=4, lens=P, B=2, plan=None, out=P, S=None, rows=None, nr=0, w=0, ws=P):
        return zp.lib.zp_prefix_decode_attn(desc or _desc(zp), q, k, v, table, stride, lens, B, plan or _groups(zp), out, S,
                                            rows, nr, w, ws, 1 << 40, None)

    assert call(desc=_desc(zp, dtype=9)) == 3
    for kw in (dict(B=-1), dict(stride=-1), dict(stride=0), dict(q=None), dict(k=None), dict(v=None), dict(table=None),
               dict(lens=None), dict(out=None), dict(ws=None), dict(S=P, w=0), dict(S=P, w=17), dict(S=P, w=4, rows=P, nr=0),
               dict(q=ctypes.c_void_p(4104)), dict(S=ctypes.c_void_p(4100), w=4), dict(ws=ctypes.c_void_p(4100)),
               *(dict(plan=_groups(zp, **{k: None})) for k in ("prefix_lens", "n_groups", "group_start", "members", "group_blocks"))):
        assert call(**kw) == 1, kw
    assert call(B=4096, stride=1 << 20) == 2
    assert call(B=0, q=None) == 0


def test_binding_checks(zp):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    desc = zp.cache_desc(32, 8, 128, 16, 10, torch.bfloat16)
    with pytest.raises(ValueError):
        zp.zp_build_slots(desc, i(2, 4), i(2), i(2), i(3), i(3))          # not on a GPU
    with pytest.raises(ValueError):
        zp.zp_build_slots(desc, i(2, 4).long(), i(2), i(2), i(3), i(3))   # not int32
    with pytest.raises(ValueError):
        zp.zp_build_slots(desc, i(2, 4), i(2), i(2), i(3), i(3), table_out=i(2, 5))
    k = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    K = torch.zeros(10, 16, 8, 128, dtype=torch.bfloat16)
    for args in ((k[:2], k, i(3), K, K), (k.float(), k, i(3), K, K), (k, k, i(3), K, K), (k, k, i(3), K[:9], K)):
        with pytest.raises(ValueError):
            zp.zp_write_kv(desc, *args)
    with pytest.raises(ValueError):
        zp.PrefixPlan(i(2), i(1), i(3), i(2), i(2))                       # not on a GPU
