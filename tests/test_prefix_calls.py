"""Calls of the prefix operators that are refused because they could not be answered
rightly (no GPU needed: the checks come before any device work)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    return m


def test_scored_output_over_the_queries(zp):
    """The score reads q after out is written: a scored call must not write its outputs there."""
    desc = ctypes.byref(zp.cache_desc(32, 8, 128, 16, 100, torch.bfloat16))
    plan = ctypes.byref(zp._PrefixGroups(*[4096] * 5))
    P, rows = ctypes.c_void_p(1 << 20), 2 * 32 * 128 * 2

    def call(out, S):
        return zp.lib.zp_prefix_decode_attn(desc, ctypes.c_void_p(1 << 24), P, P, P, 4, P, 2, plan, ctypes.c_void_p(out), S,
                                            None, 0, 16, P, 0, None)

    S = ctypes.c_void_p(1 << 26)
    for out in (1 << 24, (1 << 24) + 16, (1 << 24) - rows + 16):
        assert call(out, S) == 1
        assert b"overlaps" in zp.lib.zp_last_error()
    for out in ((1 << 24) + rows, (1 << 24) - rows):
        call(out, S)
        assert b"overlaps" not in zp.lib.zp_last_error()
    call(1 << 24, None)  # not scored: each row is read before it is written
    assert b"overlaps" not in zp.lib.zp_last_error()


def test_plan_of_another_device(zp, monkeypatch):
    """A plan's arrays are checked when it is made; a call with another device current must not hand them to its kernels."""
    class On0(torch.Tensor):  # stands in for a tensor of device 0
        def get_device(self):
            return 0
    i = lambda *s: torch.zeros(*s, dtype=torch.int32).as_subclass(On0)  # noqa: E731
    monkeypatch.setattr(zp, "_device", lambda: 0)
    plan = zp.PrefixPlan(i(2), i(1), i(3), i(2), i(2))
    desc = zp.cache_desc(32, 8, 128, 16, 10, torch.bfloat16)
    q = torch.zeros(2, 32, 128, dtype=torch.bfloat16)
    K = torch.zeros(10, 16, 8, 128, dtype=torch.bfloat16)
    monkeypatch.setattr(zp, "_device", lambda: 1)
    monkeypatch.setattr(zp, "_ptr_on", lambda t, dev, name: None if t is None else t.data_ptr())  # every other tensor is there
    monkeypatch.setattr(zp, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(zp, "lib", None)  # nothing is launched
    with pytest.raises(ValueError, match="device"):
        zp.zp_prefix_plan(desc, i(2, 4), i(2), plan)
    with pytest.raises(ValueError, match="device"):
        zp.zp_prefix_decode_attn(desc, q, K, K, i(2, 4), i(2), plan, q.clone())


def test_a_plans_arrays_are_not_replaced(zp, monkeypatch):
    """The library holds the arrays' addresses: another tensor under the same name would not be seen, and the old one's
    memory would be read after it is gone."""
    monkeypatch.setattr(zp, "_device", lambda: -1)  # (tensors of the host)
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    plan = zp.PrefixPlan(i(2), i(1), i(3), i(2), i(2))
    at = plan.members.data_ptr()
    for name in ("prefix_lens", "n_groups", "group_start", "members", "group_blocks"):
        with pytest.raises(AttributeError):
            setattr(plan, name, i(2))
    plan.members[:] = i(2) + 1
    assert plan.members.data_ptr() == at == plan._c.members and plan.members.tolist() == [1, 1]


def test_default_workspace(zp, monkeypatch):
    """The default workspace comes from torch's public allocator calls, for the stream of the work, and is given back
    also when the call fails."""
    log = []

    class Lib:
        def zp_prefix_decode_workspace_size(self, *a):
            return 1000

        def zp_prefix_decode_attn(self, *a):
            log.append(("call", a[-3:]))
            raise RuntimeError("stop")

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(zp, "lib", Lib())
    monkeypatch.setattr(zp, "_device", lambda: -1)  # (tensors of the host)
    monkeypatch.setattr(torch.cuda, "caching_allocator_alloc", lambda n, dev, st: log.append(("alloc", n, dev, st)) or 4096)
    monkeypatch.setattr(torch.cuda, "caching_allocator_delete", lambda at: log.append(("delete", at)))
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    plan = zp.PrefixPlan(i(2), i(1), i(3), i(2), i(2))
    q = torch.zeros(2, 32, 128, dtype=torch.bfloat16)
    K = torch.zeros(10, 16, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="stop"):
        zp.zp_prefix_decode_attn(zp.cache_desc(32, 8, 128, 16, 10, torch.bfloat16), q, K, K, i(2, 4), i(2), plan,
                                 torch.zeros_like(q), stream=Stream())
    assert log == [("alloc", 1000, -1, 77), ("call", (4096, 1000, 77)), ("delete", 4096)]


def test_write_kv_strides_that_mean_nothing(zp, monkeypatch):
    """One token, one kv head or one layer: the stride along that dimension is any number, and differs between k and v."""
    got = []

    class Lib:
        def zp_write_kv(self, desc, k, v, token_stride, layer_stride, slots, n, K, V, cache_layer_stride, layers, stream):
            got.append((token_stride, layer_stride, n, layers))
            return 0

    monkeypatch.setattr(zp, "lib", Lib())
    monkeypatch.setattr(zp, "_device", lambda: -1)  # (tensors of the host)
    monkeypatch.setattr(zp, "_raw_stream", lambda stream, dev: 0)
    bf, i = torch.bfloat16, lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    d = 64

    def call(k, v, n, h_kv, layers=None):
        K = torch.zeros(*([layers] if layers else []), 3, 16, h_kv, d, dtype=bf)
        zp.zp_write_kv(zp.cache_desc(8, h_kv, d, 16, 3, bf), k, v, i(n), K, K.clone())
        return got.pop()

    fused = torch.zeros(1, 12, d, dtype=bf)
    assert call(fused[:, 8:10], torch.zeros(1, 2, d, dtype=bf), 1, 2) == (2 * d, 0, 1, 1)            # one token
    assert call(torch.zeros(5, 1027, dtype=bf)[1:2, :2 * d].view(1, 2, d), torch.zeros(1, 2, d, dtype=bf), 1, 2)[0] == 2 * d
    swapped = torch.zeros(1, 7, d, dtype=bf).transpose(0, 1)                                          # one head
    assert call(swapped, torch.zeros(7, 1, d, dtype=bf), 7, 1) == (d, 0, 7, 1)
    assert call(torch.zeros(4, 7, 2, d, dtype=bf)[2:3], torch.zeros(7, 1, 2, d, dtype=bf).transpose(0, 1), 7, 2, 1) == (2 * d, 0, 7, 1)
    assert call(torch.zeros(2, 7, 6, d, dtype=bf)[:, :, :2], torch.zeros(2, 7, 6, d, dtype=bf)[:, :, 4:], 7, 2, 2) == (6 * d, 42 * d, 7, 2)
    for k, v in ((torch.zeros(7, 2, 2 * d, dtype=bf)[..., ::2], torch.zeros(7, 2, d, dtype=bf)),          # elements apart
                 (torch.zeros(2, 7, d, dtype=bf).transpose(0, 1), torch.zeros(2, 7, d, dtype=bf).transpose(0, 1)),  # heads apart
                 (torch.zeros(7, 4, d, dtype=bf)[:, :2], torch.zeros(7, 2, d, dtype=bf))):                 # other strides
        with pytest.raises(ValueError):
            call(k, v, 7, 2)
