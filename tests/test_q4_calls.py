"""Calls of the 4-bit cache as the binding and the library make them: where scratch comes from, and what is refused
because it could not be answered rightly (no GPU needed: the checks come before any device work)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    return m


def test_default_workspace(zp, monkeypatch):
    """The default workspace comes from torch's public allocator calls, for the stream of the work, and is given back
    also when the call fails."""
    log = []

    class Lib:
        def zp_q4_decode_workspace_size(self, *a):
            return 1000

        def zp_q4_decode_attn(self, *a):
            log.append(("call", a[-3:]))
            raise RuntimeError("stop")

    class Stream:
        cuda_stream = 77

    desc = zp.cache_desc(32, 8, 128, 16, 10, torch.bfloat16)
    K, V = zp.zp_q4_cache(desc, device="cpu")
    monkeypatch.setattr(zp, "lib", Lib())
    monkeypatch.setattr(zp, "_Q4_SIZES", {})
    monkeypatch.setattr(zp, "_device", lambda: -1)  # (tensors of the host)
    monkeypatch.setattr(torch.cuda, "caching_allocator_alloc", lambda n, dev, st: log.append(("alloc", n, dev, st)) or 4096)
    monkeypatch.setattr(torch.cuda, "caching_allocator_delete", lambda at: log.append(("delete", at)))
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(2, 32, 128, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="stop"):
        zp.zp_q4_decode_attn(desc, q, K, V, i(2, 4), i(2), torch.zeros_like(q), stream=Stream())
    assert log == [("alloc", 1000, -1, 77), ("call", (4096, 1000, 77)), ("delete", 4096)]


def test_current_device(zp, monkeypatch):
    """The device of a call is torch's current one, by its public name."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 5)
    assert zp._device() == 5


P = ctypes.c_void_p(4096)  # never dereferenced


def _read(zp, k, v, n, ts, ls, layers):
    """Status of a read into rows of 1024 bf16 elements (strides in elements, addresses in bytes); without a GPU a call
    that is not refused ends with ZP_ERR_CUDA."""
    desc = ctypes.byref(zp.cache_desc(32, 8, 128, 16, 100, torch.bfloat16))
    rc = zp.lib.zp_q4_read_kv(desc, 32, P, P, 100 * 8 * 1280, P, n, ctypes.c_void_p(k), ctypes.c_void_p(v), ts, ls, layers, None)
    return rc == 1 and b"lie on one another" in zp.lib.zp_last_error()


FAR = 1 << 40  # bytes


def _meet(k, v, n, ts, ls, layers):
    """Do any two of the rows have a byte in common?"""
    start = [x + 2 * (layer * ls + i * ts) for x in (k, v) for layer in range(layers) for i in range(n)]
    start.sort()
    return any(b - a < 2048 for a, b in zip(start, start[1:]))


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are none")
def test_read_rows_on_one_another(zp):
    """Rows of the output that share bytes are refused, whichever layers, tokens and tensors they are of; rows between
    one another are not."""
    row = 1024
    some = set()
    for n in (1, 2, 5):
        for ts in (row, row + 8, 2 * row, 3 * row, 12 * row):
            for layers in (1, 2, 4):
                for ls in (0, 8, row - 8, row, row + 8, 2 * row, 3 * row, 4 * row, n * ts - 8, n * ts, (n - 1) * ts + row, 5 * n * ts):
                    for dv in (0, 16, 2 * row - 16, 2 * row, 4 * row, 6 * row, 2 * n * ts, 2 * layers * ls, FAR, -2 * row, -2 * n * ts + 16):
                        if layers == 1 and ls:
                            continue
                        want = _meet(FAR, FAR + dv, n, ts, ls, layers)
                        assert _read(zp, FAR, FAR + dv, n, ts, ls, layers) == want, (n, ts, ls, layers, dv)
                        some.add((want, layers > 1, n > 1))
    assert len(some) == 8


def test_append_tokens(zp):
    """As every call: no more than 2^30 tokens."""
    desc = ctypes.byref(zp.cache_desc(32, 8, 128, 16, 100, torch.bfloat16))
    assert zp.lib.zp_q4_append_kv(desc, 32, P, P, P, P, P, 1, P, (1 << 30) + 1, None) == 2
