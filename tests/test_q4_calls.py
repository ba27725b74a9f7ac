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
