"""Plain numpy form of the 4-bit cache: quantising, the bytes of a tile, reading back."""
import numpy as np


def bf16_bits(x, up):
    """Bits (uint16) of the bf16 value next to float32 x, not below (up) or not above it."""
    u = np.asarray(x, np.float32).view(np.uint32)
    away = (u & 0xFFFF != 0) & ((u >> 31 == 0) if up else (u >> 31 == 1))
    return ((u + away.astype(np.uint32) * np.uint32(0x10000)) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits, np.uint32) << 16).astype(np.uint32).view(np.float32)


def quantise(x, group):
    """float32 rows [..., d] -> codes uint8 [..., d], words uint32 [..., d/group]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        mn, mx = g.min(-1), g.max(-1)  # (NaN where there is one)
        lo = bf16_bits(mn, False)
        flo = bf16_value(lo)
        spread = mx - flo
        step = np.maximum(bf16_value(bf16_bits(spread / np.float32(15), True)), np.float32(2.0 ** -126))
        ok = np.isfinite(flo) & np.isfinite(spread) & np.isfinite(step)
        diff = g - flo[..., None]  # 32 bits
        code = np.floor(diff.astype(np.float64) / step[..., None].astype(np.float64) + 0.5)
    code = np.where(ok[..., None], code, 0).astype(np.uint8)
    word = (step.view(np.uint32) >> 16) | (lo.astype(np.uint32) << 16)
    word = np.where(ok, word, np.uint32(0x7FC07FC0)).astype(np.uint32)
    assert code.max(initial=0) <= 15
    return code.reshape(x.shape), word


def _place(d, t, c):
    return c ^ ((t >> 1) & 3) if d == 128 else c ^ ((t >> 2) & 1)


def tile_bytes(d, group):
    return 8 * d + 64 * (d // group)


def put_row(cache, slot, head, code, word, b):
    """Write one row (codes uint8 [d], words uint32) into cache [N][h_kv][b/16][tile]."""
    d = len(code)
    tile = cache[slot // b, head, slot % b // 16]
    t = slot % 16
    byte = code[0::2] | (code[1::2] << 4)
    for c in range(d // 32):
        at = t * (d // 2) + _place(d, t, c) * 16
        tile[at:at + 16] = byte[c * 16:c * 16 + 16]
    n = 4 * len(word)
    tile[8 * d + t * n:8 * d + (t + 1) * n] = word.view(np.uint8)


def get_rows(cache, slots, d, group, b):
    """(codes [n][h_kv][d], step, lo float32 [n][h_kv][d/group]) of the rows at `slots`."""
    h_kv, slots = cache.shape[1], np.asarray(slots, np.int64)
    tiles = cache[slots // b][np.arange(len(slots)), :, slots % b // 16]   # [n][h_kv][tile]
    t = slots % 16
    n = 4 * (d // group)
    code = np.empty((len(slots), h_kv, d), np.uint8)
    word = np.empty((len(slots), h_kv, d // group), np.uint32)
    for i in range(len(slots)):
        for c in range(d // 32):
            at = t[i] * (d // 2) + _place(d, t[i], c) * 16
            byte = tiles[i, :, at:at + 16]
            code[i, :, c * 32:(c + 1) * 32:2] = byte & 15
            code[i, :, c * 32 + 1:(c + 1) * 32:2] = byte >> 4
        word[i] = np.ascontiguousarray(tiles[i, :, 8 * d + t[i] * n:8 * d + (t[i] + 1) * n]).view(np.uint32)
    return code, bf16_value(word & 0xFFFF), bf16_value(word >> 16)


def values(code, step, lo, group):
    """float64 values of rows."""
    g = code.reshape(*code.shape[:-1], -1, group).astype(np.float64)
    return (lo[..., None].astype(np.float64) + g * step[..., None].astype(np.float64)).reshape(code.shape)


def random_cache(rng, n_total, h_kv, d, group, b, poison=False):
    """A cache of quantised normal rows as bytes; poison: parameters of every row NaN instead."""
    cache = rng.integers(0, 256, size=(n_total, h_kv, b // 16, tile_bytes(d, group)), dtype=np.uint8)
    par = cache[..., 8 * d:].reshape(n_total, h_kv, b // 16, -1)
    shape = par.shape[:-1] + (par.shape[-1] // 4,)
    step = bf16_bits(rng.uniform(0.1, 0.5, size=shape), True).astype(np.uint32)
    lo = bf16_bits(rng.uniform(-3.0, -0.5, size=shape), False).astype(np.uint32)
    word = np.full(shape, 0x7FC07FC0, np.uint32) if poison else (step | lo << 16).astype(np.uint32)
    cache[..., 8 * d:] = word.view(np.uint8)
    return cache
