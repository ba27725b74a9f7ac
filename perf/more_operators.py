"""Workloads of the operators of a cache held in 4 bits.

A row (one token, one kv head) is kept as d codes of 4 bits and, per group of 32, 64
or 128 elements, a step and a lowest value in bf16: element = lo + code * step.  Sixteen
rows form a tile: their codes (d/2 bytes a row, element e in nibble e, the 16-byte
chunks of a row exchanged among themselves), then their (step, lo) words.  A cache is
[N_total][h_kv][b/16][tile bytes].

  append  one new token per sequence quantised into its slot, and read back
  write   the rows of many tokens quantised into their slots, and the cache read back
  read    rows of a list of slots as bf16 or fp32
  attn    decode attention over such a cache, optionally with the window score
  compact kept rows moved into target blocks with their global score, and read back

``run`` computes them in plain torch operations, or with ``own`` through the library's
calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of the 512-sequence serving loop, one layer (latency: it runs before every decode)
        dict(name="append_512_bf16", op="append", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, group=32, B=512, len_lo=1024,
             len_hi=4096),
        # a small fp32 prompt batch out of a fused qkv projection (rows strided)
        dict(name="write_small_f32", op="write", dtype="f32", h_q=8, h_kv=2, d=64, b=16, group=32, tokens=509, layers=1,
             fused=True),
        # a full prefill step of the serving loop (16384 tokens), four layers, Qwen3-8B heads
        dict(name="write_prefill_bf16", op="write", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, group=32, tokens=16384,
             layers=4, fused=False),
        # one 32k-token prompt taken back for a further prefill over it
        dict(name="read_32k_bf16", op="read", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, group=32, B=1, len_lo=32768,
             len_hi=32768, layers=1),
        # a ragged fp32 batch of small heads in larger blocks, one parameter pair per row
        dict(name="read_ragged_f32", op="read", dtype="f32", h_q=16, h_kv=4, d=64, b=32, group=64, B=61, len_lo=1, len_hi=777,
             layers=2),
        # the tiny fp32 parity shape: 4 sequences, 8 q / 2 kv heads
        dict(name="attn_tiny_f32", op="attn", dtype="f32", h_q=8, h_kv=2, d=64, b=16, group=32, B=4, len_lo=16, len_hi=150,
             window=0),
        # one request on a 32k-token context (latency)
        dict(name="attn_1x32k_bf16", op="attn", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, group=32, B=1, len_lo=32768,
             len_hi=32768, window=0),
        # the 64-sequence Qwen3-8B layer with contexts of 1k-4k
        dict(name="attn_64x4k_bf16", op="attn", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, group=32, B=64, len_lo=1024,
             len_hi=4096, window=0),
        # 256 sequences up to 4k with the observation-window score for the eviction
        dict(name="attn_score_256x4k_bf16", op="attn", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, group=32, B=256, len_lo=17,
             len_hi=4096, window=16),
        # small heads, large blocks, eight q heads per kv head, scored with a short window, fp32
        dict(name="attn_score_61_f32", op="attn", dtype="f32", h_q=32, h_kv=4, d=64, b=32, group=64, B=61, len_lo=33,
             len_hi=900, window=8),
        # the compressions of one step of the 64-sequence layer: 7 sequences of 2k tokens keep all but one block
        dict(name="compact_7x2k_bf16", op="compact", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, group=32, n=7, L=2048,
             keep=2032, layers=1),
        # sixteen 32k-token prompts cut to 4k tokens
        dict(name="compact_16x32k_bf16", op="compact", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, group=32, n=16, L=32768,
             keep=4080, layers=1),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "write", "read", "attn", "attn", "attn", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    group = rng.choice([32, 32, 64, d])
    h_kv, G = rng.choice([(8, 4), (8, 4), (4, 8), (4, 4), (2, 4), (1, 8), (8, 1), (4, 2), (3, 5)])
    base = dict(op=op, dtype=dtype, h_q=h_kv * G, h_kv=h_kv, d=d, b=rng.choice([16, 16, 32, 64]), group=group)
    if op == "append":
        return dict(base, B=_logint(rng, 1, 1024), len_lo=1, len_hi=_logint(rng, 16, 1024))
    if op == "write":
        return dict(base, tokens=_logint(rng, 1, 16384), layers=rng.choice([1, 2, 3]), fused=rng.random() < 0.5)
    if op == "read":
        B = _logint(rng, 1, 64)
        return dict(base, B=B, len_lo=1, len_hi=_logint(rng, 1, 32768 // B), layers=rng.choice([1, 2]))
    if op == "compact":
        n = _logint(rng, 1, 16)
        L = _logint(rng, 80, 8192)
        return dict(base, n=n, L=L, keep=_logint(rng, 16, L), layers=rng.choice([1, 2]))
    B = _logint(rng, 1, 256)
    most = min(32768 if dtype == "bf16" else 4096, (1 << 20) // B)
    window = rng.choice([0, 0, 4, base["b"]])
    hi = _logint(rng, base["b"] + 1, max(base["b"] + 2, most))
    return dict(base, B=B, len_lo=base["b"] if window else 1, len_hi=hi, window=window)


# ---------------------------------------------------------------------------- the format
def _quantise(x, group):
    """Codes and (step, lo) of rows x [..., d]: float32 [..., d/group, group] and [..., d/group, 1]."""
    x = x.float().unflatten(-1, (-1, group))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    lo = _bf16_below(lo)
    step = -_bf16_below(-((hi - lo) / hi.new_full((), 15.0)))  # (by a host number torch multiplies by 1/15)
    step = step.clamp(min=2.0 ** -126)
    code = torch.floor((x - lo).double() / step.double() + 0.5).float()
    return code, step, lo


def _bf16_below(x):
    """The largest bf16 value that is not above x, in float32."""
    y = x.to(torch.bfloat16)
    down = torch.nextafter(y, torch.full_like(y, -math.inf))
    return torch.where(y.float() > x, down, y).float()


def _chunks(d):
    """[16][d/32]: where the 16-byte chunks of the 16 rows of a tile lie."""
    t, c = np.arange(16)[:, None], np.arange(d // 32)[None, :]
    return torch.from_numpy(c ^ ((t >> 1) & 3 if d == 128 else (t >> 2) & 1)).to(DEV)


def _pack(x, group):
    """Tiles of rows x [..., 16, d] as bytes [..., tile]."""
    d = x.shape[-1]
    code, step, lo = _quantise(x, group)
    code = code.flatten(-2).to(torch.uint8)
    byte = (code[..., 0::2] | (code[..., 1::2] << 4)).unflatten(-1, (d // 32, 16))
    at = _chunks(d)[..., None].expand(byte.shape)
    byte = torch.empty_like(byte).scatter_(-2, at, byte)
    par = torch.stack([step.squeeze(-1), lo.squeeze(-1)], -1).to(torch.bfloat16).contiguous()
    return torch.cat([byte.flatten(-3), par.view(torch.uint8).flatten(-3)], -1)


def _tile_bytes(d, group):
    return 8 * d + 64 * (d // group)


def _make_cache(case, n_total, gen, layers=None):
    """A cache of rows as a model writes them: normal values, some channels of the keys far larger."""
    h_kv, d, b, group = case["h_kv"], case["d"], case["b"], case["group"]
    shape = (n_total, h_kv, b // 16, _tile_bytes(d, group))
    out = []
    for key in (True, False):
        cache = torch.empty((layers or 1,) + shape, dtype=torch.uint8, device=DEV)
        channel = torch.ones(h_kv, 1, 1, d, device=DEV)
        if key:
            channel[..., ::17] = 3.0
        per = max(1, (1 << 26) // (h_kv * b * d))
        for layer in range(layers or 1):
            for n0 in range(0, n_total, per):
                n = min(per, n_total - n0)
                x = torch.randn(n, h_kv, b // 16, 16, d, device=DEV, generator=gen) * channel
                cache[layer, n0:n0 + n] = _pack(x, group)
        out.append(cache if layers else cache[0])
    return out


def _rows(cache, slots, case):
    """Values [n][h_kv][d] (float32) of the rows at `slots` of one layer."""
    h_kv, d, b, group = case["h_kv"], case["d"], case["b"], case["group"]
    tiles = cache.view(-1, h_kv, b // 16, cache.shape[-1])
    codes = tiles[..., :8 * d].unflatten(-1, (16, d // 32, 16))
    pars = tiles[..., 8 * d:].unflatten(-1, (16, d // group, 4))
    slots = slots.long()
    blk, sub, t = slots // b, slots % b // 16, slots % 16
    byte = codes[blk, :, sub, t]                                           # [n][h_kv][chunk][16]
    byte = torch.gather(byte, 2, _chunks(d)[t][:, None, :, None].expand(byte.shape)).flatten(2)
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(2).float()
    par = pars[blk, :, sub, t].contiguous().view(torch.bfloat16).float()   # [n][h_kv][groups][2]
    return (code.unflatten(-1, (-1, group)) * par[..., :1] + par[..., 1:]).flatten(-2)


# ---------------------------------------------------------------------------- inputs
def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def _tables(rng, lens, b, longest, extra=0):
    """Block table of sequences of up to `longest` tokens in scattered blocks, and the number of blocks."""
    n_blocks = -(-lens // b)
    total = int(n_blocks.sum()) + extra
    ids = rng.permutation(total)
    table = np.full((len(lens), -(-longest // b) + 1), -1, dtype=np.int64)
    at = 0
    for s, n in enumerate(n_blocks):
        table[s, :n] = ids[at:at + n]
        at += n
    return table, total, ids[at:]


def _slots(table, lens, b):
    """Slots of every token, sequence after sequence."""
    return np.concatenate([table[s, np.arange(n) // b] * b + np.arange(n) % b for s, n in enumerate(lens)])


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"append": _prepare_append, "write": _prepare_write, "read": _prepare_read, "attn": _prepare_attn,
            "compact": _prepare_compact}[case["op"]](case, rng, gen)


def _prepare_append(case, rng, gen):
    B, b, h_kv, d = case["B"], case["b"], case["h_kv"], case["d"]
    dt = DTYPES[case["dtype"]]
    lens = rng.integers(case["len_lo"], case["len_hi"] + 1, size=B)
    table, total, _ = _tables(rng, lens, b, case["len_hi"])
    K, V = _make_cache(case, total, gen)
    k = torch.randn(B, h_kv, d, device=DEV, generator=gen, dtype=dt)
    v = torch.randn(B, h_kv, d, device=DEV, generator=gen, dtype=dt)
    # read back: the new token of each sequence and the one before it (its neighbour in the tile)
    i = np.arange(B)
    new = table[i, (lens - 1) // b] * b + (lens - 1) % b
    old = np.maximum(lens - 2, 0)
    slots = np.concatenate([new, table[i, old // b] * b + old % b])
    empty = lambda: torch.zeros(2 * B, h_kv, d, device=DEV, dtype=dt)  # noqa: E731
    return dict(case=case, n_total=total, K=K, V=V, k=k, v=v, table=_dev(table), lens=_dev(lens), new=_dev(new),
                slots=_dev(slots), k_out=empty(), v_out=empty())


def _prepare_write(case, rng, gen):
    n, l, h_kv, d, b = case["tokens"], case["layers"], case["h_kv"], case["d"], case["b"]
    dt = DTYPES[case["dtype"]]
    n_total = -(-n // b) + 7
    K, V = _make_cache(case, n_total, gen, l)
    # whole prompts in scattered blocks; every 61st token is padding (slot -1)
    block = rng.permutation(n_total)[:-(-n // b)]
    i = np.arange(n)
    slots = block[i // b] * b + i % b
    slots[i % 61 == 60] = -1
    if case["fused"]:  # k and v as they lie in the rows of a q, k, v projection
        h_q = case["h_q"]
        qkv = torch.randn(l, n, h_q + 2 * h_kv, d, device=DEV, generator=gen, dtype=dt)
        k, v = qkv[:, :, h_q:h_q + h_kv], qkv[:, :, h_q + h_kv:]
    else:
        k = torch.randn(l, n, h_kv, d, device=DEV, generator=gen, dtype=dt)
        v = torch.randn(l, n, h_kv, d, device=DEV, generator=gen, dtype=dt)
    empty = lambda: torch.zeros(l, n_total * b, h_kv, d, device=DEV, dtype=dt)  # noqa: E731
    return dict(case=case, n_total=n_total, K=K, V=V, k=k, v=v, new=_dev(slots), slots=_dev(np.arange(n_total * b)),
                k_out=empty(), v_out=empty())


def _prepare_read(case, rng, gen):
    B, b, h_kv, d, l = case["B"], case["b"], case["h_kv"], case["d"], case["layers"]
    lens = rng.permutation(np.linspace(case["len_lo"], case["len_hi"], B).astype(np.int64))
    table, total, _ = _tables(rng, lens, b, case["len_hi"], 3)
    K, V = _make_cache(case, total, gen, l)
    slots = _slots(table, lens, b)
    slots = np.concatenate([slots, np.full(5, -1)])  # padding behind the last token: rows left as they are
    empty = lambda: torch.zeros(l, len(slots), h_kv, d, device=DEV, dtype=DTYPES[case["dtype"]])  # noqa: E731
    return dict(case=case, n_total=total, K=K, V=V, slots=_dev(slots), k_out=empty(), v_out=empty())


def _prepare_attn(case, rng, gen):
    B, b, h_q, h_kv, d, w = case["B"], case["b"], case["h_q"], case["h_kv"], case["d"], case["window"]
    lens = rng.integers(case["len_lo"], case["len_hi"] + 1, size=B)
    if w:  # every sequence on the first step of its window, where scores are written, not added
        lens = np.maximum(lens // b, 1) * b - w + 1
    table, total, _ = _tables(rng, lens, b, case["len_hi"])
    K, V = _make_cache(case, total, gen)
    q = torch.randn(B, h_q, d, device=DEV, generator=gen, dtype=DTYPES[case["dtype"]])
    state = dict(case=case, n_total=total, q=q, K=K, V=V, table=_dev(table), lens=_dev(lens), out=torch.zeros_like(q),
                 max_len=int(lens.max()))
    if w:
        rows = rng.permutation(B)
        rows[rng.permutation(B)[:B // 8]] = -1  # requests without a score row
        state["rows"] = _dev(rows)
        state["S"] = torch.zeros(B, h_kv, table.shape[1] * b, device=DEV)
    return state


def _prepare_compact(case, rng, gen):
    n, L, k, l, b, h_kv, d = case["n"], case["L"], case["keep"], case["layers"], case["b"], case["h_kv"], case["d"]
    lens = np.full(n, L)
    lens[1::3] -= rng.integers(0, min(b, L - k + 1), size=len(lens[1::3]))
    targets = -(-k // b)
    # targets of their own, as behind a shared prompt; as many blocks in all whatever the lengths drawn
    table, total, fresh = _tables(rng, lens, b, L, n * (targets + -(-L // b)) - int((-(-lens // b)).sum()))
    K, V = _make_cache(case, total, gen, l)
    dst = fresh[:n * targets].reshape(n, targets)
    # keep sets: k of the L positions, ascending
    score = torch.rand(l, n, h_kv, L, device=DEV, generator=gen)
    score = torch.where(torch.arange(L, device=DEV) < _dev(lens)[:, None, None], score, -1.0)
    keep = score.topk(k, dim=-1).indices.sort(-1).values.int().contiguous()
    S = torch.rand(l, n, h_kv, L, device=DEV, generator=gen)
    F = torch.zeros(l, total, b, h_kv, device=DEV)
    slots = dst[:, np.arange(k) // b] * b + np.arange(k) % b
    empty = lambda: torch.zeros(l, n * k, h_kv, d, device=DEV, dtype=DTYPES[case["dtype"]])  # noqa: E731
    return dict(case=case, n_total=total, K=K, V=V, table=_dev(table), lens=_dev(lens), dst=_dev(dst), keep=keep, S=S, F=F,
                slots=_dev(slots.reshape(-1)), k_out=empty(), v_out=empty())


# ---------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "write": _own_write, "read": _own_read, "attn": _own_attn,
                "compact": _own_compact}[op](state)
    return {"append": _plain_append, "write": _plain_write, "read": _plain_read, "attn": _plain_attn,
            "compact": _plain_compact}[op](state)


def _lib(st):
    import compressed_paged_kv_zp_gb300 as zp
    c = st["case"]
    return zp, zp.cache_desc(c["h_q"], c["h_kv"], c["d"], c["b"], st["n_total"], DTYPES[c["dtype"]]), c["group"]


def _own_append(st):
    zp, desc, group = _lib(st)
    zp.zp_q4_append_kv(desc, st["k"], st["v"], st["K"], st["V"], st["table"], st["lens"], group=group)
    zp.zp_q4_read_kv(desc, st["K"], st["V"], st["slots"], st["k_out"], st["v_out"], group=group)
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_write(st):
    zp, desc, group = _lib(st)
    zp.zp_q4_write_kv(desc, st["k"], st["v"], st["new"], st["K"], st["V"], group=group)
    zp.zp_q4_read_kv(desc, st["K"], st["V"], st["slots"], st["k_out"], st["v_out"], group=group)
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_read(st):
    zp, desc, group = _lib(st)
    zp.zp_q4_read_kv(desc, st["K"], st["V"], st["slots"], st["k_out"], st["v_out"], group=group)
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_attn(st):
    zp, desc, group = _lib(st)
    w = st["case"]["window"]
    if not w:
        zp.zp_q4_decode_attn(desc, st["q"], st["K"], st["V"], st["table"], st["lens"], st["out"], group=group)
        return {"out": st["out"]}
    zp.zp_q4_decode_attn(desc, st["q"], st["K"], st["V"], st["table"], st["lens"], st["out"], group=group,
                         score_accum=st["S"], window=w, score_rows=st["rows"])
    return {"out": st["out"], "S": st["S"]}


def _own_compact(st):
    zp, desc, group = _lib(st)
    zp.zp_q4_compact_pages(desc, st["K"], st["V"], st["table"], st["dst"], st["lens"], st["keep"], global_F=st["F"],
                           scores=st["S"], group=group)
    zp.zp_q4_read_kv(desc, st["K"], st["V"], st["slots"], st["k_out"], st["v_out"], group=group)
    return {"k": st["k_out"], "v": st["v_out"], "F": st["F"]}


def _stored(x, group):
    """The values that rows x [..., d] are kept as."""
    code, step, lo = _quantise(x, group)
    return (code * step + lo).flatten(-2)


def _plain_append(st):
    c = st["case"]
    out = {}
    for name, cache, x in (("k", st["K"], st["k"]), ("v", st["V"], st["v"])):
        got = _rows(cache, st["slots"], c)
        B = x.shape[0]
        new = _stored(x, c["group"])
        same = (st["lens"] == 1)[:, None, None]  # a sequence of one token: its neighbour is itself
        got = torch.cat([new, torch.where(same, new, got[B:])])
        out[name] = got.to(x.dtype)
    return out


def _plain_write(st):
    c = st["case"]
    new = st["new"].long()
    n_slots = st["slots"].numel()
    src = torch.full((n_slots + 1,), -1, dtype=torch.int64, device=DEV)  # the token each slot takes, none (-1) for some
    src[torch.where(new < 0, n_slots, new)] = torch.arange(new.numel(), device=DEV)
    src = src[:n_slots]
    hit = (src >= 0)[:, None, None]
    src = src.clamp(min=0)
    out = {}
    for name, cache, x in (("k", st["K"], st["k"]), ("v", st["V"], st["v"])):
        out[name] = torch.stack([torch.where(hit, _stored(x[i], c["group"])[src], _rows(cache[i], st["slots"], c)).to(x.dtype)
                                 for i in range(c["layers"])])
    return out


def _plain_read(st):
    c = st["case"]
    out = {}
    live = (st["slots"] >= 0)[:, None, None]
    for name, cache in (("k", st["K"]), ("v", st["V"])):
        out[name] = torch.stack([torch.where(live, _rows(layer, st["slots"].clamp(min=0), c), 0.0).to(st["k_out"].dtype)
                                 for layer in cache])
    return out


def _plain_attn(st):
    c = st["case"]
    B, b, h_kv, d = c["B"], c["b"], c["h_kv"], c["d"]
    G, T = c["h_q"] // h_kv, st["max_len"]
    t = torch.arange(T, device=DEV)
    slot = (st["table"].clamp(min=0)[:, t // b].long() * b + t % b).flatten()
    seen = t[None, :] < st["lens"][:, None]
    k = _rows(st["K"], slot, c).view(B, T, h_kv, d).permute(0, 2, 3, 1)     # [B][h_kv][d][t]
    x = torch.matmul(st["q"].float().view(B, h_kv, G, d), k) / math.sqrt(d)
    del k
    x = torch.where(seen[:, None, None, :], x, -math.inf)
    p = torch.exp(x - x.max(-1, keepdim=True).values)
    p = p / p.sum(-1, keepdim=True)
    v = _rows(st["V"], slot, c).view(B, T, h_kv, d).permute(0, 2, 1, 3)     # [B][h_kv][t][d]
    out = torch.matmul(p, v).view(B, c["h_q"], d).to(st["q"].dtype)
    del v
    if not c["window"]:
        return {"out": out}
    new = p.max(2).values / c["window"]
    S = st["S"]
    ext = torch.cat([S, S.new_zeros(1, *S.shape[1:])])  # entries without a row score into one more
    rows = torch.where(st["rows"] < 0, S.shape[0], st["rows"]).long()
    ext[rows, :, :T] = torch.where(seen[:, None, :], new, ext[rows, :, :T])
    return {"out": out, "S": ext[:S.shape[0]]}


def _plain_compact(st):
    c = st["case"]
    n, k, l, b, h_kv = c["n"], c["keep"], c["layers"], c["b"], c["h_kv"]
    out = {"k": [], "v": []}
    F = torch.zeros_like(st["F"])
    for layer in range(l):
        keep = st["keep"][layer].long()                                     # [n][h_kv][k]
        slot = torch.gather(st["table"].long()[:, None].expand(n, h_kv, -1), 2, keep // b) * b + keep % b
        head = torch.arange(h_kv, device=DEV)[None, :, None].expand(slot.shape)
        for name, cache in (("k", st["K"][layer]), ("v", st["V"][layer])):
            got = _rows_of_head(cache, slot.reshape(-1), head.reshape(-1), c).view(n, h_kv, k, -1)
            out[name].append(got.transpose(1, 2).reshape(n * k, h_kv, -1).to(st["k_out"].dtype))
        score = torch.gather(st["S"][layer], 2, keep).transpose(1, 2).reshape(n * k, h_kv)
        F[layer].view(-1, h_kv)[st["slots"].long()] = score
    return {"k": torch.stack(out["k"]), "v": torch.stack(out["v"]), "F": F}


def _rows_of_head(cache, slots, heads, case):
    """Values [n][d] (float32) of the rows at (slot, kv head) pairs of one layer."""
    h_kv, d, b, group = case["h_kv"], case["d"], case["b"], case["group"]
    tiles = cache.view(-1, h_kv, b // 16, cache.shape[-1])
    codes = tiles[..., :8 * d].unflatten(-1, (16, d // 32, 16))
    pars = tiles[..., 8 * d:].unflatten(-1, (16, d // group, 4))
    blk, sub, t = slots // b, slots % b // 16, slots % 16
    byte = codes[blk, heads, sub, t]
    byte = torch.gather(byte, 1, _chunks(d)[t][:, :, None].expand(byte.shape)).flatten(1)
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(1).float()
    par = pars[blk, heads, sub, t].contiguous().view(torch.bfloat16).float()
    return (code.unflatten(-1, (-1, group)) * par[..., :1] + par[..., 1:]).flatten(-2)


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    h_kv, d = case["h_kv"], case["d"]
    row = d // 2 + 4 * (d // case["group"])   # bytes of a row in 4 bits
    full = d * es                             # and as it is given or taken back
    mean = lambda: (case["len_lo"] + case["len_hi"]) / 2  # noqa: E731
    if case["op"] == "append":
        # rows in, rows kept; the new and the previous row read and given back
        return {"bytes": 2 * h_kv * case["B"] * (full + row + 2 * (row + full)) + 20 * case["B"], "flops": 0}
    if case["op"] == "write":
        n, slots = case["tokens"] * 60 / 61, (-(-case["tokens"] // case["b"]) + 7) * case["b"]
        return {"bytes": 2 * h_kv * case["layers"] * (n * (full + row) + slots * (row + full)) + 4 * (case["tokens"] + slots),
                "flops": 0}
    if case["op"] == "read":
        n = case["B"] * mean()
        return {"bytes": 2 * h_kv * case["layers"] * n * (row + full) + 4 * n, "flops": 0}
    if case["op"] == "compact":
        n = case["n"] * case["keep"]
        return {"bytes": case["layers"] * h_kv * n * (2 * (3 * row + full) + 12), "flops": 0}
    tokens = case["B"] * mean()
    moved = tokens * h_kv * 2 * row + 2 * case["B"] * case["h_q"] * d * es
    if case["window"]:
        moved += 4 * tokens * h_kv * 7 / 8
    return {"bytes": moved, "flops": 4 * tokens * case["h_q"] * d}


# ---------------------------------------------------------------------------- 64 bits
def _values(cache, slots, case):
    """Rows [n][h_kv][d] at `slots`, from the bytes, in 64 bits."""
    h_kv, d, b, group = case["h_kv"], case["d"], case["b"], case["group"]
    flat = cache.reshape(-1)
    tile = cache.shape[-1]
    s = slots.long()[:, None, None]
    head = torch.arange(h_kv, device=DEV)[None, :, None]
    e = torch.arange(d, device=DEV)[None, None, :]
    base = ((s // b * h_kv + head) * (b // 16) + s % b // 16) * tile
    t = s % 16
    swap = (t // 2) % 4 if d == 128 else t // 4 % 2
    byte = flat[base + t * (d // 2) + (torch.bitwise_xor(e // 32, swap)) * 16 + e % 32 // 2].long()
    code = torch.where(e % 2 == 0, byte % 16, byte // 16).double()
    g = torch.arange(d // group, device=DEV)[None, None, :]
    at = base + 8 * d + (t * (d // group) + g) * 4
    half = lambda o: ((flat[at + o].int() + 256 * flat[at + o + 1].int()) * 65536).view(torch.float32).double()  # noqa: E731
    step, lo = half(0).repeat_interleave(group, 2), half(2).repeat_interleave(group, 2)
    return lo + code * step


def _kept(x, group):
    """What rows x [n][h_kv][d] are kept as, by the definition: lo the bf16 value at or below the
    smallest, the step the bf16 value at or above a fifteenth of the spread (both of 32-bit numbers)."""
    x = x.float()
    g = x.reshape(*x.shape[:-1], -1, group)
    lo, hi = g.min(-1).values, g.max(-1).values

    def cut(v, up):  # to 16 bits, away from zero or not, by the bit pattern
        bits = v.contiguous().view(torch.int32)
        trunc = bits & -65536
        away = (bits != trunc) & ((v > 0) if up else (v < 0))
        return (trunc + away * 65536).int().view(torch.float32)

    lo = cut(lo, False)
    step = torch.maximum(cut((hi - lo) / hi.new_full((), 15.0), True), hi.new_full((), 2.0 ** -126))
    code = torch.floor((g - lo[..., None]).double() / step[..., None].double() + 0.5)
    return (lo[..., None].double() + code * step[..., None].double()).reshape(x.shape)


def exact(case, seed):
    """The operators by their definition, in 64 bits."""
    st = prepare(case, seed)
    op, b, h_kv, d = case["op"], case["b"], case["h_kv"], case["d"]
    if op == "append":
        out = {}
        for name, cache, x in (("k", st["K"], st["k"]), ("v", st["V"], st["v"])):
            got, new = _values(cache, st["slots"], case), _kept(x, case["group"])
            B = case["B"]
            got[:B] = new
            one = (st["lens"] == 1).nonzero().flatten()
            got[B + one] = new[one]
            out[name] = got
        return out
    if op == "write":
        at = st["new"].cpu().numpy()
        tok = torch.from_numpy(np.nonzero(at >= 0)[0]).to(DEV)
        to = torch.from_numpy(at[at >= 0]).to(DEV).long()
        out = {"k": [], "v": []}
        for i in range(case["layers"]):
            for name, cache, x in (("k", st["K"], st["k"]), ("v", st["V"], st["v"])):
                got = torch.cat([_values(cache[i], s, case) for s in st["slots"].split(8192)])
                got[to] = _kept(x[i, tok], case["group"])
                out[name].append(got)
        return {name: torch.stack(x) for name, x in out.items()}
    if op == "read":
        n = int((st["slots"] >= 0).sum())
        out = {}
        for name, cache in (("k", st["K"]), ("v", st["V"])):
            res = torch.zeros(st["k_out"].shape, dtype=torch.float64, device=DEV)
            for i in range(case["layers"]):
                res[i, :n] = torch.cat([_values(cache[i], s, case) for s in st["slots"][:n].split(8192)])
            out[name] = res
        return out
    table, lens = st["table"].cpu().numpy(), st["lens"].cpu().numpy()
    seq = lambda s: torch.from_numpy(table[s, np.arange(lens[s]) // b] * b + np.arange(lens[s]) % b).to(DEV)  # noqa: E731
    if op == "compact":
        out = {"k": [], "v": []}
        F = torch.zeros(st["F"].shape, dtype=torch.float64, device=DEV)
        k, dst = case["keep"], st["slots"].long().view(case["n"], -1)
        for i in range(case["layers"]):
            rows = {"k": [], "v": []}
            for s in range(case["n"]):
                keep = st["keep"][i, s].long()                              # [h_kv][k]
                for name, cache in (("k", st["K"]), ("v", st["V"])):
                    x = torch.cat([_values(cache[i], part, case) for part in seq(s).split(8192)])
                    rows[name].append(torch.stack([x[keep[h], h] for h in range(h_kv)], 1))
                F[i, dst[s] // b, dst[s] % b] = torch.gather(st["S"][i, s].double(), 1, keep).T
            for name in out:
                out[name].append(torch.cat(rows[name]))
        return {"k": torch.stack(out["k"]), "v": torch.stack(out["v"]), "F": F}
    w, G = case["window"], case["h_q"] // h_kv
    out = torch.zeros(case["B"], case["h_q"], d, dtype=torch.float64, device=DEV)
    S = st["S"].double() if w else None
    rows = st["rows"].cpu().numpy() if w else None
    for s in range(case["B"]):
        at = seq(s)
        ks, vs = _values(st["K"], at, case), _values(st["V"], at, case)
        for h in range(h_kv):
            logit = st["q"][s, h * G:(h + 1) * G].double() @ ks[:, h].T * d ** -0.5
            prob = torch.softmax(logit, dim=1)
            out[s, h * G:(h + 1) * G] = prob @ vs[:, h]
            if w and rows[s] >= 0:
                S[int(rows[s]), h, :len(at)] = prob.amax(0) / w
    return {"out": out, "S": S} if w else {"out": out}
