"""Workloads of the operators around a prompt shared by many requests.

Four operators of the paged cache, in the order a serving step uses them:

  slots   block tables grown and slot maps built from request lengths
  write   keys and values of many tokens (a prompt) stored into their slots
  plan    groups of sequences that share their leading blocks, from the tables
  attn    decode attention of a batch whose sequences share a prefix, computed
          once for all members, optionally with the observation-window score

``run`` computes them in plain torch operations, or with ``own`` through the
library's calls.
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
        # one decode step of the 512-sequence serving loop: every request grows by one token
        # (latency: this runs before every step)
        dict(name="slots_step_512", op="slots", B=512, old_lo=1024, old_hi=2048, grow_lo=1, grow_hi=1, b=16, pad=0),
        # 16 prompts of 32k tokens admitted at once (the long-context prefill workload)
        dict(name="slots_prefill_16x32k", op="slots", B=16, old_lo=0, old_hi=0, grow_lo=32000, grow_hi=32768, b=16,
             pad=512),
        # a small fp32 prompt batch out of a fused qkv projection (rows strided)
        dict(name="write_small_f32", op="write", tokens=509, layers=1, h_q=8, h_kv=2, d=64, b=16, dtype="f32", fused=True),
        # a full prefill step of the serving loop (16384 tokens), four layers, Qwen3-8B heads
        dict(name="write_prefill_bf16", op="write", tokens=16384, layers=4, h_q=32, h_kv=8, d=128, b=16, dtype="bf16",
             fused=False),
        # 256 sequences behind one 1k-token prompt, up to 8k tokens of their own
        dict(name="plan_256x1k", op="plan", B=256, groups=1, prefix=64, own_lo=1, own_hi=8192, b=16, lone=9),
        # a large batch with sixteen prompts of 2k-4k tokens and some requests that share nothing
        dict(name="plan_2048x16", op="plan", B=2048, groups=16, prefix=256, own_lo=1, own_hi=512, b=16, lone=100),
        # the tiny fp32 parity shape: 4 sequences, 8 q / 2 kv heads
        dict(name="attn_tiny_f32", op="attn", dtype="f32", h_q=8, h_kv=2, d=64, b=16, B=4, groups=1, prefix=4, own_lo=16,
             own_hi=86, lone=0, window=0),
        # few requests on a 2k-token system prompt, just started (latency)
        dict(name="attn_8x2k_bf16", op="attn", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, B=8, groups=1, prefix=128,
             own_lo=1, own_hi=64, lone=0, window=0),
        # the mixed prefix-shared batch, one layer: 256 sequences, 1k shared and up to 8k private tokens
        dict(name="attn_256x1k_bf16", op="attn", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, B=256, groups=1, prefix=64,
             own_lo=1, own_hi=8192, lone=0, window=0),
        # 64 questions on one 32k-token document
        dict(name="attn_64x32k_bf16", op="attn", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, B=64, groups=1, prefix=2048,
             own_lo=1, own_hi=512, lone=0, window=0),
        # sampling 256 answers to 4k-token prompts with the observation-window score for the eviction
        dict(name="attn_score_256x4k_bf16", op="attn", dtype="bf16", h_q=32, h_kv=8, d=128, b=16, B=256, groups=2,
             prefix=256, own_lo=17, own_hi=1024, lone=3, window=16),
        # small heads, large blocks, many groups of odd size, scored with a short window, fp32
        dict(name="attn_score_groups_f32", op="attn", dtype="f32", h_q=16, h_kv=4, d=64, b=32, B=61, groups=7, prefix=21,
             own_lo=33, own_hi=300, lone=5, window=8),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["slots", "write", "plan", "attn", "attn", "attn"])
    if op == "slots":
        B = _logint(rng, 1, 4096)
        most = max(1, min(32768, 500000 // B))
        if rng.random() < 0.4:
            return dict(op=op, B=B, old_lo=1, old_hi=_logint(rng, 16, 4096), grow_lo=1, grow_hi=1, b=rng.choice([16, 32]), pad=0)
        hi = _logint(rng, 1, most)
        return dict(op=op, B=B, old_lo=0, old_hi=_logint(rng, 1, 2048), grow_lo=rng.randint(0, hi), grow_hi=hi,
                    b=rng.choice([16, 32, 64]), pad=rng.choice([0, 1, 300]))
    if op == "write":
        return dict(op=op, tokens=_logint(rng, 1, 16384), layers=rng.choice([1, 2, 3, 4]), h_q=rng.choice([8, 32]),
                    h_kv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), b=rng.choice([16, 32]),
                    dtype=rng.choice(["bf16", "f32"]), fused=rng.random() < 0.5)
    if op == "plan":
        B = _logint(rng, 8, 2048)
        groups = rng.randint(1, max(1, min(24, B // 4)))
        return dict(op=op, B=B, groups=groups, prefix=_logint(rng, 1, 256), own_lo=1, own_hi=_logint(rng, 16, 4096),
                    b=rng.choice([16, 32]), lone=rng.randint(1, B // 4))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    h_kv, G = rng.choice([(8, 4), (8, 4), (4, 8), (4, 4), (2, 4), (2, 8)])
    d = rng.choice([64, 128])
    b = rng.choice([16, 16, 32])
    B = _logint(rng, 4, 256)
    groups = rng.randint(1, max(1, min(8, B // 4)))
    # tokens of a sequence, so that no drawn case has more of them in all than the largest listed one
    most = min(16384 if dtype == "bf16" else 2048, (1 << 20) // B)
    prefix = _logint(rng, 1, max(1, most // b // 2))
    own_hi = _logint(rng, 2 * b + 2, max(2 * b + 2, min(4096, most // 2)))
    window = rng.choice([0, 0, 4, b])
    return dict(op=op, dtype=dtype, h_q=h_kv * G, h_kv=h_kv, d=d, b=b, B=B, groups=groups, prefix=prefix, own_lo=b + 1 if window else 1,
                own_hi=own_hi, lone=rng.randint(0, B // 4), window=window)


# ---------------------------------------------------------------------------- inputs
def _lens(rng, case, B):
    """Private tokens of each sequence.  Scored cases put every sequence on the
    first step of its observation window, where scores are written, not added."""
    n = rng.integers(case["own_lo"], case["own_hi"] + 1, size=B)
    w, b = case.get("window", 0), case["b"]
    if w:
        n = np.maximum(n // b, 1) * b - w + 1
    return n.astype(np.int64)


def _group_sizes(case):
    """Members of each group; the last group is the largest."""
    n = case["B"] - case["lone"]
    base = n // case["groups"]
    size = [base] * case["groups"]
    size[-1] += n - base * case["groups"]
    return size


def _shared_tables(rng, case, shuffle):
    """Lengths, table [B][stride], group (or -1) and prefix blocks per sequence,
    and the number of blocks.  Group g's prompt is `prefix - g` blocks long."""
    B, b = case["B"], case["b"]
    group = np.concatenate([np.repeat(np.arange(case["groups"]), _group_sizes(case)), np.full(case["lone"], -1)])
    if shuffle:
        group = group[rng.permutation(B)]
    pre_of = np.array([max(1, case["prefix"] - g) for g in range(case["groups"])] + [0])
    pre = pre_of[group]
    lens = pre * b + _lens(rng, case, B)
    n_blocks = -(-lens // b)
    stride = case["prefix"] - (-case["own_hi"] // b) + 1
    mine = n_blocks - pre
    total = int(mine.sum() + pre_of.sum())
    ids = rng.permutation(total).astype(np.int32)
    start = np.concatenate([[0], np.cumsum(pre_of[:-1])])
    table = np.full((B, stride), -1, dtype=np.int32)
    first = int(pre_of.sum()) + np.concatenate([[0], np.cumsum(mine)[:-1]])
    for s in range(B):
        if group[s] >= 0:
            table[s, :pre[s]] = ids[start[group[s]]:start[group[s]] + pre[s]]
        table[s, pre[s]:n_blocks[s]] = ids[first[s]:first[s] + mine[s]]
    return lens, table, group, pre, total


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"slots": _prepare_slots, "write": _prepare_write, "plan": _prepare_plan, "attn": _prepare_attn}[case["op"]](
        case, rng, gen)


def _prepare_slots(case, rng, gen):
    B, b = case["B"], case["b"]
    old = rng.integers(case["old_lo"], case["old_hi"] + 1, size=B)
    new = old + rng.integers(case["grow_lo"], case["grow_hi"] + 1, size=B)
    have = -(-old // b)
    want = -(-new // b)
    ahead = (rng.random(B) < 0.125) & (want > have)  # a request may hold its next block already
    held = have + ahead
    stride = -(-(case["old_hi"] + case["grow_hi"]) // b) + 2
    total = int(np.maximum(want, held).sum())
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((B, stride), -1, dtype=np.int32)
    used = 0
    for s in range(B):
        table[s, :held[s]] = ids[used:used + held[s]]
        used += held[s]
    n_tokens = int((new - old).sum())
    room = B * case["grow_hi"] + case["pad"]  # buffers of the largest step; the rest is padding
    empty = lambda *n: torch.empty(*n, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(case=case, n_total=total, table=_dev(table), old=_dev(old), new=_dev(new), fresh=_dev(ids[used:]),
                room=room, n_tokens=n_tokens, table_out=empty(B, stride), slots=empty(room), positions=empty(room),
                cu=empty(B + 1), n_used=empty(1))


def _prepare_write(case, rng, gen):
    n, l, h_kv, d, b = case["tokens"], case["layers"], case["h_kv"], case["d"], case["b"]
    dt = DTYPES[case["dtype"]]
    n_total = -(-n // b) + 7
    K = torch.randn(l, n_total, b, h_kv, d, device=DEV, generator=gen, dtype=dt)
    V = torch.randn(l, n_total, b, h_kv, d, device=DEV, generator=gen, dtype=dt)
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
    return dict(case=case, n_total=n_total, K=K, V=V, k=k, v=v, slots=_dev(slots))


def _prepare_plan(case, rng, gen):
    lens, table, group, pre, total = _shared_tables(rng, case, True)
    B = case["B"]
    # one request in ten leaves its group's prompt somewhere before the end
    for s in np.nonzero((rng.random(B) < 0.1) & (group >= 0) & (pre > 1))[0]:
        c = int(rng.integers(1, pre[s]))
        table[s, c:pre[s]] = np.arange(total, total + pre[s] - c)
        total += int(pre[s]) - c
    empty = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(case=case, n_total=total, table=_dev(table), lens=_dev(lens), prefix_lens=empty(B), n_groups=empty(1),
                group_start=empty(B + 1), members=empty(B), group_blocks=empty(B))


def _prepare_attn(case, rng, gen):
    B, b, h_q, h_kv, d = case["B"], case["b"], case["h_q"], case["h_kv"], case["d"]
    dt = DTYPES[case["dtype"]]
    lens, table, group, pre, total = _shared_tables(rng, case, True)
    K = torch.randn(total, b, h_kv, d, device=DEV, generator=gen, dtype=dt)
    V = torch.randn(total, b, h_kv, d, device=DEV, generator=gen, dtype=dt)
    q = torch.randn(B, h_q, d, device=DEV, generator=gen, dtype=dt)
    # the groups as a scheduler that shares prompts knows them (and as the plan operator finds them)
    G = case["groups"]
    mem = [np.nonzero(group == g)[0] for g in range(G)]
    order = sorted(range(G), key=lambda g: mem[g][0])
    members = np.full(B, -1)
    start, blocks = np.zeros(B + 1), np.zeros(B)
    at = 0
    for i, g in enumerate(order):
        members[at:at + len(mem[g])] = mem[g]
        blocks[i] = pre[mem[g][0]]
        at += len(mem[g])
        start[i + 1:] = at
    state = dict(case=case, n_total=total, q=q, K=K, V=V, table=_dev(table), lens=_dev(lens), out=torch.zeros_like(q),
                 prefix_lens=_dev(pre * b), n_groups=_dev(np.array([G])), group_start=_dev(start), members=_dev(members),
                 group_blocks=_dev(blocks), max_len=int(lens.max()))
    if case["window"]:
        rows = rng.permutation(B)
        rows[rng.permutation(B)[:B // 8]] = -1  # requests without a score row
        state["rows"] = _dev(rows)
        state["S"] = torch.zeros(B, h_kv, table.shape[1] * b, device=DEV)
    return state


# ---------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"slots": _own_slots, "write": _own_write, "plan": _own_plan, "attn": _own_attn}[op](state)
    return {"slots": _plain_slots, "write": _plain_write, "plan": _plain_plan, "attn": _plain_attn}[op](state)


def _lib():
    import compressed_paged_kv_zp_gb300 as zp
    return zp


def _own_slots(st):
    zp = _lib()
    desc = zp.cache_desc(32, 8, 128, st["case"]["b"], st["n_total"], torch.bfloat16)
    zp.zp_build_slots(desc, st["table"], st["old"], st["new"], st["slots"], st["cu"], fresh=st["fresh"],
                      table_out=st["table_out"], positions=st["positions"], n_used=st["n_used"])
    return {k: st[k] for k in ("table_out", "slots", "positions", "cu", "n_used")}


def _own_write(st):
    zp = _lib()
    c = st["case"]
    desc = zp.cache_desc(c["h_q"], c["h_kv"], c["d"], c["b"], st["n_total"], DTYPES[c["dtype"]])
    zp.zp_write_kv(desc, st["k"], st["v"], st["slots"], st["K"], st["V"])
    return {"K": st["K"], "V": st["V"]}


def _own_plan(st):
    zp = _lib()
    desc = zp.cache_desc(32, 8, 128, st["case"]["b"], st["n_total"], torch.bfloat16)
    plan = zp.PrefixPlan(st["prefix_lens"], st["n_groups"], st["group_start"], st["members"], st["group_blocks"])
    zp.zp_prefix_plan(desc, st["table"], st["lens"], plan, min_blocks=1, min_members=2)
    return {k: st[k] for k in ("prefix_lens", "n_groups", "group_start", "members", "group_blocks")}


def _own_attn(st):
    zp = _lib()
    c = st["case"]
    desc = zp.cache_desc(c["h_q"], c["h_kv"], c["d"], c["b"], st["n_total"], DTYPES[c["dtype"]])
    plan = zp.PrefixPlan(st["prefix_lens"], st["n_groups"], st["group_start"], st["members"], st["group_blocks"])
    if not c["window"]:
        zp.zp_prefix_decode_attn(desc, st["q"], st["K"], st["V"], st["table"], st["lens"], plan, st["out"])
        return {"out": st["out"]}
    zp.zp_prefix_decode_attn(desc, st["q"], st["K"], st["V"], st["table"], st["lens"], plan, st["out"],
                             score_accum=st["S"], window=c["window"], score_rows=st["rows"])
    return {"out": st["out"], "S": st["S"]}


def _plain_slots(st):
    b, table, old, new = st["case"]["b"], st["table"], st["old"].long(), st["new"].long()
    B, stride = table.shape
    n = st["n_tokens"]
    col = torch.arange(stride, device=DEV)
    lo, hi = (old + b - 1) // b, (new + b - 1) // b
    need = (col >= lo[:, None]) & (col < hi[:, None]) & (table < 0)
    rank = torch.cumsum(need.reshape(-1).long(), 0).reshape(B, stride) - 1
    fresh = torch.cat([st["fresh"], st["fresh"].new_full((1,), -1)])  # one more: the list may be empty
    out = torch.where(need, fresh[rank.clamp(0, fresh.numel() - 1)], table)
    cu = torch.cat([old.new_zeros(1), torch.cumsum(new - old, 0)])
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), new - old, output_size=n)
    t = torch.arange(n, device=DEV) - cu[seq] + old[seq]
    pad = torch.full((st["room"] - n,), -1, dtype=torch.int32, device=DEV)
    slot = out[seq, t // b].long() * b + t % b
    return {"table_out": out, "slots": torch.cat([slot.int(), pad]), "positions": torch.cat([t.int(), pad]),
            "cu": cu.int(), "n_used": need.sum().int().reshape(1)}


def _plain_write(st):
    c = st["case"]
    layers, h_kv, d = c["layers"], c["h_kv"], c["d"]
    K, V = st["K"].view(layers, -1, h_kv, d), st["V"].view(layers, -1, h_kv, d)
    slots = st["slots"].long()
    n_slots = K.shape[1]
    # the token each slot takes, none (-1) for most
    src = torch.full((n_slots + 1,), -1, dtype=torch.int64, device=DEV)
    src[torch.where(slots < 0, n_slots, slots)] = torch.arange(slots.numel(), device=DEV)
    src = src[:n_slots]
    hit = (src >= 0)[None, :, None, None]
    src = src.clamp(min=0)
    K.copy_(torch.where(hit, st["k"][:, src], K))
    V.copy_(torch.where(hit, st["v"][:, src], V))
    return {"K": st["K"], "V": st["V"]}


def _plain_plan(st):
    b, table, lens = st["case"]["b"], st["table"], st["lens"].long()
    B, stride = table.shape
    idx = torch.arange(B, device=DEV)
    full = (lens - 1).clamp(min=0) // b                    # blocks before the newest token's
    first = table[:, 0]
    can = (full >= 1) & (first >= 0)
    same = (first[:, None] == first[None, :]) & can[:, None] & can[None, :]
    key = torch.where(same, (full * B + (B - 1 - idx))[None, :], -1)
    leader = key.argmax(1)
    col = torch.arange(stride, device=DEV)
    eq = (table == table[leader]) & (table >= 0) & (col < torch.minimum(full, full[leader])[:, None])
    lcp = torch.cumprod(eq.long(), 1).sum(1) * can
    count = (same & (lcp[None, :] >= lcp[:, None])).sum(1)
    gain = lcp * (count - 1) * (stride + 1) + lcp          # blocks saved, then the longer prefix
    best = torch.where(same, gain[None, :], -1).argmax(1)  # a member that gives the class its prefix
    blocks = lcp[best]
    member = can & (lcp >= blocks) & (count[best] >= 2)
    lowest = torch.where(same & member[None, :], idx[None, :], B).min(1).values
    key = torch.where(member, lowest * B + idx, B * B)
    order = torch.argsort(key)
    members = torch.where(key[order] < B * B, order, -1)
    head = member & (lowest == idx)
    n_groups = head.sum()
    heads = torch.argsort(torch.where(head, idx, B + idx))  # first members, ascending, then the rest
    live = idx < n_groups
    size = (same & member[None, :]).sum(1)[heads] * live
    start = torch.cat([size.new_zeros(1), torch.cumsum(size, 0)])
    return {"prefix_lens": (blocks * member * b).int(), "n_groups": n_groups.int().reshape(1),
            "group_start": start.int(), "members": members.int(), "group_blocks": (blocks[heads] * live).int()}


def _plain_attn(st):
    c = st["case"]
    B, b, h_kv, d = c["B"], c["b"], c["h_kv"], c["d"]
    G = c["h_q"] // h_kv
    t = torch.arange(st["max_len"], device=DEV)
    slot = st["table"].clamp(min=0)[:, t // b].long() * b + t % b
    seen = t[None, :] < st["lens"][:, None]
    k = st["K"].view(-1, h_kv, d)[slot].float().permute(0, 2, 3, 1)      # [B][h_kv][d][t]
    x = torch.matmul(st["q"].float().view(B, h_kv, G, d), k) / math.sqrt(d)
    del k
    x = torch.where(seen[:, None, None, :], x, -math.inf)
    p = torch.exp(x - x.max(-1, keepdim=True).values)
    p = p / p.sum(-1, keepdim=True)
    v = st["V"].view(-1, h_kv, d)[slot].float().permute(0, 2, 1, 3)      # [B][h_kv][t][d]
    out = torch.matmul(p, v).view(B, c["h_q"], d).to(st["q"].dtype)
    del v
    if not c["window"]:
        return {"out": out}
    new = p.max(2).values / c["window"]
    S = st["S"]
    ext = torch.cat([S, S.new_zeros(1, *S.shape[1:])])  # entries without a row score into one more
    rows = torch.where(st["rows"] < 0, S.shape[0], st["rows"]).long()
    T = st["max_len"]
    ext[rows, :, :T] = torch.where(seen[:, None, :], new, ext[rows, :, :T])
    return {"out": out, "S": ext[:S.shape[0]]}


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    mean = lambda lo, hi: (lo + hi) / 2  # noqa: E731
    if case["op"] == "slots":
        B, n = case["B"], case["B"] * mean(case["grow_lo"], case["grow_hi"])
        stride = -(-(case["old_hi"] + case["grow_hi"]) // case["b"]) + 2
        return {"bytes": 8 * B * stride + 12 * B + 4 * n / case["b"] + 8 * (B * case["grow_hi"] + case["pad"]), "flops": 0}
    if case["op"] == "write":
        es = 2 if case["dtype"] == "bf16" else 4
        rows = case["tokens"] * 60 / 61
        return {"bytes": 4 * rows * case["layers"] * case["h_kv"] * case["d"] * es + 4 * case["tokens"], "flops": 0}
    if case["op"] == "plan":
        n = case["B"] - case["lone"]
        return {"bytes": 4 * n * case["prefix"] + 4 * case["B"] * 6, "flops": 0}
    es = 2 if case["dtype"] == "bf16" else 4
    mine = mean(case["own_lo"], case["own_hi"])
    pre = [max(1, case["prefix"] - g) * case["b"] for g in range(case["groups"])]
    size = _group_sizes(case)
    tokens = case["B"] * mine + sum(pre)
    pairs = case["B"] * mine + sum(p * n for p, n in zip(pre, size))
    moved = tokens * case["h_kv"] * case["d"] * 2 * es + 2 * case["B"] * case["h_q"] * case["d"] * es
    if case["window"]:
        moved += 4 * pairs * case["h_kv"] * 7 / 8
    return {"bytes": moved, "flops": 4 * pairs * case["h_q"] * case["d"]}


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """Attention by its definition, one sequence at a time, in 64 bits, and the
    stored rows; the other operators have whole numbers only."""
    if case["op"] not in ("attn", "write"):
        return None
    st = prepare(case, seed)
    if case["op"] == "write":
        at = st["slots"].cpu().numpy()
        tok = torch.from_numpy(np.nonzero(at >= 0)[0]).to(DEV)
        blk, row = torch.from_numpy(at[at >= 0] // case["b"]).to(DEV), torch.from_numpy(at[at >= 0] % case["b"]).to(DEV)
        K, V = st["K"].double(), st["V"].double()
        for layer in range(case["layers"]):
            K[layer, blk.long(), row.long()] = st["k"][layer, tok].double()
            V[layer, blk.long(), row.long()] = st["v"][layer, tok].double()
        return {"K": K, "V": V}
    b, h_kv, d, w = case["b"], case["h_kv"], case["d"], case["window"]
    G = case["h_q"] // h_kv
    table, lens = st["table"].cpu().numpy(), st["lens"].cpu().numpy()
    K, V = st["K"], st["V"]
    out = torch.zeros(case["B"], case["h_q"], d, dtype=torch.float64, device=DEV)
    S = st["S"].double() if w else None
    rows = st["rows"].cpu().numpy() if w else None
    for s in range(case["B"]):
        L = int(lens[s])
        blocks = torch.from_numpy(table[s, :-(-L // b)].astype(np.int64)).to(DEV)
        ks = K[blocks].reshape(-1, h_kv, d)[:L].double()
        vs = V[blocks].reshape(-1, h_kv, d)[:L].double()
        for h in range(h_kv):
            logit = st["q"][s, h * G:(h + 1) * G].double() @ ks[:, h].T * d ** -0.5
            prob = torch.softmax(logit, dim=1)
            out[s, h * G:(h + 1) * G] = prob @ vs[:, h]
            if w and rows[s] >= 0:
                S[int(rows[s]), h, :L] = prob.amax(0) / w
    return {"out": out, "S": S} if w else {"out": out}
