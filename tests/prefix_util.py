"""Cases and references of the shared-prompt operators' tests (plain numpy, 64 bits)."""
import numpy as np

import oracle


def make_groups(seed, sizes, prefix_blocks, own, b, lone=0, zero=0, shuffle=True, spare=0):
    """Batch of groups: group g has sizes[g] sequences sharing prefix_blocks[g]
    blocks, each with own[...] private tokens (drawn from the range own =
    (lo, hi)); `lone` sequences share nothing and `zero` entries have L = 0.
    Returns lens, table (int32, -1 unused), group of each entry (-1), n_total."""
    rng = np.random.default_rng(seed)
    group = np.concatenate([np.repeat(np.arange(len(sizes)), sizes), np.full(lone, -1), np.full(zero, -2)]).astype(int)
    if shuffle:
        group = group[rng.permutation(len(group))]
    B = len(group)
    pre = np.array([prefix_blocks[g] if g >= 0 else 0 for g in group])
    lens = pre * b + rng.integers(own[0], own[1] + 1, size=B)
    lens[group == -2] = 0
    pre[group == -2] = 0
    nb = -(-lens // b)
    stride = max(int(nb.max()), 1) + 1
    total = int(sum(prefix_blocks)) + int((nb - pre).sum()) + spare
    ids = rng.permutation(total).astype(np.int32)
    at, heads = 0, []
    for p in prefix_blocks:
        heads.append(ids[at:at + p])
        at += p
    table = np.full((B, stride), -1, np.int32)
    for s in range(B):
        if pre[s]:
            table[s, :pre[s]] = heads[group[s]]
        n = nb[s] - pre[s]
        table[s, pre[s]:nb[s]] = ids[at:at + n]
        at += n
    return lens.astype(np.int32), table, group, total


def plan_ref(table, lens, b, n_total, min_blocks, min_members):
    """The grouping rule, entry by entry."""
    B, stride = table.shape
    full = [min((int(L) - 1) // b, stride) if L > 0 else 0 for L in lens]
    classes = {}
    for s in range(B):
        f = int(table[s, 0])
        if full[s] >= 1 and 0 <= f < n_total:
            classes.setdefault(f, []).append(s)
    prefix_lens = np.zeros(B, np.int32)
    groups = []
    for mem in classes.values():
        leader = max(mem, key=lambda s: (full[s], -s))
        lcp = {}
        for s in mem:
            n = 0
            while n < min(full[s], full[leader]) and table[s, n] == table[leader, n] and 0 <= table[s, n] < n_total:
                n += 1
            lcp[s] = n
        p = max(set(lcp.values()), key=lambda c: (c * (sum(v >= c for v in lcp.values()) - 1), c))
        got = [s for s in mem if lcp[s] >= p]
        if p >= min_blocks and len(got) >= min_members:
            groups.append((got, p))
            prefix_lens[got] = p * b
    groups.sort(key=lambda g: g[0][0])
    start = np.zeros(B + 1, np.int32)
    members = np.full(B, -1, np.int32)
    blocks = np.zeros(B, np.int32)
    at = 0
    for i, (got, p) in enumerate(groups):
        members[at:at + len(got)] = got
        blocks[i] = p
        at += len(got)
        start[i + 1:] = at
    return dict(prefix_lens=prefix_lens, n_groups=np.array([len(groups)], np.int32), group_start=start, members=members,
                group_blocks=blocks)


def attention_bounds(q, K, V, table, lens, bf16):
    """Output and probabilities in 64 bits, and the bounds of an fp32-accumulating kernel.

    Logits: a dot product of d terms is off by at most (d + 4) 2^-24 X, X = sum |q_i k_i| / sqrt(d)
    (twice that where the tensor cores truncate instead of rounding); a probability is then off by
    twice that relative (its own logit and the sum's), plus n 2^-24 for the sum of n terms and a few
    steps for the exponential (2^-21).  The output adds the same for the sum over v.  bf16: the
    probabilities are rounded to bf16 for the second product (half a step, 2^-8, of sum p |v|) and
    the output too (2^-8 of itself)."""
    out, probs = oracle.decode_attention(q, K, V, table, lens, want_probs=True)
    absv = oracle.decode_attention(q, K, np.abs(V), table, lens)
    d, n = q.shape[-1], max(int(np.max(lens)), 1)
    X = 0.0
    b, h_kv = K.shape[1], K.shape[2]
    G = q.shape[1] // h_kv
    for s in range(len(lens)):
        L = int(lens[s])
        if L == 0:
            continue
        t = np.arange(L)
        k = np.abs(K[table[s, t // b], t % b])
        X = max(X, float(np.einsum("hgd,thd->hgt", np.abs(q[s]).reshape(h_kv, G, d), k).max()) / np.sqrt(d))
    rel = 2.0 ** -24 * (4 * (d + 4) * X + 2 * n) + 2.0 ** -21
    tol = rel * absv + 1e-30
    if bf16:
        tol = tol + 2.0 ** -8 * (1 + rel) * (absv + np.abs(out) * 1.01)
    return out, tol, probs, rel


def window_ref(probs, lens, prefix_of, S, rows, h_kv, b, w):
    """Score rows S [R][h_kv][stride*b] (64 bits, updated) after one decode step."""
    G = probs.shape[1] // h_kv
    for s, L in enumerate(lens):
        L = int(L)
        r = int(rows[s])
        if L == 0 or r < 0 or (L - 1) % b < b - w:
            continue
        val = probs[s, :, :L].reshape(h_kv, G, L).max(1) / w
        if (L - 1) % b == b - w:
            S[r, :, :L] = val
        else:
            S[r, :, :L - 1] += val[:, :L - 1]
            S[r, :, L - 1] = val[:, L - 1]
    return S
