"""Inputs that show what a decode over a 4-bit cache does to every token's weight, and a bound for them.

Values come in pairs of tokens, half a sequence apart, that are exact opposites (lo = -7.5 steps, codes c and
15 - c), so that an output is the sum of what the two weights of a pair differ by, and its own rounding, relative to
it, is small beside what a rounded, lost or doubled weight changes.  A query has one element, so that logits are
exact to a few roundings."""
import numpy as np
import torch

import q4_util as q4
from test_gpu_q4_decode import Case


class Fine(Case):
    """kind of steps: "near" (within a factor of four), "flat" (a group without steps among any 32 tokens and the last),
    "up" and "down" (2^7 times larger, 2^15 times smaller, in the second half of either half), "far" (2^-40 to 1 among all)."""

    def __init__(self, zp, lens, h_q=32, h_kv=8, d=128, group=32, b=16, seed=0, extra=1, kind="near", spread=0.4):
        super().__init__(zp, lens, "bf16", h_q, h_kv, d, group, b, seed, extra)
        self.kind = kind
        rng = np.random.default_rng(seed + 1000)
        q = np.zeros((self.B, h_q, d), np.float32)
        at = rng.integers(0, d, size=(self.B, h_q))
        np.put_along_axis(q, at[..., None], rng.uniform(0.5, 1.0, size=(self.B, h_q, 1)) * spread, 2)
        self.q = torch.from_numpy(q).bfloat16()
        n = d // group
        for s in range(self.B):
            half = (int(self.lens[s]) + 1) // 2
            for t in range(half):
                for h in range(h_kv):
                    code = rng.integers(0, 16, size=d).astype(np.uint8)
                    f = {"near": 1.0, "flat": 1.0 if t % 16 != 1 and t + half != self.lens[s] - 1 else 0.0, "far": 2.0 ** -rng.integers(0, 41),
                         "up": 1.0 if 2 * t < half else 2.0 ** 7, "down": 1.0 if 2 * t < half else 2.0 ** -15}[kind]
                    step = (rng.integers(8, 16, size=n) / 16.0 * 2.0 ** rng.integers(-1, 1, size=n) * f).astype(np.float32)
                    if f == 0.0:
                        step[0] = 0.0
                        step[1:] = 0.25
                    lo = -7.5 * step                       # (four bits times fifteen: exact)
                    step = np.maximum(step, 2.0 ** -126)
                    word = q4.bf16_bits(step, True).astype(np.uint32) | q4.bf16_bits(lo, False).astype(np.uint32) << 16
                    for u, c in ((t, code), (t + half, 15 - code)):
                        if u < self.lens[s]:
                            q4.put_row(self.V, int(self.table[s, u // b]) * b + u % b, h, c, word, b)

    def weights(self, s):
        """Probabilities [h_q][L], values [h_kv][L][d] and the magnitudes of their parts, rounding of a probability
        [h_q], steps, and code * step [h_kv][L][d]."""
        L, G = int(self.lens[s]), self.h_q // self.h_kv
        p = np.arange(L)
        slots = self.table[s, p // self.b].astype(np.int64) * self.b + p % self.b
        kc = q4.get_rows(self.K, slots, self.d, self.group, self.b)
        vc = q4.get_rows(self.V, slots, self.d, self.group, self.b)
        k, v = q4.values(*kc, self.group), q4.values(*vc, self.group)
        k_abs, v_abs = (q4.values(x[0], x[1], np.abs(x[2]), self.group) for x in (kc, vc))
        q = self.q[s].double().numpy()
        x = np.stack([k[:, h // G] @ q[h] for h in range(self.h_q)]) / np.sqrt(self.d)
        size = np.stack([k_abs[:, h // G] @ np.abs(q[h]) for h in range(self.h_q)]).max(1) / np.sqrt(self.d)
        e = np.exp(x - x.max(1, keepdims=True))
        # a logit: lo and the code's part each a product, their sum, the scales, the difference from the maximum, fewer
        # than 12 roundings of the size of its parts; the exponential 2^-22
        code = q4.values(vc[0], vc[1], np.zeros_like(vc[2]), self.group)
        return (e / e.sum(1, keepdims=True), *(x.transpose(1, 0, 2) for x in (v, v_abs)), 12 * 2.0 ** -24 * size + 2.0 ** -22,
                vc[1], code.transpose(1, 0, 2))

    def outputs(self, prob, v):
        G = self.h_q // self.h_kv
        return np.stack([prob[h] @ v[h // G] for h in range(self.h_q)])

    def reference(self, s):
        """As Case.reference, with the bound that the roundings of the weights have."""
        prob, v, v_abs, ptol, step, codes = self.weights(s)
        L = int(self.lens[s])
        out, a, a_code = self.outputs(prob, v), self.outputs(prob, v_abs), self.outputs(prob, codes)
        # With the codes: a weight and its product with a step in fp16, each off by 2^-11 of itself at most; where steps of
        # all sizes meet among 32 tokens, the weight in two bf16 parts (2^-17), its product in two (2^-15).
        each = 2.0 ** -15 + 2.0 ** -17 if self.kind == "flat" and L >= 8 else 2 * 2.0 ** -11
        # With lo, and in the sum that divides: two bf16 parts, off by 2^-17 (8 bits, then 8 of what is left, which is
        # signed).  Sums in 32 bits: a range is 256 tokens at most here, two additions for 16 of them that each drop
        # 2^-23 at most, and up to 40 records.
        rel = 2 * 2.0 ** -17 + 2 * ptol + 256 / 16 * 2 * 2.0 ** -23 + 40 * 2.0 ** -24
        # What fp16 drops below its smallest number, 2^-24: half of it for each of two roundings of a weight, times a
        # code of 15, with the heaviest weight at 2^11 or more and a step that counts as one 2^4 times the first
        # unit's largest or less.
        lost = 2 * L * 15 * 2.0 ** -25 * 2.0 ** -11 * 2.0 ** 4 * float(step.max())
        tol = each * a_code + rel[:, None] * a + lost + torch.finfo(torch.bfloat16).eps / 2 * 1.01 * np.abs(out)
        return out, tol, prob, ptol
