"""Decode over a 4-bit cache with logits far from zero, where a float's step is a few units and more."""
import numpy as np
import pytest
import torch

import q4_util as q4
from test_gpu_q4_decode import Case, zp  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = 4096  # table columns past every cluster: the units of all pairs are cut evenly
BOTH = pytest.mark.parametrize("extra", [1, WIDE])
DTYPES = pytest.mark.parametrize("dtype", ["bf16", "f32"])


def out_type(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _words(step, lo):
    return (q4.bf16_bits(step, True).astype(np.uint32) | q4.bf16_bits(lo, False).astype(np.uint32) << 16).astype(np.uint32)


def _set_live(c, cache, token):
    """Every live row of a cache (those behind the sequences stay NaN) gets the codes and words token(s, t) gives."""
    for s in range(c.B):
        for t in range(int(c.lens[s])):
            slot = int(c.table[s, t // c.b]) * c.b + t % c.b
            for h in range(c.h_kv):
                code, word = token(s, t, h)
                q4.put_row(cache, slot, h, code, word, c.b)


def _mean_of_values(c, s):
    """Mean and mean magnitude (lo and code apart) of a sequence's values, [h_q][d]."""
    p = np.arange(int(c.lens[s]))
    rows = q4.get_rows(c.V, c.table[s, p // c.b].astype(np.int64) * c.b + p % c.b, c.d, c.group, c.b)
    v = q4.values(*rows, c.group).mean(0)
    a = q4.values(rows[0], rows[1], np.abs(rows[2]), c.group).mean(0)
    return (np.repeat(x, c.h_q // c.h_kv, axis=0) for x in (v, a))


@BOTH
@DTYPES
@pytest.mark.parametrize("top", [3e7, 1.5e8, 2.6e8, 5e8, 1e12, -3e7, -1.5e8, -2.6e8, -1e12])
def test_equal_logits(zp, dtype, top, extra):  # noqa: F811
    """One key for all tokens, whose logit is `top` in units of log 2: the mean of the values."""
    c = Case(zp, [300, 33, 1], dtype, 8, 2, 128, 32, 16, seed=5, extra=extra)
    rng = np.random.default_rng(6)
    code = rng.integers(0, 16, size=(2, 128)).astype(np.uint8)
    code[:, :32] = 0
    step, lo = np.full(4, 0.25, np.float32), np.full(4, -1.0, np.float32)
    lo[0] = top / (32 / np.sqrt(128) * np.log2(np.e))  # 32 ones of the query meet it
    word = _words(step, lo)
    _set_live(c, c.K, lambda s, t, h: (code[h], word))
    c.q[..., :32] = 1.0
    out = c.run().double().numpy()
    for s in range(c.B):
        want, a = _mean_of_values(c, s)
        L = int(c.lens[s])
        # equal weights, a power of two each: what is summed is exact to 2^-24, the output rounded once (by half a
        # step at most, that is eps / 2 of the value: bf16 has 8 bits, 2^-8)
        tol = (2 * L + 8) * 2.0 ** -24 * a + torch.finfo(out_type(dtype)).eps / 2 * 1.01 * np.abs(want)
        assert (np.abs(out[s] - want) <= tol).all(), (s, float((np.abs(out[s] - want) / tol).max()))


@BOTH
@DTYPES
@pytest.mark.parametrize("scale", [3e6, 6e6, 1.2e7, 2.5e7, 5e7, 1e8, 1e10])
def test_one_value(zp, dtype, scale, extra):  # noqa: F811
    """Logits of all sizes up to some 5 * scale, known to a float's step only: the same value in all tokens, which is
    the output whatever the weights."""
    c = Case(zp, [300, 33, 1, 700], dtype, 8, 2, 128, 32, 16, seed=8, extra=extra, q_scale=scale)
    rng = np.random.default_rng(9)
    code = rng.integers(0, 16, size=(2, 128)).astype(np.uint8)
    word = _words(rng.uniform(0.1, 0.4, size=(2, 4)).astype(np.float32), rng.uniform(-3, -0.5, size=(2, 4)).astype(np.float32))
    _set_live(c, c.V, lambda s, t, h: (code[h], word[h]))
    out = c.run().double().numpy()
    for s in range(c.B):
        want, a = _mean_of_values(c, s)
        # a weight and its product with a step: 11 bits or more each in bf16 (half a step: 2^-11), far more in fp32
        each, L = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22, int(c.lens[s])
        tol = (2 * each + L * 2.0 ** -23) * a + torch.finfo(out_type(dtype)).eps / 2 * 1.01 * np.abs(want)
        assert (np.abs(out[s] - want) <= tol).all(), (s, float((np.abs(out[s] - want) / tol).max()))


@BOTH
@DTYPES
@pytest.mark.parametrize("top", [0.0, 3e4, 3e7, 1.5e8, 1e12, -3e4, -3e7, -1.5e8, -1e12])
def test_score_of_equal_logits(zp, dtype, top, extra):  # noqa: F811
    """Scored on the first step of the window: each of L tokens has a share of 1 / L."""
    c = Case(zp, [289, 33, 1, 4097], dtype, 8, 2, 64, 32, 16, seed=5, extra=extra)
    code = np.zeros(64, np.uint8)
    word = _words(np.full(2, 0.25, np.float32), np.array([top / (32 / 8 * np.log2(np.e)), -1.0], np.float32))
    _set_live(c, c.K, lambda s, t, h: (code, word))
    c.q[..., :32] = 1.0
    S = torch.full((4, 2, c.table.shape[1] * 16), 9.0, device="cuda")
    c.run(16, S)
    for s in range(c.B):
        L = int(c.lens[s])
        got = S[s, :, :L].cpu().double().numpy() * 16 * L
        # two differences of at most 32 rounded to 32 bits (2^-20 each), a logarithm, an exponential and a product
        assert (np.abs(got - 1) <= 2.0 ** -18 + L * 2.0 ** -24).all(), (s, float(np.abs(got - 1).max()))
        assert (S[s, :, L:] == 9.0).all()


@BOTH
@DTYPES
@pytest.mark.parametrize("scale", [1.0, 1e3, 3e6, 2.5e7, 1e8, 1e10])
def test_scores_add_up(zp, dtype, scale, extra):  # noqa: F811
    """One q head per kv head: the scores of a sequence are its probabilities, whatever the logits are."""
    c = Case(zp, [289, 33, 1, 1025], dtype, 2, 2, 64, 32, 16, seed=11, extra=extra, q_scale=scale)
    S = torch.zeros(4, 2, c.table.shape[1] * 16, device="cuda")
    c.run(16, S)
    for s in range(c.B):
        total = S[s].cpu().double().numpy().sum(-1) * 16
        assert (np.abs(total - 1) <= 2.0 ** -18 + int(c.lens[s]) * 2.0 ** -24).all(), (s, total)
