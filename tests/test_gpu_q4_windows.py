"""Decode over a 4-bit cache whose values' steps change by far along a sequence (bf16 products take their steps
relative to a window of sizes): groups that are flat, tiny or huge for a while, then not."""
import numpy as np
import pytest
import torch

import q4_util as q4
from test_gpu_q4_decode import Case, zp  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = 4096  # table columns past every cluster: the units of all pairs are cut evenly
TINY = 2.0 ** -126


def _scale_tokens(c, factor):
    """Steps and lowest values of token t of every sequence times factor(t, rng) (0: a flat group at zero)."""
    head = 8 * c.d
    n = c.d // c.group
    word = np.ascontiguousarray(c.V[..., head:]).view(np.uint32).reshape(c.n_total, c.h_kv, c.b // 16, 16, n)
    for s in range(c.B):
        t = np.arange(int(c.lens[s]))
        f = factor(t)[:, None, None]
        at = (c.table[s, t // c.b], slice(None), t % c.b // 16, t % 16)
        w = word[at]
        step = np.maximum(q4.bf16_value(w & 0xFFFF) * f, TINY).astype(np.float32)
        lo = (q4.bf16_value(w >> 16) * f).astype(np.float32)
        word[at] = q4.bf16_bits(step, True).astype(np.uint32) | q4.bf16_bits(lo, False).astype(np.uint32) << 16
    c.V[..., head:] = word.reshape(c.n_total, c.h_kv, c.b // 16, 16 * n).view(np.uint8).reshape(c.V[..., head:].shape)


SHAPES = pytest.mark.parametrize("lens,h_q,h_kv,extra", [([900, 40], 8, 2, 1), ([900, 40], 8, 2, WIDE), ([2500] * 30, 4, 1, 1),
                                                         ([200] * 500, 8, 8, 1)])


@SHAPES
@pytest.mark.parametrize("first", ["zero", 2.0 ** -60, 2.0 ** -30, 2.0 ** 40])
@pytest.mark.parametrize("then", [1.0, 2.0 ** 10, 2.0 ** 20, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("q_scale", [0.0, 1.0])
def test_then_large(zp, lens, h_q, h_kv, extra, first, then, q_scale):  # noqa: F811
    """Stretches of 100 tokens of one size among tokens of another, over flat and ordinary logits."""
    c = Case(zp, lens, "bf16", h_q, h_kv, 64, 32, 16, seed=3, extra=extra, q_scale=q_scale)
    f = 0.0 if first == "zero" else first
    _scale_tokens(c, lambda t: np.where(t // 100 % 3 == 0, f, then))
    out = c.run()
    assert bool(torch.isfinite(out.float()).all())
    for s in sorted({0, 1, c.B // 2, c.B - 1}):
        want, tol, _, _ = c.reference(s)
        assert (np.abs(out[s].double().numpy() - want) <= tol).all(), (s, float((np.abs(out[s].double().numpy() - want) / tol).max()))


@pytest.mark.parametrize("extra", [1, WIDE])
@pytest.mark.parametrize("at", [0, 31, 32, 250])
@pytest.mark.parametrize("size", [2.0 ** 25, 2.0 ** 60, 2.0 ** 80])
def test_one_large_token(zp, extra, at, size):  # noqa: F811
    """One token of a great range among flat ones."""
    c = Case(zp, [300], "bf16", 8, 2, 128, 64, 16, seed=4, extra=extra, q_scale=0.5)
    _scale_tokens(c, lambda t: np.where(t == at, size, 0.0))
    c.check(c.run())
