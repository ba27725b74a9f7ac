"""The bound that the decode over a 4-bit cache is held to notices what it is there to notice: weights rounded to
fewer bits, and tokens that are lost or doubled, planted in the definition (no GPU needed)."""
import numpy as np
import pytest

from q4_fine import Fine


@pytest.fixture(scope="module")
def zp():
    import compressed_paged_kv_zp_gb300 as m
    return m


def _cut(x, bits):
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 2.0 ** bits), e - bits)


def _worst(c, s, plant=lambda p: p, bits=60):
    """Largest error over bound with `plant` in place of probabilities [h_q][L], and with probabilities and their
    products with the steps cut to `bits` bits where they meet the codes."""
    want, tol, prob, _ = c.reference(s)
    _, v, _, _, step, code = c.weights(s)  # step [L][h_kv][groups]
    prob, G = plant(prob.copy()), c.h_q // c.h_kv
    got = c.outputs(prob, v - code)
    for h in range(c.h_q):
        st = np.repeat(step[:, h // G].astype(np.float64), c.group, axis=1)
        got[h] += (_cut(_cut(prob[h], bits)[:, None] * st, bits) * (code[h // G] / st)).sum(0)
    return float((np.abs(got - want) / tol).max())


@pytest.mark.parametrize("kind", ["near", "flat", "up", "down", "far"])
@pytest.mark.parametrize("L", [2, 10, 34, 64, 200])
def test_bits(zp, kind, L):
    """The bits that are promised pass.  8 do not over few tokens, nor 11 where more are promised."""
    c = Fine(zp, [L], kind=kind, seed=L)
    more = kind == "flat" and L >= 8
    assert _worst(c, 0, bits=16 if more else 11) < 1
    assert L > 10 or _worst(c, 0, bits=8) > 1.5
    assert not more or _worst(c, 0, bits=8) > 4
    assert not more or L > 64 or _worst(c, 0, bits=11) > 1


@pytest.mark.parametrize("L,places", [(64, (31, 32)), (700, (31, 64, 96, 352)), (2600, (31, 32, 96, 1023, 1024, 2400, 2598))])
def test_tokens(zp, L, places):
    """One token lost or twice, and a unit lost."""
    c = Fine(zp, [L], h_q=8, h_kv=2, seed=L, kind="flat")
    for t in places:
        for f in (0.0, 2.0):
            def one(p):
                p[:, t] *= f
                return p / p.sum(1, keepdims=True)
            assert _worst(c, 0, one) > 1.5

    def unit(p):
        p[:, 32:64] = 0
        return p / p.sum(1, keepdims=True)
    assert _worst(c, 0, unit) > 1.5
