"""Prefix-shared decode where a CTA takes many short items one after another: the
queries of the next item follow the records of the last in the same shared memory."""
import numpy as np
import pytest
import torch

from tests.prefix_util import attention_bounds
from tests.test_gpu_prefix_attn import BF16, DEV, F32, Case, zp  # noqa: F401 (zp is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(32, 8, 128, 16, BF16), (16, 2, 128, 16, BF16), (32, 4, 64, 16, BF16), (32, 8, 128, 16, F32)],
                         ids=["g4", "g8", "d64", "f32"])
@pytest.mark.parametrize("scored", [False, True])
def test_many_items_per_cta(zp, heads, scored):  # noqa: F811
    """380 groups, one to three tiles each, some with more rows than one stream has: against the oracle, and the
    same bits every time."""
    sizes = [2 + (i % 7 == 0) * 3 + (i % 95 == 0) * 40 for i in range(380)]
    c = Case(zp, 201, heads, sizes, [1 + (5 * i) % 24 for i in range(380)], (1, 20), 3, 1)
    if scored:
        c.score_rows(202, 11)
    out, S = c.run(zp)
    c.check(out, S)
    for _ in range(8):
        out2, S2 = c.run(zp)
        assert torch.equal(out, out2) and (S is None or torch.equal(S, S2))


def test_hundreds_of_whole_sequences_per_cta(zp):  # noqa: F811
    """One sequence with most of the private tokens among many just begun: the CTAs behind its end see some 150
    whole sequences each."""
    h_q, h_kv, d, b, B, long_blocks = 4, 1, 64, 16, 600, 23000
    g = torch.Generator(device=DEV).manual_seed(211)
    rng = np.random.default_rng(211)
    lens = 3 * b + rng.integers(1, 17, size=B)
    lens[0] = long_blocks * b
    n_total = long_blocks + 3 + B
    ids = rng.permutation(n_total).astype(np.int32)
    table = np.full((B, long_blocks), -1, np.int32)
    table[:, :3] = ids[:3]
    table[1:, 3] = ids[3:3 + B - 1]
    table[0, 3:] = ids[3 + B - 1:3 + B - 1 + long_blocks - 3]
    desc = zp.cache_desc(h_q, h_kv, d, b, n_total, BF16)
    mk = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    K, V, q = mk(n_total, b, h_kv, d), mk(n_total, b, h_kv, d), mk(B, h_q, d)
    td, ld = (torch.from_numpy(x.astype(np.int32)).to(DEV) for x in (table, lens))
    plan = zp.prefix_plan(B)
    zp.zp_prefix_plan(desc, td, ld, plan)
    assert plan.n_groups.tolist() == [1] and plan.prefix_lens.tolist() == [3 * b] * B
    out, alone = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    zp.zp_prefix_decode_attn(desc, q, K, V, td, ld, plan, out)
    zp.zp_paged_decode_attn(desc, q, K, V, td, ld, alone)
    torch.cuda.synchronize()
    assert zp.zp_device_status() == (0, 0)
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    ref, tol, _, _ = attention_bounds(f(q)[1:], f(K), f(V), np.maximum(table[1:, :4], 0), lens[1:].astype(np.int32), True)
    assert (np.abs(f(out)[1:] - ref) <= tol).all()
    # the long one: both within 2^-8 (sum p |v| + |out|) of the same value; |v| is below 6
    torch.testing.assert_close(out[0].float(), alone[0].float(), rtol=2.0 ** -7, atol=6 * 2.0 ** -7)
