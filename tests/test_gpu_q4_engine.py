"""The decode loop over a 4-bit cache against the same loop over an fp32 cache of the values that the
codes stand for: tables, lengths and pool exact; outputs, scores and keep sets to rounding."""
import numpy as np
import pytest
import torch


pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,b,budgets,async_compress", [(32, 16, None, False), (64, 32, None, True), (32, 16, "own", False)])
def test_loop(group, b, budgets, async_compress):
    import compressed_paged_kv_zp_gb300 as zp
    from compressed_paged_kv_zp_gb300.engine import DecodeLoop
    zp.zp_device_status(clear=True)
    h_q, h_kv, d, layers, B, N_max, n_total, stride = 16, 4, 64, 2, 5, 4, 90, 12
    rng = np.random.default_rng(group + b)
    lens0 = rng.integers(b + 3, (N_max - 1) * b, size=B).astype(np.int32)
    own = None if budgets is None else np.array([4, 3, 2, 4, 3], np.int32)
    loops = []
    for bits in (4, 16):
        prm = zp.score_params(window=b, use_similarity=False)
        loop = DecodeLoop(h_q, h_kv, d, b, n_total, N_max, stride, layers=layers, dtype=torch.float32, window=b, params=prm,
                          async_compress=async_compress, kv_bits=bits, kv_group=group)
        loop.add_sequences(lens0, max_blocks=own)
        loops.append(loop)
    four, full = loops
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731

    every = torch.arange(n_total * b, dtype=torch.int32, device="cuda")

    def stored(k, v):
        """The values that new rows [layers][n][h_kv][d] are kept as."""
        n = k.shape[1]
        desc = zp.cache_desc(h_q, h_kv, d, b, -(-n // b), torch.float32)
        K, V = zp.zp_q4_cache(desc, group, layers)
        at = torch.arange(n, dtype=torch.int32, device="cuda")
        zp.zp_q4_write_kv(desc, k, v, at, K, V, group=group)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        zp.zp_q4_read_kv(desc, K, V, at, ko, vo, group=group)
        return ko, vo

    k, v = rnd(layers, n_total * b, h_kv, d), rnd(layers, n_total * b, h_kv, d)
    zp.zp_q4_write_kv(four.desc, k, v, every, four.K, four.V, group=group)
    zp.zp_q4_read_kv(four.desc, four.K, four.V, every, full.K.view(layers, -1, h_kv, d), full.V.view(layers, -1, h_kv, d), group=group)
    compressed = 0
    for step in range(3 * b):
        q, kn, vn = rnd(layers, B, h_q, d), rnd(layers, B, h_kv, d), rnd(layers, B, h_kv, d)
        for loop in loops:
            if async_compress:
                loop.drain()
        trig = four.step(q, kn, vn)
        assert trig == full.step(q, *stored(kn, vn))
        torch.cuda.synchronize()
        assert np.array_equal(four.table, full.table) and np.array_equal(four.lens, full.lens)
        # fp32 on both sides: products of 64 terms and sums of up to 128 tokens, each rounded by 2^-24 of values
        # below 64 in the logits; a logit error e changes a weight by the factor 1 + e
        assert torch.allclose(four.out, full.out, rtol=1e-4, atol=1e-4)
        if trig:
            compressed += len(trig)
            seqs, keep = four.last_keep
            keep, other = keep.cpu().numpy(), full.last_keep[1].cpu().numpy()
            for loop in loops:
                loop.drain()
            torch.cuda.synchronize()
            assert np.array_equal(keep, other)
            slots = torch.cat([torch.as_tensor(four.table[s, :four.N_seq[s] - 1], device="cuda")[:, None] * b +
                               torch.arange(b, device="cuda") for s in seqs]).flatten().int()
            got = torch.empty(2, layers, slots.numel(), h_kv, d, device="cuda")
            zp.zp_q4_read_kv(four.desc, four.K, four.V, slots, got[0], got[1], group=group)
            for x, cache, F in ((got[0], full.K, four.F), (got[1], full.V, full.F)):
                assert torch.equal(x, cache.view(layers, -1, h_kv, d)[:, slots.long()])
            assert torch.allclose(four.F.view(layers, -1, h_kv)[:, slots.long()], full.F.view(layers, -1, h_kv)[:, slots.long()],
                                  rtol=1e-4, atol=1e-8)
    assert compressed >= B
    assert four.pool.num_free == full.pool.num_free
    assert zp.zp_device_status() == (0, 0)


def test_refusals():
    import compressed_paged_kv_zp_gb300 as zp
    from compressed_paged_kv_zp_gb300.engine import DecodeLoop
    for kw in (dict(kv_bits=8), dict(kv_bits=4, prefix_decode=True), dict(kv_bits=4, params=zp.score_params(use_similarity=True))):
        with pytest.raises(ValueError):
            DecodeLoop(8, 2, 64, 16, 20, 4, 8, **kw)
