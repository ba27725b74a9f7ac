"""The decode loop over a 4-bit cache in bf16 with heads of 128 against the same loop in fp32 over the values that the
codes stand for: tables, lengths, pool and moved rows exact; outputs, scores and keep sets to rounding."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h_q,h_kv,group,b,async_compress", [(32, 8, 32, 16, False), (16, 4, 128, 32, True)])
def test_loop(h_q, h_kv, group, b, async_compress):
    import compressed_paged_kv_zp_gb300 as zp
    from compressed_paged_kv_zp_gb300.engine import DecodeLoop
    zp.zp_device_status(clear=True)
    d, layers, B, N_max, n_total, stride = 128, 2, 5, 4, 90, 12
    rng = np.random.default_rng(group + b)
    lens0 = rng.integers(b + 3, (N_max - 1) * b, size=B).astype(np.int32)
    loops = []
    for bits, dtype in ((4, torch.bfloat16), (16, torch.float32)):
        prm = zp.score_params(window=b, use_similarity=False)
        loop = DecodeLoop(h_q, h_kv, d, b, n_total, N_max, stride, layers=layers, dtype=dtype, window=b, params=prm,
                          async_compress=async_compress, kv_bits=bits, kv_group=group)
        loop.add_sequences(lens0)
        loops.append(loop)
    four, full = loops
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    every = torch.arange(n_total * b, dtype=torch.int32, device="cuda")

    def stored(k, v):
        """The values that new rows [layers][n][h_kv][d] are kept as, in fp32."""
        n = k.shape[1]
        desc = zp.cache_desc(h_q, h_kv, d, b, -(-n // b), torch.float32)
        K, V = zp.zp_q4_cache(desc, group, layers)
        at = torch.arange(n, dtype=torch.int32, device="cuda")
        zp.zp_q4_write_kv(desc, k.float(), v.float(), at, K, V, group=group)
        ko, vo = torch.empty_like(k, dtype=torch.float32), torch.empty_like(v, dtype=torch.float32)
        zp.zp_q4_read_kv(desc, K, V, at, ko, vo, group=group)
        return ko, vo

    k, v = rnd(layers, n_total * b, h_kv, d), rnd(layers, n_total * b, h_kv, d)
    zp.zp_q4_write_kv(four.desc, k, v, every, four.K, four.V, group=group)
    zp.zp_q4_read_kv(full.desc, four.K, four.V, every, full.K.view(layers, -1, h_kv, d), full.V.view(layers, -1, h_kv, d), group=group)
    # a weight and its product with a step are off by 2^-11 each, with values whose parts are below 17 (normal ones of
    # 5.5 at most: |lo| + 15 steps, three times that), the output by 2^-8 of itself
    tol = dict(rtol=2.0 ** -8, atol=17 * 2.0 ** -10)
    compressed = 0
    for step in range(3 * b):
        q, kn, vn = rnd(layers, B, h_q, d), rnd(layers, B, h_kv, d), rnd(layers, B, h_kv, d)
        for loop in loops:
            if async_compress:
                loop.drain()
        trig = four.step(q, kn, vn)
        assert trig == full.step(q.float(), *stored(kn, vn))
        torch.cuda.synchronize()
        assert np.array_equal(four.table, full.table) and np.array_equal(four.lens, full.lens)
        assert torch.allclose(four.out.float(), full.out, **tol)
        if trig:
            compressed += len(trig)
            seqs, keep = four.last_keep
            other = full.last_keep[1].cpu().numpy()
            for loop in loops:
                loop.drain()
            torch.cuda.synchronize()
            assert np.array_equal(keep.cpu().numpy(), other)
            slots = torch.cat([torch.as_tensor(four.table[s, :four.N_seq[s] - 1], device="cuda")[:, None] * b +
                               torch.arange(b, device="cuda") for s in seqs]).flatten().int()
            got = torch.empty(2, layers, slots.numel(), h_kv, d, device="cuda")
            zp.zp_q4_read_kv(full.desc, four.K, four.V, slots, got[0], got[1], group=group)
            for x, cache in ((got[0], full.K), (got[1], full.V)):
                assert torch.equal(x, cache.view(layers, -1, h_kv, d)[:, slots.long()])
            assert torch.allclose(four.F.view(layers, -1, h_kv)[:, slots.long()], full.F.view(layers, -1, h_kv)[:, slots.long()],
                                  rtol=1e-4, atol=1e-8)
    assert compressed >= B
    assert four.pool.num_free == full.pool.num_free
    assert zp.zp_device_status() == (0, 0)
