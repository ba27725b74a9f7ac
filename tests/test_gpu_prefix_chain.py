"""Prefix-shared decode followed at once by the compression call on the same stream.

The last kernel of the prefix decode (the joining kernel, or the score) lets the
compression's first kernel start early, and the decode's default workspace is given
back as soon as its launches are issued, so that the compression's scratch is the same
memory.  Bit for bit the state of the same calls with a synchronisation between them.
"""
import numpy as np
import pytest
import torch

import zp_inputs

pytestmark = pytest.mark.gpu

B, H_Q, H_KV, D, BS, N_MAX, SHARED = 64, 32, 8, 128, 16, 8, 40


@pytest.mark.parametrize("scored", [True, False])
def test_prefix_decode_then_compression_is_bit_exact(scored):
    import compressed_paged_kv_zp_gb300 as zp
    g = torch.Generator().manual_seed(77)
    lens = (torch.randint(1024, 2049, (B,), generator=g) // BS * BS).tolist()
    c = zp_inputs.make_paged_case(77, B, H_Q, H_KV, D, BS, lens=lens, dtype="bf16")
    comp = list(range(0, B, 4))
    table = c.block_table.numpy().copy()
    table[:, :SHARED] = table[0, :SHARED]
    k, n = (N_MAX - 1) * BS, len(comp)
    targets = torch.arange(c.n_total, c.n_total + n * (N_MAX - 1), dtype=torch.int32).view(n, N_MAX - 1)  # fresh blocks
    n_total = c.n_total + targets.numel()
    desc = zp.cache_desc(H_Q, H_KV, D, BS, n_total, torch.bfloat16)
    wide = lambda x: torch.cat([x, torch.zeros(targets.numel(), BS, H_KV, D, dtype=x.dtype)]).cuda()  # noqa: E731
    K0, V0 = wide(c.k_cache[0]), wide(c.v_cache[0])
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    td, ld, q = dev(table), dev(c.seq_lens.numpy()), c.q.cuda()
    c_table, c_lens, rows, c_targets = dev(table[comp]), dev(c.seq_lens.numpy()[comp]), dev(comp), targets.cuda()
    first = torch.tensor([i % 2 for i in range(n)], dtype=torch.uint8, device="cuda")
    Lmax = int(c.seq_lens.max())
    plan = zp.prefix_plan(B)
    zp.zp_prefix_plan(desc, td, ld, plan)
    assert plan.prefix_lens.tolist() == [SHARED * BS] * B
    S0 = torch.rand(B, H_KV, td.shape[1] * BS, generator=g).cuda()
    F0 = (torch.rand(n_total, BS, H_KV, generator=g) * 1e-3).cuda()
    params = zp.score_params(window=BS)

    def run(chained):
        K, V, F, S = K0.clone(), V0.clone(), F0.clone(), S0.clone()
        out = torch.empty_like(q)
        keep = torch.empty(n, H_KV, k, dtype=torch.int32, device="cuda")
        kw = dict(score_accum=S, window=BS) if scored else {}
        torch.cuda.synchronize()
        zp.zp_prefix_decode_attn(desc, q, K, V, td, ld, plan, out, **kw)
        if not chained:
            torch.cuda.synchronize()
        zp.zp_compress_layers(desc, params, K, V, c_table, c_lens, first, S, F, c_targets, k, keep, Lmax, rows=rows)
        torch.cuda.synchronize()
        assert zp.zp_device_status() == (0, 0)
        return dict(out=out, S=S, K=K, V=V, F=F, keep=keep)

    ref = run(False)
    for _ in range(6):
        got = run(True)
        for name in ref:
            assert torch.equal(got[name], ref[name]), name
