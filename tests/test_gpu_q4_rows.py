"""Rows of a 4-bit cache as the kernels keep and give them: their distance from what was stored, and rows of several
layers and both tensors between one another."""
import numpy as np
import pytest
import torch

import q4_util as q4
from test_gpu_q4_store import _dev, _rows, zp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,layers", [(1, 3), (40, 2)])
def test_rows_between_one_another(zp, dtype, n, layers):  # noqa: F811
    """[token][layer][k, v][h_kv][d], taken and given."""
    rng = np.random.default_rng(n)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    h_kv, d = 3, 64
    desc = zp.cache_desc(h_kv, h_kv, d, 16, 4, t)
    x = _rows(rng, (n, layers, 2, h_kv, d), dtype)
    xd = x.cuda().permute(2, 1, 0, 3, 4)
    K, V = zp.zp_q4_cache(desc, 32, layers)
    slots = _dev(rng.permutation(64)[:n].astype(np.int32))
    zp.zp_q4_write_kv(desc, xd[0], xd[1], slots, K, V)
    got = torch.full_like(x, 7.0, device="cuda")
    gd = got.permute(2, 1, 0, 3, 4)
    zp.zp_q4_read_kv(desc, K, V, slots, gd[0], gd[1])
    code, word = q4.quantise(x.float().numpy(), 32)
    want = q4.values(code, q4.bf16_value(word & 0xFFFF), q4.bf16_value(word >> 16), 32)
    assert torch.equal(got.cpu(), torch.from_numpy(want).float().to(t))
    with pytest.raises(zp.ZPError, match="on one another"):
        zp.zp_q4_read_kv(desc, K, V, slots, gd[0], gd[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,group", [(128, 32), (128, 64), (64, 64), (128, 128)])
def test_distance(zp, dtype, d, group):  # noqa: F811
    """What the kernel keeps is no further from a row than half a step and what x - lo is rounded by (2^-24 of it);
    for bf16 rows lo is the smallest element."""
    rng = np.random.default_rng(d + group)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = _rows(rng, (300, 4, d), dtype)
    desc = zp.cache_desc(4, 4, d, 16, 20, t)
    K, V = zp.zp_q4_cache(desc, group)
    slots = rng.permutation(320)[:300].astype(np.int32)
    zp.zp_q4_write_kv(desc, x.cuda(), x.cuda(), _dev(slots), K, V, group=group)
    code, step, lo = q4.get_rows(K.cpu().numpy(), slots, d, group, 16)
    g = x.double().numpy().reshape(300, 4, -1, group)
    ok = np.isfinite(lo)  # (a spread past the largest float reads as NaN)
    assert ok.mean() > 0.9 and np.array_equal(ok, ~np.isnan(step))
    err = np.abs(q4.values(code, step, lo, group).reshape(g.shape) - g)
    with np.errstate(invalid="ignore"):
        bound = step[..., None].astype(np.float64) / 2 + 2.0 ** -24 * np.abs(g - lo[..., None])
    assert (err <= bound)[ok].all(), float((err / bound)[ok].max())
    if dtype == "bf16":
        assert np.array_equal(lo[ok], g.min(-1)[ok].astype(np.float32))
