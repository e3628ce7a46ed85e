"""mla_kv_append with values that are not finite: what the header says of the
tile, block or row, and every other byte as without them."""
import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M
from tests.test_gpu_cache_fill import new_cache

pytestmark = pytest.mark.gpu

INF = float("inf")
T, ROW, AT = 5, 2, 133       # the third row's value 133: FP8 tile 1, E2M1 block 8


def store(kv, fmt, gamma=None, eps=1e-6):
    d = kv.shape[1]
    cache, scale = new_cache(fmt, 1)
    vals = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    M.mla_kv_append(kv.cuda(), d, T, d, None if gamma is None else gamma.cuda(), eps, None, None, slots, cache, scale, fmt, 1, vals)
    torch.cuda.synchronize()
    return cache.cpu().numpy(), None if scale is None else scale.cpu().numpy(), vals.float().cpu().numpy()


def rows(d):
    g = torch.Generator().manual_seed(5)
    return torch.randn(T, d, generator=g).bfloat16()


def differing(a, b):
    """(row, byte) places where two stores differ."""
    return {(int(r), int(c)) for r, c in zip(*np.nonzero(a != b))}


@pytest.mark.parametrize("x", [INF, -INF])
def test_bf16_stores_infinities(x):
    kv = rows(576)
    base, _, _ = store(kv, M.MLA_KV_BF16)
    kv[ROW, AT] = x
    got, _, vals = store(kv, M.MLA_KV_BF16)
    assert differing(got, base) <= {(ROW, 2 * AT), (ROW, 2 * AT + 1)}
    assert np.array_equal(vals, kv.float().numpy())


@pytest.mark.parametrize("x", [INF, -INF, float("nan")])
def test_fp8_tile(x):
    kv = rows(576)
    base, _, _ = store(kv, M.MLA_KV_FP8_E4M3)
    kv[ROW, AT] = x
    got, _, vals = store(kv, M.MLA_KV_FP8_E4M3)
    tile = AT // 128
    mine = {(ROW, c) for c in [*range(128 * tile, 128 * tile + 128), *range(512 + 4 * tile, 516 + 4 * tile)]}
    assert differing(got, base) <= mine
    if np.isinf(x):
        assert got[ROW, 512 + 4 * tile:516 + 4 * tile].view(np.float32)[0] == INF
        assert np.isnan(vals[ROW, 128 * tile:128 * tile + 128]).all()


@pytest.mark.parametrize("fmt", [M.MLA_KV_FP4_E2M1, M.MLA_KV_NVFP4])
@pytest.mark.parametrize("x", [INF, -INF, float("nan")])
def test_e2m1_block(fmt, x):
    kv = rows(576 if fmt == M.MLA_KV_FP4_E2M1 else 512)
    base, bs, _ = store(kv, fmt)
    kv[ROW, AT] = x
    got, gs, vals = store(kv, fmt)
    if fmt == M.MLA_KV_FP4_E2M1:
        bs, gs, base, got = base[:, 256:], got[:, 256:], base[:, :256], got[:, :256]   # codes | scales and RoPE
    blk = AT // 16
    assert differing(got, base) <= {(ROW, c) for c in range(8 * blk, 8 * blk + 8)}
    assert differing(gs, bs) <= {(ROW, blk)}
    if np.isinf(x):
        assert gs[ROW, blk] == 0x7E and vals[ROW, AT] == np.sign(x) * 2688
        others = np.delete(np.arange(16 * blk, 16 * blk + 16), AT % 16)
        assert np.all(vals[ROW, others] == 0)          # at most 4 of a step of 224


@pytest.mark.parametrize("fmt", [M.MLA_KV_BF16, M.MLA_KV_FP8_E4M3, M.MLA_KV_NVFP4, M.MLA_KV_FP4_E2M1])
@pytest.mark.parametrize("x", [INF, float("nan")])
def test_norm_keeps_them_in_their_row(fmt, x):
    kv = rows(512 if fmt == M.MLA_KV_NVFP4 else 576)
    gamma = torch.ones(512)
    base, bs, _ = store(kv, fmt, gamma)
    kv[ROW, AT] = x
    got, gs, _ = store(kv, fmt, gamma)
    keep = np.arange(64) != ROW
    assert np.array_equal(got[keep], base[keep]) and (gs is None or np.array_equal(gs[keep], bs[keep]))


def test_zero_row_under_the_norm():
    kv = rows(576)
    kv[ROW] = 0
    _, _, vals = store(kv, M.MLA_KV_BF16, torch.ones(512), eps=0.0)
    assert np.isnan(vals[ROW, :512]).all() and np.isfinite(np.delete(vals, ROW, 0)).all()
    _, _, vals = store(kv, M.MLA_KV_BF16, torch.ones(512), eps=1e-6)
    assert np.all(vals[ROW] == 0)
