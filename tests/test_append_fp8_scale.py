"""The FP8 scale that mla_kv_append forms, amax * fl(1/448), beside the quotient
amax / 448 of the records that the test data and mla_out_rope_fp8 hold: at most
the last bit apart, the same as torch's scalar division on the GPU, and no less
near to the row."""
import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M
from oracle import mla_oracle as O
from workloads import mla_workloads as W


def test_product_and_quotient_are_a_bit_apart():
    """For every finite positive bf16 maximum whose scale is a normal fp32: from
    448 * 2^-126 = 1.75 * 2^-118, bf16 0x04E0, on."""
    amax = (np.arange(0x04E0, 0x7F80, dtype=np.uint32) << 16).view(np.float32)
    prod, quot = amax * (np.float32(1) / np.float32(448)), amax / np.float32(448)
    assert quot.min() >= np.finfo(np.float32).tiny
    apart = np.abs(prod.view(np.int32) - quot.view(np.int32))
    assert apart.max() == 1 and 0.5 < (apart > 0).mean() < 0.6


@pytest.mark.gpu
def test_appended_scales():
    rng = np.random.default_rng(3)
    rows = torch.from_numpy((rng.standard_normal((640, 576)) * np.exp(rng.uniform(-8, 8, (640, 1)))).astype(np.float32)).bfloat16()
    cache = torch.zeros(10, 64, 656, dtype=torch.uint8, device="cuda")
    M.mla_kv_append(rows.cuda(), 576, 640, 576, None, 0.0, None, None, torch.arange(640, dtype=torch.int32, device="cuda"), cache, None,
                    M.MLA_KV_FP8_E4M3, 10)
    got = cache.cpu().view(640, 656)
    scale = got[:, 512:528].contiguous().view(torch.float32)
    on_gpu = (rows.cuda().float()[:, :512].reshape(640, 4, 128).abs().amax(-1) / 448.0).cpu()
    assert torch.equal(scale, on_gpu)
    host = W.quantize_fp8_records(rows.float().view(10, 64, 576)).view(640, 656)
    assert torch.equal(got[:, 528:], host[:, 528:])
    hs = host[:, 512:528].contiguous().view(torch.float32)
    assert (scale.view(torch.int32) - hs.view(torch.int32)).abs().max() == 1
    # either record: half an e4m3 step (2^-4 of a value, 2^-10 of the scale for subnormal codes), the scale's and the
    # quotient's fp32 roundings (2^-22), the value's rounding to bf16 (2^-8)
    x = rows.double().numpy()[:, :512]
    for rec in (got, host):
        v = O.dequant_fp8_records(rec.view(10, 64, 656).numpy()).reshape(640, 576)[:, :512]
        assert np.all(np.abs(v - x) <= (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -11) * np.abs(x) + 2.0 ** -10 * np.repeat(hs.numpy(), 128, 1))
