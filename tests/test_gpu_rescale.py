"""Rows whose running maximum jumps while their neighbours' does not: the
decode kernels multiply a row's accumulated output by a factor when its maximum
grows by more than 2^8, so heads that share a warp must be free to differ.

One key per RoPE dim stands out for the heads that look at that dim, in a later
tile than the others'; every third head looks at none. The share of the keys
before it stays large (all values have mean 1), so a factor that is lost,
applied twice or applied to a neighbour is far outside the tolerance."""
import dataclasses

import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M
from oracle import mla_oracle as O
from tests import gpu_helpers as G
from workloads import mla_workloads as W

TOKENS = 1664           # 13 tiles of 128: an odd number, so that a pair's last step is half empty
JUMP_LOG2 = 11.0        # of the key that stands out, over scores of 0 +- 1.5


def jump_inputs(kv, h_q, sparse):
    w = dataclasses.replace(W.get_workload("tiny"), batch=1, s_q=1, h_q=h_q, seqlens=[TOKENS], causal=False, kv=kv, seed=7 + h_q)
    inp = W.make_inputs(w)
    rng = np.random.default_rng(h_q)
    src = rng.standard_normal((inp.num_pages, 64, 576)).astype(np.float32)
    src[..., :512] += 1.0
    src[..., 512:] = 0.0
    pages = inp.block_table[0].numpy()
    for dim in range(64):
        t = 128 * (1 + dim % 12) + int(rng.integers(128))
        src[pages[t // 64], t % 64, 512 + dim] = 16.0
    q = rng.standard_normal((1, 1, h_q, 576)) / 4
    q[..., :512] -= q[..., :512].mean(-1, keepdims=True)     # the values' mean does not move the scores
    q[..., 512:] = 0.0
    for h in range(h_q):
        if h % 3:
            q[0, 0, h, 512 + (7 * h) % 64] = JUMP_LOG2 * np.log(2) / (16.0 * w.scale)
    src = torch.from_numpy(src)
    cache = src.bfloat16().unsqueeze(2) if kv == "bf16" else W.quantize_fp4_records(src) if kv == "fp4" else W.quantize_fp8_records(src)
    idx = torch.arange(TOKENS, dtype=torch.int32).view(1, 1, TOKENS) if sparse else None
    return dataclasses.replace(inp, q=torch.from_numpy(q.astype(np.float32)).bfloat16(), kcache=cache.contiguous(), indices=idx,
                               workload=dataclasses.replace(w, topk=TOKENS if sparse else 0))


def rescaled_rows(inp, step):
    """[steps, rows]: which rows grow past the threshold in a step of `step` keys after their first."""
    q, cache = O.inputs_to_f64(inp)
    rows = O.gather_rows(cache, inp.block_table[0].numpy(), np.arange(TOKENS))
    s = q[0, 0] @ rows.T * inp.workload.scale / np.log(2)
    used, hit = np.full(len(s), -np.inf), []
    for t in range(0, TOKENS, step):
        top = s[:, t:t + step].max(1)
        grow = top - used > 8
        hit.append(grow & (t > 0))
        used = np.where(grow, top, used)
    return np.array(hit)


CASES = [(kv, h_q, sparse) for kv in ("fp4", "bf16", "fp8") for h_q in (16, 48, 80, 128) for sparse in (False, True)]


@pytest.mark.parametrize("kv,h_q,sparse", CASES)
def test_rows_of_a_warp_differ(kv, h_q, sparse):
    """What the GPU test below relies on: in some step some rows of a warp (16
    of a single CTA, 32 of a pair) need the factor and some do not."""
    hit = rescaled_rows(jump_inputs(kv, h_q, sparse), 256 if h_q > 64 else 128)
    per = 32 if h_q > 64 else 16
    for r0 in range(0, h_q, per):
        some = hit[:, r0:r0 + per]
        assert (some.any(1) & ~some.all(1)).any(), r0
    assert not hit[:, ::3].any()


@pytest.mark.gpu
@pytest.mark.parametrize("kv,h_q,sparse", CASES)
@pytest.mark.parametrize("parts", [1, 2])
def test_rescaled_rows(kv, h_q, sparse, parts):
    """Every element: the probabilities' rounding (at most half a bf16 step,
    2^-8, of each, so of the largest value), the output's (2^-8 of it), and 2e-4
    for the fp32 scores (below 2^5, off by 2^-18 of it)."""
    inp = jump_inputs(kv, h_q, sparse)
    out, lse, r = G.run_gpu(inp, dict(num_sm_parts=parts))
    assert r.status() == (M.MLA_OK, 0)
    ref_o, ref_l = O.reference_decode(inp)
    assert np.abs(ref_l).max() < 100
    vmax = np.abs(O.inputs_to_f64(inp)[1][..., :512]).max()
    assert np.all(np.abs(out - ref_o) <= 2.0 ** -8 * (np.abs(ref_o) + vmax) + 2e-4)
    assert np.abs(lse - ref_l).max() <= G.LSE_ATOL
