"""4-bit decoding of rows with one large probability over very many small ones:
the small ones count in the output as they do in the row's sum, down to 2^-31 of
the largest."""
import dataclasses

import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M
from oracle import mla_oracle as O
from tests import gpu_helpers as G
from workloads import mla_workloads as W

pytestmark = pytest.mark.gpu

# score of a head's peak over the other keys' 0, in nats: probabilities of 2^-12.3 .. 2^-30.3
PEAKS = (8.5, 10.0, 12.0, 13.5, 15.0, 16.5, 17.5, 18.0, 19.0, 20.0, 21.0)


def peaked_inputs(h_q, tokens, sparse):
    w = dataclasses.replace(W.get_workload("tiny"), batch=1, s_q=1, h_q=h_q, seqlens=[tokens], causal=False, kv="fp4", scale=1.0,
                            topk=tokens if sparse else 0, seed=301)
    inp = W.make_inputs(dataclasses.replace(w, topk=0))
    rng = np.random.default_rng(h_q)
    src = np.zeros((inp.num_pages, 64, 576), np.float32)
    src[..., :512] = (1.0 + rng.standard_normal(src[..., :512].shape) / 4).clip(0.25)   # the small keys' values: mean 1
    pages = inp.block_table[0].numpy()
    for j, peak in enumerate(PEAKS):
        t = 0 if j % 2 == 0 else int(rng.integers(tokens))                 # first, or anywhere
        src[pages[t // 64], t % 64, :512] = 0.0
        src[pages[t // 64], t % 64, 512 + j] = peak
    q = torch.zeros(1, 1, h_q, 576)
    for h in range(h_q):
        q[0, 0, h, 512 + h % len(PEAKS)] = 1.0
    idx = torch.arange(tokens, dtype=torch.int32).view(1, 1, tokens) if sparse else None
    return dataclasses.replace(inp, q=q.bfloat16(), kcache=W.quantize_fp4_records(torch.from_numpy(src)), indices=idx, workload=w)


@pytest.mark.parametrize("h_q", [11, 64, 128])
@pytest.mark.parametrize("tokens,sparse", [(6016, False), (6016, True), (65536, False)])
def test_small_probabilities_count(h_q, tokens, sparse):
    """Bound per element. A probability p (of the row's largest) is held with 2^7
    in front of it as f16: off by 2^-11 p, or 2^-25 of that scale, 2^-32, where f16
    is subnormal. The output is rounded to bf16, by 2^-8 of it at most. The fp32
    exponents (below 2^5, a few roundings of 2^-24 of it) move a p by 2^-16 of it;
    the fp32 accumulators, which may truncate, move by 2^-23 for each 16 keys."""
    inp = peaked_inputs(h_q, tokens, sparse)
    out, lse, r = G.run_gpu(inp, dict(num_sm_parts=1))
    assert r.status() == (M.MLA_OK, 0)
    ref_o, ref_l = O.reference_decode(inp)
    v = O.inputs_to_f64(inp)[1][..., :512]
    assert v.min() >= 0                                  # so that the sum of p |v| is the output itself
    bound = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16 + tokens * 2.0 ** -27) * ref_o + tokens * 2.0 ** -32 * v.max()
    assert np.all(np.abs(out - ref_o) <= bound), np.max((np.abs(out - ref_o) - bound) / ref_o)
    assert np.abs(lse - ref_l).max() <= G.LSE_ATOL
