"""4-bit decoding with RoPE keys of up to 2^100 and queries that match them."""
import dataclasses

import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M
from oracle import mla_oracle as O
from tests import gpu_helpers as G
from workloads import mla_workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h_q", [16, 128])
@pytest.mark.parametrize("exp", [-100, 97])
def test_rope_keys_far_from_one(h_q, exp):
    """Keys' RoPE dims times 2^exp (|values| below 2^3), the query's times 2^-exp and
    its latent part 0: the scores are those of RoPE alone."""
    w = dataclasses.replace(W.get_workload("tiny"), batch=2, s_q=1, h_q=h_q, seqlens=[300, 129], causal=False, kv="fp4", scale=0.125, seed=307)
    inp = W.make_inputs(w, poison_tail=False)
    inp.q[..., :512] = 0
    inp.q[..., 512:] = (inp.q[..., 512:].double() * 2.0 ** -exp).to(torch.bfloat16)
    rope = inp.kcache[..., 288:].contiguous().view(torch.bfloat16)
    inp.kcache[..., 288:] = (rope.double() * 2.0 ** exp).to(torch.bfloat16).view(torch.uint8)
    out, lse, r = G.run_gpu(inp)
    assert r.status() == (M.MLA_OK, 0)
    ref_o, ref_l = O.reference_decode(inp)
    vmax = np.abs(O.inputs_to_f64(inp)[1][..., :512]).max()
    # half a bf16 step of the output, half an f16 step of each probability (so of the largest value), 1e-4 for fp32 scores below 2^4
    assert np.all(np.abs(out - ref_o) <= 2.0 ** -8 * np.abs(ref_o) + 2.0 ** -11 * vmax + 1e-4)
    assert np.abs(lse - ref_l).max() <= G.LSE_ATOL
