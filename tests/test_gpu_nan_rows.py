"""A query row with a NaN gives NaN in its output and its log-sum-exp, however its
unit is split, and is not taken for a row without keys; the other rows are bit
for bit what they are without it."""
import dataclasses

import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M
from tests import gpu_helpers as G
from workloads import mla_workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,h_q,topk", [(kv, h, t) for kv in ("fp4", "bf16", "fp8") for h, t in ((16, 0), (128, 0), (16, 512), (128, 512))])
@pytest.mark.parametrize("parts", [1, 5])
def test_nan_query_rows(kv, h_q, topk, parts):
    w = dataclasses.replace(W.get_workload("tiny"), batch=2, s_q=1, h_q=h_q, seqlens=[1500, 600], causal=False, kv=kv, topk=topk, seed=311)
    inp = W.make_inputs(w, poison_tail=True)
    out, lse, _ = G.run_gpu(inp, dict(num_sm_parts=parts))
    bad = np.zeros((2, 1, h_q), bool)
    bad[0, 0, 3] = bad[0, 0, h_q - 1] = bad[1, 0, 0] = True
    q = inp.q.clone()
    q[0, 0, 3, 7] = q[0, 0, h_q - 1, 570] = q[1, 0, 0, 511] = float("nan")
    out2, lse2, r = G.run_gpu(dataclasses.replace(inp, q=q), dict(num_sm_parts=parts))
    assert r.status() == (M.MLA_OK, 0)
    assert np.isnan(out2[bad]).all() and np.isnan(lse2[bad]).all()
    assert np.array_equal(out2[~bad], out[~bad]) and np.array_equal(lse2[~bad], lse[~bad])
