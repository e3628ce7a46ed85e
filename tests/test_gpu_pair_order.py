"""CTA pairs read one another's operands on the word of a barrier: many decodes
of the same inputs under load, each bit for bit the first."""
import dataclasses

import pytest
import torch

import head_latent_attention_get_b200 as M
from tests import gpu_helpers as G
from workloads import mla_workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
@pytest.mark.parametrize("topk", [0, 2048])
def test_many_pair_decodes(kv, topk):
    w = dataclasses.replace(W.get_workload("tiny"), batch=20, s_q=1, h_q=128, seqlens=[2500 + 97 * i for i in range(20)], causal=False,
                            topk=topk, kv=kv, seed=223)
    inp = W.make_inputs(w, poison_tail=True)
    out, lse, r = G.run_gpu(inp)
    G.compare_full(inp, out, lse, f"{kv} {topk}")
    want = r.out.clone(), r.lse.clone()
    other = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    bad = torch.zeros((), dtype=torch.int32, device="cuda")
    for i in range(200):
        with torch.cuda.stream(side):
            other.add_(1)                 # traffic that shifts the roles against one another
        r.out.zero_()
        r.run()
        bad += (r.out != want[0]).any() | (r.lse != want[1]).any()
    torch.cuda.synchronize()
    assert int(bad) == 0 and r.status() == (M.MLA_OK, 0)
