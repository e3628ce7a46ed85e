"""A decode that gave up leaves nothing behind: its copies have landed before
its blocks end, so the next decodes are as if it had not been."""
import dataclasses

import pytest
import torch

import head_latent_attention_get_b200 as M
from tests import gpu_helpers as G
from workloads import mla_workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h_q", [16, 64, 128])
@pytest.mark.parametrize("topk", [0, 1024])
def test_decodes_after_timeouts(h_q, topk):
    """Scores withheld: the loaders stop with copies in flight, for every part
    of the grid at once. A good decode follows in the same stream each time."""
    check_after_timeouts("fp4", h_q, topk)


@pytest.mark.parametrize("kv,h_q,topk", [("bf16", 16, 0), ("bf16", 16, 1024), ("bf16", 128, 0), ("bf16", 128, 1024), ("fp8", 64, 0),
                                         ("fp8", 64, 1024)])
def test_decodes_after_timeouts_other_caches(kv, h_q, topk):
    check_after_timeouts(kv, h_q, topk)


def check_after_timeouts(kv, h_q, topk):
    w = dataclasses.replace(W.get_workload("tiny"), batch=40, s_q=1, h_q=h_q, seqlens=[1500 + 37 * i for i in range(40)], causal=False,
                            topk=topk, kv=kv, seed=211)
    d = G.to_device(W.make_inputs(w, poison_tail=True))
    make = lambda **kw: M.DecodeRunner(d["q"], d["kcache"], d["block_table"], d["cache_seqlens"], softmax_scale=w.scale,  # noqa: E731
                                       indices=d["indices"], **kw)
    good, bad = make(), make(timeout_ns=2_000_000, debug_flags=M.MLA_DEBUG_WITHHOLD_SCORES)
    good.plan()
    bad.plan()
    want = [t.clone() for t in good.run()]
    for _ in range(5):
        bad.run()
        out, lse = good.run()
        code, bits = bad.status()
        assert code == M.MLA_ERR_DEVICE_TIMEOUT and bits == M.MLA_DEVICE_STATUS_TIMEOUT
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        M.mla_clear_device_status(bad.workspace)
    assert good.status() == (M.MLA_OK, 0)


@pytest.mark.parametrize("kv,h_q", [("fp4", 16), ("fp4", 128), ("bf16", 16), ("bf16", 128), ("fp8", 64)])
def test_shortest_limit(kv, h_q):
    """A limit of 1 ns counts as 1 ms: a block's last waits are for its own
    copies and MMAs, so no limit may let it end before those. The decode takes
    microseconds and is not disturbed."""
    w = dataclasses.replace(W.get_workload("tiny"), batch=6, s_q=1, h_q=h_q, seqlens=[700 + 37 * i for i in range(6)], causal=False, kv=kv,
                            seed=227)
    inp = W.make_inputs(w, poison_tail=True)
    for _ in range(3):       # something else may hold the GPU for a millisecond
        out, lse, r = G.run_gpu(inp, dict(timeout_ns=1))
        if r.status() == (M.MLA_OK, 0):
            break
    assert r.status() == (M.MLA_OK, 0)
    G.compare_full(inp, out, lse, kv)


@pytest.mark.parametrize("h_q", [16, 128])
def test_limits_that_run_out_anywhere(h_q):
    """Two units of 160000 tokens in one part: the wait for the second one's query
    spans the first, which takes 1.4 ms at least (1088 x 2 x 160000 multiplications
    and additions for each of the 128 rows that a pair's or 64 that a CTA's MMAs work
    on, at 2.25 PFLOP/s / 148 a CTA). Limits below that run out, and with them
    every other role's wait, at some point of the work. The call returns, says so,
    and the next decode is right. The table names ten pages over and over."""
    w = dataclasses.replace(W.get_workload("tiny"), batch=2, s_q=1, h_q=h_q, seqlens=[640, 640], causal=False, kv="fp4", seed=229)
    d = G.to_device(W.make_inputs(w))
    table, lens = d["block_table"].repeat(1, 250), torch.full((2,), 160000, dtype=torch.int32, device="cuda")
    make = lambda **kw: M.DecodeRunner(d["q"], d["kcache"], table, lens, softmax_scale=w.scale, num_sm_parts=1, **kw)  # noqa: E731
    good = make()
    good.plan()
    want = [t.clone() for t in good.run()]
    for limit in (1_000_000, 1_050_000, 1_110_000, 1_170_000, 1_230_000, 1_290_000, 3_000_000, 10_000_000):
        r = make(timeout_ns=limit)
        r.plan()
        r.run()
        code, bits = r.status()
        gave_up = M.MLA_ERR_DEVICE_TIMEOUT, M.MLA_DEVICE_STATUS_TIMEOUT
        assert (code, bits) == gave_up if limit < 1_400_000 else (code, bits) in (gave_up, (M.MLA_OK, 0))
        out, lse = good.run()
        assert good.status() == (M.MLA_OK, 0)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
