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


@pytest.mark.parametrize("kv,h_q", [("fp4", 16), ("fp4", 128)])
def test_limits_that_run_out_anywhere(kv, h_q):
    """Units of 2 to 8 ms on few parts under limits of 1 to 8 ms: the wait for the
    next unit's query, and with it every other role's, runs out at some point of
    the work. The call returns, says so, and the next decode is right."""
    w = dataclasses.replace(W.get_workload("tiny"), batch=3, s_q=1, h_q=h_q, seqlens=[120000, 40000, 33333], causal=False, kv=kv, seed=229)
    check_limits(w, 2, (1.0, 1.3, 1.7, 2.2, 2.9, 3.7, 4.8, 6.2, 8.0))


def check_limits(w, parts, limits):
    d = G.to_device(W.make_inputs(w))
    make = lambda **kw: M.DecodeRunner(d["q"], d["kcache"], d["block_table"], d["cache_seqlens"], softmax_scale=w.scale,  # noqa: E731
                                       num_sm_parts=parts, **kw)
    good = make()
    good.plan()
    want = [t.clone() for t in good.run()]
    gave_up = 0
    for ms in limits:
        r = make(timeout_ns=int(ms * 1e6))
        r.plan()
        r.run()
        code, bits = r.status()
        assert (code, bits) in ((M.MLA_OK, 0), (M.MLA_ERR_DEVICE_TIMEOUT, M.MLA_DEVICE_STATUS_TIMEOUT))
        gave_up += code != M.MLA_OK
        out, lse = good.run()
        assert good.status() == (M.MLA_OK, 0)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert gave_up > 0
