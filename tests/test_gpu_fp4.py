"""GPU parity of decoding over 4-bit token records (MLA_KV_FP4_E2M1), paged and
token-sparse, on both kernels (units of at most 64 rows, and of 65-128 rows),
against the fp64 oracle. The tolerances are the bf16 path's (gpu_helpers):
the stored values are exact in bf16, so the arithmetic is the same."""
import dataclasses

import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M
from oracle import mla_oracle as O
from tests import gpu_helpers as G
from workloads import mla_workloads as W

pytestmark = pytest.mark.gpu


def _w(**kw):
    base = dict(batch=2, s_q=1, h_q=16, seqlens=[70, 129], causal=False, kv="fp4", seed=31)
    return dataclasses.replace(W.get_workload("tiny"), **{**base, **kw})


def _check(w, sink=False, where="", few=True, **runner):
    inp = W.make_inputs(w, poison_tail=True, extra_pages=2)
    if sink:
        inp = W.with_sink(inp, seed=w.seed)
    out, lse, r = G.run_gpu(inp, runner)
    assert r.status() == (M.MLA_OK, 0)
    if sink and any(L == 0 for L in w.seqlens):
        ref_o, ref_l = O.reference_decode(inp)
        assert np.abs(out - ref_o).max() <= G.OUT_ATOL and np.abs(lse - ref_l).max() <= G.LSE_ATOL
    else:
        G.compare_full(inp, out, lse, where or str(w), few_keys=few)
    return inp, out, lse


@pytest.mark.parametrize("lens", [[1], [0, 1, 63], [64, 65, 127], [128, 129, 255, 256, 257], [1000, 3, 0, 700]])
@pytest.mark.parametrize("h_q", [1, 16, 40, 64, 65, 128])
def test_paged_lengths(lens, h_q):
    _check(_w(batch=len(lens), h_q=h_q, seqlens=lens, seed=40 + h_q))


@pytest.mark.parametrize("s_q,h_q", [(2, 16), (3, 5), (6, 64), (2, 128), (7, 31)])
@pytest.mark.parametrize("sink", [False, True])
def test_causal_query_blocks(s_q, h_q, sink):
    _check(_w(batch=4, s_q=s_q, h_q=h_q, seqlens=[1, 4, 130, 900], causal=True, seed=51), sink=sink)


@pytest.mark.parametrize("parts", [1, 3, 37])
@pytest.mark.parametrize("h_q", [16, 128])
def test_split_units(parts, h_q):
    _check(_w(batch=3, h_q=h_q, seqlens=[5000, 129, 2300], seed=61), num_sm_parts=parts)


@pytest.mark.parametrize("h_q,topk", [(1, 64), (16, 64), (48, 192), (64, 320), (96, 64), (128, 2048)])
@pytest.mark.parametrize("s_q", [1, 2])
def test_sparse(h_q, topk, s_q):
    _check(_w(batch=4, s_q=s_q, h_q=h_q, seqlens=[300, 1, 2500, 64], topk=topk, neg_frac=0.1, seed=71))


@pytest.mark.parametrize("h_q", [16, 128])
def test_sparse_empty_and_out_of_range(h_q):
    """All indices -1 gives out 0 and lse -inf; out-of-range values are ignored
    and reported."""
    w = _w(batch=2, h_q=h_q, seqlens=[200, 300], topk=128, neg_frac=0.0, seed=81)
    inp = W.make_inputs(w)
    inp.indices[0] = -1
    out, lse, r = G.run_gpu(inp)
    assert r.status() == (M.MLA_OK, 0)
    G.compare_full(inp, out, lse, "empty", few_keys=True)
    inp.indices[1, 0, :7] = torch.tensor([300, -2, 1 << 30, -(1 << 31), 301, 999999, 2147483647], dtype=torch.int32)
    out, lse, r = G.run_gpu(inp)
    assert r.status() == (M.MLA_ERR_DEVICE_BOUNDS, M.MLA_DEVICE_STATUS_BOUNDS)
    G.compare_full(inp, out, lse, "out of range", few_keys=True)


@pytest.mark.parametrize("h_q", [32, 128])
def test_sparse_of_all_positions_equals_paged(h_q):
    """Every position listed in order is paged decoding, bit for bit: the
    kernels do the same arithmetic in the same order."""
    w = _w(batch=2, h_q=h_q, seqlens=[512, 512], seed=91)
    inp = W.make_inputs(w)
    out, lse, _ = G.run_gpu(inp, dict(num_sm_parts=2))
    idx = torch.arange(512, dtype=torch.int32).expand(2, 1, 512).contiguous()
    sp = dataclasses.replace(inp, indices=idx, workload=dataclasses.replace(w, topk=512))
    out2, lse2, _ = G.run_gpu(sp, dict(num_sm_parts=2))
    assert np.array_equal(out, out2) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("h_q", [16, 128])
def test_extreme_scales_and_codes(h_q):
    """All 16 codes under the smallest, an ordinary and the largest scale
    (a UE4M3 sign bit is ignored): every stored value is exact, so a row that
    sees one key returns that key's value, rounded to bf16 once."""
    w = _w(batch=6, h_q=h_q, seqlens=[1] * 6, seed=93)
    inp = W.make_inputs(w)
    for b, sc in enumerate([0x01, 0x07, 0x38, 0x7E, 0xFE, 0x00]):
        rec = inp.kcache[int(inp.block_table[b, 0]), 0]
        rec[:256] = torch.arange(256, dtype=torch.uint8)
        rec[256:288] = sc
    out, lse, _ = G.run_gpu(inp)
    _, cache = O.inputs_to_f64(inp)
    for b in range(6):
        v = torch.from_numpy(cache[int(inp.block_table[b, 0]), 0, :512]).to(torch.bfloat16).float().numpy()
        assert np.array_equal(out[b, 0], np.broadcast_to(v, (h_q, 512)))


@pytest.mark.parametrize("h_q", [16, 128])
def test_bad_page_ids_are_reported(h_q):
    w = _w(batch=2, h_q=h_q, seqlens=[200, 300], seed=95)
    inp = W.make_inputs(w)
    inp.block_table[1, 2] = 1 << 20
    out, lse, r = G.run_gpu(inp)
    assert r.status() == (M.MLA_ERR_DEVICE_BOUNDS, M.MLA_DEVICE_STATUS_BOUNDS)
    ref_o, ref_l = O.reference_decode(W.restrict(inp, [0]))
    assert np.abs(out[:1] - ref_o).max() <= G.OUT_ATOL and np.abs(lse[:1] - ref_l).max() <= G.LSE_ATOL


@pytest.mark.parametrize("h_q", [16, 128])
def test_repeats_are_bit_identical(h_q):
    w = _w(batch=5, h_q=h_q, seqlens=[3000, 129, 64, 2500, 1], seed=97)
    inp = W.make_inputs(w, poison_tail=True)
    d = G.to_device(inp)
    r = M.DecodeRunner(d["q"], d["kcache"], d["block_table"], d["cache_seqlens"], softmax_scale=w.scale)
    r.plan()
    first = [t.clone() for t in r.run()]
    for _ in range(10):
        out, lse = r.run()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("h_q", [16, 128])
def test_wait_limit_is_reported(h_q):
    w = _w(batch=2, h_q=h_q, seqlens=[300, 129], seed=99)
    inp = W.make_inputs(w)
    d = G.to_device(inp)
    r = M.DecodeRunner(d["q"], d["kcache"], d["block_table"], d["cache_seqlens"], softmax_scale=w.scale,
                       timeout_ns=20_000_000, debug_flags=M.MLA_DEBUG_WITHHOLD_SCORES)
    r.plan()
    r.run()
    torch.cuda.synchronize()
    code, bits = r.status()
    assert code == M.MLA_ERR_DEVICE_TIMEOUT and bits & M.MLA_DEVICE_STATUS_TIMEOUT


def test_noalloc_entry_point():
    w = _w(batch=3, h_q=16, seqlens=[3000, 129, 64], seed=101)
    inp = W.make_inputs(w, poison_tail=True)
    out, lse, r = G.run_gpu(inp)
    d = G.to_device(inp)
    o2, l2 = torch.empty_like(r.out), torch.empty_like(r.lse)
    a = M.make_args(q=d["q"], kcache=d["kcache"], block_table=d["block_table"], cache_seqlens=d["cache_seqlens"],
                    tile_md=r.tile_md, num_splits=r.num_splits, out=o2, lse=l2, workspace=None, workspace_bytes=0,
                    batch=3, s_q=1, h_q=16, h_kv=1, num_pages=d["kcache"].shape[0], num_sm_parts=r.parts,
                    softmax_scale=w.scale, causal=False, kv_format=M.MLA_KV_FP4_E2M1)
    from head_latent_attention_get_b200 import _capi as C
    C.mla_decode_paged_noalloc(a)
    torch.cuda.synchronize()
    assert np.array_equal(o2.float().cpu().numpy(), out) and np.array_equal(l2.cpu().numpy(), lse)


@pytest.mark.parametrize("h_q", [16, 128])
def test_graph_replay_with_new_lengths(h_q):
    """Plan and decode captured once, replayed after the lengths and the query
    changed in place."""
    w = _w(batch=3, h_q=h_q, seqlens=[900, 900, 900], seed=103)
    inp = W.make_inputs(w)
    d = G.to_device(inp)
    r = M.DecodeRunner(d["q"], d["kcache"], d["block_table"], d["cache_seqlens"], softmax_scale=w.scale)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r.plan()
        r.run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.plan()
        r.run()
    for lens in ([900, 1, 0], [64, 513, 899]):
        d["cache_seqlens"].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        sub = dataclasses.replace(inp, cache_seqlens=torch.tensor(lens, dtype=torch.int32))
        ref_o, ref_l = O.reference_decode(sub)
        G.compare(r.out.float().cpu().numpy(), r.lse.cpu().numpy(), ref_o, ref_l, str(lens), inp=sub)


@pytest.mark.parametrize("h_q", [16, 128])
def test_long_context(h_q):
    _check(_w(batch=1, h_q=h_q, seqlens=[131072], seed=105), few=False)


@pytest.mark.parametrize("h_q,topk", [(16, 0), (128, 0), (16, 64), (128, 64)])
def test_cache_beyond_4_gib(h_q, topk):
    """Pages past the cache's first 2^32 bytes, through the append and both
    decode kernels: the same results as for a small cache with the same rows."""
    w = _w(batch=2, h_q=h_q, seqlens=[200, 129], topk=topk, seed=107)
    inp = W.make_inputs(w, poison_tail=True)
    out, lse, _ = G.run_gpu(inp)
    pages = (1 << 32) // (64 * 416) + 64
    big = torch.empty(pages, 64, 416, dtype=torch.uint8, device="cuda")
    shift = pages - inp.num_pages
    big[shift:].copy_(inp.kcache)
    moved = dataclasses.replace(inp, block_table=torch.where(inp.block_table >= 0, inp.block_table + shift, inp.block_table))
    d = G.to_device(dataclasses.replace(moved, kcache=inp.kcache[:1]))
    d["kcache"] = big
    out2, lse2, r = G.run_gpu(moved, dev_inputs=d)
    assert r.status() == (M.MLA_OK, 0)
    assert np.array_equal(out, out2) and np.array_equal(lse, lse2)
    kv = torch.randn(3, 576, device="cuda").bfloat16()
    last = torch.tensor([pages * 64 - 1, 0, pages * 64 - 66], dtype=torch.int32, device="cuda")
    small = torch.zeros(2, 64, 416, dtype=torch.uint8, device="cuda")
    M.mla_kv_append(kv, 576, 3, 576, None, 0.0, None, None, last, big, None, M.MLA_KV_FP4_E2M1, pages)
    M.mla_kv_append(kv, 576, 3, 576, None, 0.0, None, None, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), small,
                    None, M.MLA_KV_FP4_E2M1, 2)
    torch.cuda.synchronize()
    assert torch.equal(big.view(-1, 416)[last.long()], small.view(-1, 416)[:3])


def test_two_decodes_at_once():
    """Two decodes on two streams, each with its own workspace."""
    runs = []
    for h_q, seed in ((16, 111), (128, 113)):
        w = _w(batch=6, h_q=h_q, seqlens=[3000, 129, 64, 2500, 1, 700], seed=seed)
        d = G.to_device(W.make_inputs(w, poison_tail=True))
        r = M.DecodeRunner(d["q"], d["kcache"], d["block_table"], d["cache_seqlens"], softmax_scale=w.scale)
        r.plan()
        alone = [t.clone() for t in r.run()]
        runs.append((r, alone, torch.cuda.Stream(), d))
    torch.cuda.synchronize()
    for _ in range(5):
        for r, _, s, _ in runs:
            r.plan(s)
            r.run(s)
    torch.cuda.synchronize()
    for r, alone, _, _ in runs:
        assert torch.equal(r.out, alone[0]) and torch.equal(r.lse, alone[1])


def test_queries_of_any_magnitude():
    """A row's query is scaled by a power of two on its way to the tensor core:
    rows from 2^-100 to 2^12 times a common one, and a zero row, with the scale
    undone by softmax_scale for one of them at a time."""
    w = _w(batch=1, h_q=16, seqlens=[300], seed=115)
    inp = W.make_inputs(w)
    base = inp.q[0, 0, :1].clone()
    for i in range(16):
        inp.q[0, 0, i] = (base.float() * 2.0 ** (12 - 7 * i)).to(torch.bfloat16)
    inp.q[0, 0, 15] = 0
    for scale in (w.scale, w.scale * 2.0 ** 9, w.scale * 2.0 ** 86):
        sub = dataclasses.replace(inp, workload=dataclasses.replace(w, scale=scale))
        out, lse, _ = G.run_gpu(sub)
        ref_o, ref_l = O.reference_decode(sub)
        # rows whose scores are spread over thousands are a maximum; fp32 scores are off by 2^-20 of the largest one
        tol = 2.0 ** -20 * np.abs(ref_l)
        assert np.all(np.abs(lse - ref_l) <= G.LSE_ATOL + tol)
        tame = tol[..., None] < 1e-4
        assert np.all(np.abs(out - ref_o) * tame <= G.OUT_ATOL + 2.0 ** -8 * np.abs(ref_o))


@pytest.mark.parametrize("h_q", [4, 80])
@pytest.mark.parametrize("row_exp,scale_exp", [((115, 125, 0, -120), -115), ((-120, -126, -90, -120), 120),
                                               ((-120, -126, 0, -60), -100)])
def test_queries_at_the_ends_of_the_range(h_q, row_exp, scale_exp):
    """The largest and the smallest queries that bf16 holds, the rows' power of
    two undone by softmax_scale, and one so small in total that every score is
    0: its row is the mean of the values, masked keys still without weight."""
    w = _w(batch=1, h_q=h_q, seqlens=[300], seed=117)
    inp = W.make_inputs(w)
    base = inp.q[0, 0, :1].double().clamp(-4, 4)
    for i in range(h_q):
        inp.q[0, 0, i] = (base * 2.0 ** row_exp[i % 4]).to(torch.bfloat16)
    sub = dataclasses.replace(inp, workload=dataclasses.replace(w, scale=w.scale * 2.0 ** scale_exp))
    out, lse, _ = G.run_gpu(sub)
    ref_o, ref_l = O.reference_decode(sub)
    tol = 2.0 ** -20 * np.abs(ref_l)   # fp32 scores, as above
    assert np.all(np.abs(lse - ref_l) <= G.LSE_ATOL + tol)
    tame = tol[..., None] < 1e-4
    assert np.all(np.abs(out - ref_o) * tame <= G.OUT_ATOL + 2.0 ** -8 * np.abs(ref_o))
