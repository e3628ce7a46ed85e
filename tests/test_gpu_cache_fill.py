"""GPU tests of mla_extend_tables and mla_kv_append against plain host
implementations, and of a run of them with decoding over the cache they fill."""
import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M
from oracle import mla_oracle as O
from tests import gpu_helpers as G
from workloads import mla_workloads as W

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------------- block tables and slots
def ref_tables(ctx, new, free, begin, end, num_pages, bt, stride, max_tokens):
    """Request by request, as the definition reads."""
    bt = bt.copy()
    slots, pos = np.full(max_tokens, -1), np.full(max_tokens, -1)
    lens, start, bits, tok, place = [], [], 0, 0, begin
    if not 0 <= begin <= end <= len(free):
        begin_ok, bits = False, M.MLA_DEVICE_STATUS_BOUNDS
    else:
        begin_ok = True
    avail, want, taken = (end - begin if begin_ok else 0), 0, 0
    for b, (c, a) in enumerate(zip(ctx.tolist(), new.tolist())):
        start.append(tok)
        t0, tok = tok, tok + max(a, 0)
        if c < 0 or a < 0 or c + a > stride * 64 or tok > max_tokens:
            bits |= M.MLA_DEVICE_STATUS_BOUNDS
            lens.append(max(c, 0))
            continue
        have, need = -(-c // 64), -(-(c + a) // 64) - -(-c // 64)
        want += need
        if need and want > avail:
            bits |= M.MLA_DEVICE_STATUS_NO_PAGES
            lens.append(c)
            continue
        for j in range(need):
            pg = free[begin + want - need + j]
            if not 0 <= pg < num_pages:
                pg, bits = -1, bits | M.MLA_DEVICE_STATUS_BOUNDS
            bt[b, have + j] = pg
        if need:
            taken = want
        lens.append(c + a)
        for i in range(a):
            p = c + i
            pg = bt[b, p // 64]
            pos[t0 + i] = p
            if 0 <= pg < num_pages:
                slots[t0 + i] = pg * 64 + p % 64
            else:
                bits |= M.MLA_DEVICE_STATUS_BOUNDS
    return dict(block_table=bt, seqlens=lens, token_start=start + [tok], slots=slots, positions=pos,
                free_next=[begin + taken]), bits


def run_tables(ctx, new, free, begin, end, num_pages, bt, max_tokens, stream=None):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    B = len(ctx)
    out = dict(block_table=d(bt), seqlens=d(np.full(B, 77)), token_start=d(np.full(B + 1, 77)),
               slots=d(np.full(max_tokens, 77)), positions=d(np.full(max_tokens, 77)), free_next=d([77]))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.mla_extend_tables(d(ctx), d(new), B, d(free) if len(free) else None, d([begin, end]), num_pages,
                        out["block_table"], bt.shape[1], out["seqlens"], out["token_start"], out["slots"],
                        out["positions"], max_tokens, out["free_next"], st, stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}, int(st.item())


def make_tables(ctx, stride, spare, seed):
    rng = np.random.default_rng(seed)
    have = [-(-max(int(c), 0) // 64) for c in ctx]
    P = sum(have) + spare
    perm = rng.permutation(P)
    bt = np.full((len(ctx), stride), -1)
    off = 0
    for b, h in enumerate(have):
        h = min(h, stride)
        bt[b, :h] = perm[off:off + h]
        off += h
    return bt, perm[off:], P


def check_tables(ctx, new, stride, max_tokens, spare=64, begin=0, end=None, seed=1, edit=None):
    ctx, new = np.asarray(ctx), np.asarray(new)
    bt, free, P = make_tables(ctx, stride, spare, seed)
    if edit:
        edit(bt, free)
    end = len(free) if end is None else end
    want, bits = ref_tables(ctx, new, free, begin, end, P, bt, stride, max_tokens)
    got, st = run_tables(ctx, new, free, begin, end, P, bt, max_tokens)
    for k in want:
        assert np.array_equal(got[k], np.asarray(want[k])), k
    assert st == bits
    return bits


@pytest.mark.parametrize("B", [1, 7, 255, 2047, 2048, 2049, 5000])
@pytest.mark.parametrize("hi_new", [1, 3, 70])
def test_tables_random(B, hi_new):
    rng = np.random.default_rng(B + hi_new)
    ctx, new = rng.integers(0, 500, B), rng.integers(0, hi_new + 1, B)
    assert check_tables(ctx, new, 10, int(new.sum()) + rng.integers(1, 700), spare=2 * B + 8, begin=3) == 0


@pytest.mark.parametrize("ctx,new", [([0], [1]), ([0], [0]), ([63, 64, 65], [1, 1, 1]), ([0, 0, 0], [64, 65, 128]),
                                     ([1, 640, 5], [639, 0, 635]), ([127, 0], [0, 2048])])
def test_tables_page_edges(ctx, new):
    bits = check_tables(ctx, new, 40, 4096)
    assert bits == 0


def test_tables_long_prefill():
    check_tables([0, 70, 8192, 63], [8192, 30000, 1, 4097], 800, 50000, spare=1000)


def test_tables_refusals():
    """Negative lengths, full rows, tokens past the axis and an empty free list
    refuse single requests; the others are served."""
    B, NP = M.MLA_DEVICE_STATUS_BOUNDS, M.MLA_DEVICE_STATUS_NO_PAGES
    assert check_tables([-1, 5, 10, 640], [3, -2, 4, 1], 10, 64) == B
    assert check_tables([60, 60, 60], [2, 2, 2], 10, 5) == B                       # the third's tokens end at 6
    assert check_tables([64, 64, 10, 64, 3], [70, 1, 5, 1, 2], 10, 200, end=2) == NP    # 64 + 1 finds none, 10 + 5 needs none
    assert check_tables([64, 3], [1, 1], 10, 8, end=0) == NP
    assert check_tables([64, 3], [1, 1], 10, 8, begin=5, end=4) == B | NP               # a range that is none
    assert check_tables([64, 3], [1, 1], 10, 8, end=1000) == B | NP


def test_tables_empty_free_list():
    got, st = run_tables(np.array([3, 64]), np.array([2, 1]), np.array([]), 0, 0, 4, np.array([[1, -1], [2, -1]]), 4)
    assert st == M.MLA_DEVICE_STATUS_NO_PAGES and got["seqlens"].tolist() == [5, 64]
    assert got["slots"].tolist() == [67, 68, -1, -1] and got["free_next"].tolist() == [0]


def test_tables_bad_page_ids():
    def edit(bt, free):
        bt[0, 0] = 9999
        free[1] = -7
    assert check_tables([10, 64, 64], [3, 1, 1], 10, 8, edit=edit) == M.MLA_DEVICE_STATUS_BOUNDS


def test_tables_other_entries_are_left():
    def edit(bt, free):
        bt[:, 5:] = 123456
    check_tables([100, 0], [10, 70], 10, 100, edit=edit)


# -------------------------------------------------------------------------- append
def ref_rows(kv, gamma, eps, cos, sin, d):
    """bf16 rows after norm and RoPE, by the header's roundings: the factor from
    64 bits, each fp32 operation rounded once."""
    f = np.float32
    x = O.torch_bf16_to_f64(kv)
    y = x[:, :512].astype(f)
    if gamma is not None:
        r = (1.0 / np.sqrt((x[:, :512] ** 2).sum(1, keepdims=True) / 512 + np.float64(f(eps)))).astype(f)
        y = ((y * r).astype(f) * gamma.numpy()).astype(f)
    row = np.concatenate([y, x[:, 512:].astype(f)], axis=1)[:, :d]
    if cos is not None:
        c, s = cos.numpy(), sin.numpy()
        a, b = row[:, d - 64::2].copy(), row[:, d - 63::2].copy()
        row[:, d - 64::2] = (a * c).astype(f) - (b * s).astype(f)
        row[:, d - 63::2] = (a * s).astype(f) + (b * c).astype(f)
    return O.f32_round_to_bf16(row)


def e2m1_encode(q):
    """Nearest E2M1 magnitude of |q| (fp64), ties to the even code, sign kept."""
    mags = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    d = np.abs(np.minimum(np.abs(q), 6.0)[..., None] - mags)
    best = d.min(-1, keepdims=True)
    near = d == best
    code = np.where(near[..., ::2].any(-1), 2 * near[..., ::2].argmax(-1), near.argmax(-1))
    return (code | np.where(np.signbit(q), 8, 0)).astype(np.uint8)


def ref_store(row, kv_format):
    """(bytes of the record, scale bytes or None, dequantised fp64 row)."""
    lat = row[:, :512]
    T = len(row)
    bf = lambda a: (np.ascontiguousarray(a, np.float32).view(np.uint32) >> 16).astype(np.uint16).view(np.uint8).reshape(T, -1)  # noqa: E731
    if kv_format == M.MLA_KV_BF16:
        return bf(row), None, row.astype(np.float64)
    if kv_format == M.MLA_KV_FP8_E4M3:
        t = lat.reshape(T, 4, 128)
        amax = np.abs(t).max(-1)
        sc = np.where(amax > 0, (amax * (np.float32(1) / np.float32(448))).astype(np.float32), np.float32(1))
        codes = O.e4m3_encode((t / sc[..., None]).astype(np.float32)).reshape(T, 512)
        rec = np.concatenate([codes, sc.astype(np.float32).view(np.uint8).reshape(T, 16), bf(row[:, 512:])], 1)
        return rec, None, O.dequant_fp8_records(_pad64(rec)).reshape(-1, 576)[:T]
    blk = lat.reshape(T, 32, 16)
    s8 = O.e4m3_encode((np.abs(blk).max(-1).astype(np.float32) * (np.float32(1) / np.float32(6))).astype(np.float32))
    s = O.e4m3_to_f64(s8)[..., None]
    q = np.where(s > 0, blk.astype(np.float64) / np.where(s > 0, s, 1), 0.0)
    codes = e2m1_encode(q).reshape(T, 512)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    val = O.dequant_nvfp4(packed, s8)
    if kv_format == M.MLA_KV_NVFP4:
        return packed, s8, val
    return (np.concatenate([packed, s8, bf(row[:, 512:])], 1), None,
            np.concatenate([val, row[:, 512:].astype(np.float64)], 1))


def _pad64(rec):
    n = -(-len(rec) // 64) * 64
    out = np.zeros((n, rec.shape[1]), np.uint8)
    out[:len(rec)] = rec
    return out.reshape(n // 64, 64, -1)


def new_cache(kv_format, pages, fill=0xA5):
    rec = {M.MLA_KV_BF16: 1152, M.MLA_KV_FP8_E4M3: 656, M.MLA_KV_NVFP4: 256, M.MLA_KV_FP4_E2M1: 416}[kv_format]
    c = torch.full((pages * 64, rec), fill, dtype=torch.uint8, device="cuda")
    s = torch.full((pages * 64, 32), fill, dtype=torch.uint8, device="cuda") if kv_format == M.MLA_KV_NVFP4 else None
    return c, s


FORMATS = [M.MLA_KV_BF16, M.MLA_KV_FP8_E4M3, M.MLA_KV_NVFP4, M.MLA_KV_FP4_E2M1]


def rows_input(T, d, seed, stride=None):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, stride or d)) * np.exp(rng.uniform(-6, 6, size=(T, 1)))
    x[:, ::37] *= 30                                     # outliers
    if T > 3:
        x[1], x[2, :300] = 0, 0                          # a zero row, zero blocks
        x[3, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -0.0]   # ties
    th = rng.uniform(-1000, 1000, size=(T, 32))
    return (torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16), torch.from_numpy(np.cos(th).astype(np.float32)),
            torch.from_numpy(np.sin(th).astype(np.float32)), W.norm_weight(512, seed))


@pytest.mark.parametrize("kv_format", FORMATS)
@pytest.mark.parametrize("norm,rope", [(True, True), (False, False), (False, True), (True, False)])
@pytest.mark.parametrize("T,extra", [(1, 0), (7, 8), (1000, 1536)])
def test_append_bytes(kv_format, norm, rope, T, extra):
    d = 512 if kv_format == M.MLA_KV_NVFP4 else 576
    kv, cos, sin, gamma = rows_input(T, d, T + extra, d + extra)
    pages = T // 64 + 3
    rng = np.random.default_rng(T)
    slots = rng.permutation(pages * 64)[:T]
    if T > 5:
        slots[[2, T - 1]] = -1
    cache, cs = new_cache(kv_format, pages)
    before = cache.cpu().numpy().copy()
    out = torch.full((T, d), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dv = lambda t, on=True: t.cuda() if on else None  # noqa: E731
    M.mla_kv_append(kv.cuda(), d + extra, T, d, dv(gamma, norm), 1e-5, dv(cos, rope), dv(sin, rope),
                    torch.from_numpy(slots.astype(np.int32)).cuda(), cache, cs, kv_format, pages, out, st)
    torch.cuda.synchronize()
    row = ref_rows(kv[:, :d], gamma if norm else None, 1e-5, cos if rope else None, sin if rope else None, d)
    rec, s8, val = ref_store(row, kv_format)
    live = slots >= 0
    want = before.copy()
    want[slots[live]] = rec[live]
    got = cache.cpu().numpy()
    assert np.array_equal(got, want)                                     # every byte, also of the slots not named
    if cs is not None:
        ws = np.full((pages * 64, 32), 0xA5, np.uint8)
        ws[slots[live]] = s8[live]
        assert np.array_equal(cs.cpu().numpy(), ws)
    vo = O.torch_bf16_to_f64(out.cpu())
    assert np.array_equal(vo[live], val[live]) and np.all(vo[~live] == 3.0)
    assert int(st.item()) == 0
    # and the stored values against the 64-bit chain: half a bf16 step (2^-8), half an e4m3 step (2^-4) or, for
    # E2M1, half its largest step (1.0 scale; a saturated value is nearer), plus what a zero scale drops (6 * 2^-10);
    # the fp32 chain adds a few 2^-24 of the row's largest value
    y = O.rms_norm(O.torch_bf16_to_f64(kv[:, :512]), gamma.numpy(), np.float32(1e-5)) if norm else O.torch_bf16_to_f64(kv[:, :512])
    full = y if d == 512 else np.concatenate([y, O.torch_bf16_to_f64(kv[:, 512:576])], 1)
    if rope:
        full[:, d - 64:] = O.rope_rotate(full[:, d - 64:], cos.numpy(), sin.numpy())
    err = np.abs(val - full)
    base = 2.0 ** -8 * np.abs(full) + 2.0 ** -20 * np.abs(full).max(1, keepdims=True)
    if kv_format == M.MLA_KV_FP8_E4M3:
        sc = np.repeat(rec[:, 512:528].copy().view(np.float32), 128, axis=1)
        base[:, :512] += 2.0 ** -4 * np.abs(full[:, :512]) + 2.0 ** -10 * sc + 2.0 ** -8 * np.abs(full[:, :512])
    elif kv_format != M.MLA_KV_BF16:
        sc = O.ue4m3_to_f64(s8 if s8 is not None else rec[:, 256:288])
        base[:, :512] += np.repeat(sc, 16, axis=1) + 6 * 2.0 ** -10
    big = np.repeat(np.abs(full[:, :512]).reshape(T, 32, 16).max(-1), 16, axis=1) > 6 * 448   # the scale saturates
    ok = err <= base
    if kv_format in (M.MLA_KV_NVFP4, M.MLA_KV_FP4_E2M1):
        ok[:, :512] |= big
    assert ok.all(), np.max(err - base)


@pytest.mark.parametrize("kv_format", FORMATS)
def test_append_bad_slots(kv_format):
    d = 512 if kv_format == M.MLA_KV_NVFP4 else 576
    kv, cos, sin, gamma = rows_input(6, d, 5)
    cache, cs = new_cache(kv_format, 2)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([128, -2, -1, 2147483647, -2147483648, 127], dtype=torch.int32, device="cuda")
    M.mla_kv_append(kv.cuda(), d, 6, d, gamma.cuda(), 1e-6, cos.cuda(), sin.cuda(), slots, cache, cs, kv_format, 2, None, st)
    torch.cuda.synchronize()
    assert int(st.item()) == M.MLA_DEVICE_STATUS_BOUNDS
    got = cache.cpu().numpy()
    assert np.all(got[:127] == 0xA5) and not np.all(got[127] == 0xA5)


def test_append_nan_rows_without_a_slot():
    kv = torch.full((3, 576), float("nan"), dtype=torch.bfloat16)
    kv[1] = 1.0
    cache, _ = new_cache(M.MLA_KV_FP4_E2M1, 1)
    M.mla_kv_append(kv.cuda(), 576, 3, 576, None, 0.0, None, None, torch.tensor([-1, 5, -1], dtype=torch.int32).cuda(), cache,
                    None, M.MLA_KV_FP4_E2M1, 1)
    torch.cuda.synchronize()
    got = cache.cpu().numpy()
    assert np.all(got[np.arange(64) != 5] == 0xA5)
    assert np.array_equal(got[5, 288:].view(np.uint16), np.full(64, 0x3F80, np.uint16))


def test_append_values_in_place():
    kv, cos, sin, gamma = rows_input(70, 576, 9)
    cache, _ = new_cache(M.MLA_KV_FP8_E4M3, 2)
    c2, _ = new_cache(M.MLA_KV_FP8_E4M3, 2)
    slots = torch.arange(70, dtype=torch.int32, device="cuda")
    a, b = kv.cuda(), torch.empty(70, 576, dtype=torch.bfloat16, device="cuda")
    M.mla_kv_append(a, 576, 70, 576, gamma.cuda(), 1e-6, cos.cuda(), sin.cuda(), slots, cache, None, M.MLA_KV_FP8_E4M3, 2, b)
    M.mla_kv_append(a, 576, 70, 576, gamma.cuda(), 1e-6, cos.cuda(), sin.cuda(), slots, c2, None, M.MLA_KV_FP8_E4M3, 2, a)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(cache, c2)


# -------------------------------------------------------------------------- together
@pytest.mark.parametrize("h_q", [16, 128])
@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(h_q, graph):
    """A prefill step and decode steps on another stream: tables, rows, decode.
    Every step's output is checked against the oracle over the values that the
    cache was said to hold. With `graph`, the decode step is captured once and
    replayed, its lengths and free list carried along by device copies."""
    B, steps, stride, pages = 3, 4, 8, 20
    rng = np.random.default_rng(h_q)
    dev = dict(dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
    rngd = torch.tensor([0, pages], **dev)
    ctx, new = torch.zeros(B, **dev), torch.tensor([100, 0, 63], **dev)
    bt = torch.full((B, stride), -1, **dev)
    cache = torch.zeros(pages, 64, 416, dtype=torch.uint8, device="cuda")
    lens, start, nxt = torch.zeros(B, **dev), torch.zeros(B + 1, **dev), torch.zeros(1, **dev)
    gamma = W.norm_weight(512, 3).cuda()
    status = torch.zeros(1, **dev)
    side = torch.cuda.Stream()
    history = [np.zeros((0, 576)) for _ in range(B)]

    def fill(T, kv, cos, sin, slots, pos, vals):
        M.mla_extend_tables(ctx, new, B, free, rngd, pages, bt, stride, lens, start, slots, pos, T, nxt, status)
        M.mla_kv_append(kv, 576, T, 576, gamma, 1e-6, cos, sin, slots, cache, None, M.MLA_KV_FP4_E2M1, pages, vals, status)

    def carry():
        ctx.copy_(lens)
        rngd[0:1].copy_(nxt)

    def rows(T, seed):
        kv, cos, sin, _ = rows_input(T, 576, seed)
        kv[:, 512:] = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, 64))).to(torch.bfloat16)
        return kv.cuda(), cos.cuda(), sin.cuda()

    def remember(vals, count):
        v = O.torch_bf16_to_f64(vals.cpu())
        at = 0
        for b in range(B):
            history[b] = np.concatenate([history[b], v[at:at + count[b]]])
            at += count[b]

    T0 = 170
    kv, cos, sin = rows(T0, 11)
    slots, pos = torch.zeros(T0, **dev), torch.zeros(T0, **dev)
    vals = torch.zeros(T0, 576, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        fill(T0, kv, cos, sin, slots, pos, vals)
        carry()
    torch.cuda.synchronize()
    assert lens.tolist() == [100, 0, 63] and int(nxt) == 3 and int(status) == 0
    remember(vals, [100, 0, 63])
    new.fill_(1)
    q = torch.zeros(B, 1, h_q, 576, dtype=torch.bfloat16, device="cuda")
    r = M.DecodeRunner(q, cache, bt, lens, softmax_scale=576 ** -0.5)
    kv, cos, sin = rows(B, 12)
    slots, pos = torch.zeros(B, **dev), torch.zeros(B, **dev)
    vals = torch.zeros(B, 576, dtype=torch.bfloat16, device="cuda")

    def step():
        fill(B, kv, cos, sin, slots, pos, vals)
        r.plan()
        r.run()
        carry()

    torch.cuda.synchronize()
    g = None
    if graph:
        keep = [t.clone() for t in (ctx, rngd, bt, cache)]
        with torch.cuda.stream(side):
            step()                                    # warm-up, undone below
        torch.cuda.synchronize()
        for t, k in zip((ctx, rngd, bt, cache), keep):
            t.copy_(k)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    for i in range(steps):
        a, b, c = rows(B, 20 + i)
        kv.copy_(a), cos.copy_(b), sin.copy_(c)
        q.copy_(torch.from_numpy(rng.standard_normal((B, 1, h_q, 576)).astype(np.float32)).to(torch.bfloat16))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay() if graph else step()
        torch.cuda.synchronize()
        remember(vals, [1, 1, 1])
        assert lens.tolist() == [len(h) for h in history] and pos.tolist() == [len(h) - 1 for h in history]
        assert r.status(side)[0] == M.MLA_OK and int(status) == 0
        out, lse = r.out.float().cpu().numpy(), r.lse.cpu().numpy()
        qf = O.torch_bf16_to_f64(q.cpu())
        for b in range(B):
            o, l = O.attend(qf[b, 0], history[b], 576 ** -0.5)
            # bf16 probabilities and output: 2^-8 of the largest value and of the result; lse as in gpu_helpers
            bound = 2.0 ** -8 * (np.abs(o) + 1.01 * np.abs(history[b][:, :512]).max()) + 1e-4
            assert np.all(np.abs(out[b, 0] - o) <= bound)
            assert np.all(np.abs(lse[b, 0] - l) <= G.LSE_ATOL * np.maximum(1.0, np.abs(l)))
    # the cache holds what the rows said
    full = O.dequant_fp4_records(cache.cpu().numpy())
    for b in range(B):
        got = O.gather_rows(full, bt[b].cpu().numpy(), np.arange(len(history[b])))
        assert np.array_equal(got, history[b])


def test_two_streams_at_once():
    """Two independent steps on two streams, each with its own buffers."""
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    inputs = []
    for i in range(2):
        kv, cos, sin, gamma = rows_input(3000, 576, 40 + i)
        cache, _ = new_cache(M.MLA_KV_FP4_E2M1, 50)
        inputs.append((kv.cuda(), cos.cuda(), sin.cuda(), gamma.cuda(), torch.randperm(3200)[:3000].int().cuda(), cache))
    torch.cuda.synchronize()
    for rep in range(5):
        for i in range(2):
            kv, cos, sin, gamma, slots, cache = inputs[i]
            M.mla_kv_append(kv, 576, 3000, 576, gamma, 1e-6, cos, sin, slots, cache, None, M.MLA_KV_FP4_E2M1, 50,
                            stream=streams[i])
    torch.cuda.synchronize()
    for kv, cos, sin, gamma, slots, cache in inputs:
        c2, _ = new_cache(M.MLA_KV_FP4_E2M1, 50)
        M.mla_kv_append(kv, 576, 3000, 576, gamma, 1e-6, cos, sin, slots, c2, None, M.MLA_KV_FP4_E2M1, 50)
        torch.cuda.synchronize()
        outs.append(torch.equal(cache, c2))
    assert outs == [True, True]
