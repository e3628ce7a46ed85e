"""Serving operators around a 4-bit latent cache, as measured cases: block
tables and slot maps built from request lengths, the cache append (norm, RoPE,
quantisation and scatter), and paged or token-sparse decoding over E2M1
records. Each case runs either in plain torch operations (`own` false) or
through the library's entry points (`own` true), on the same prepared inputs.
"""
import random

import numpy as np
import torch

own = False

PAGE = 64
D_LAT, D_ROPE, D_QK = 512, 64, 576
FP8_REC = 656      # 512 e4m3 codes | 4 fp32 scales | 64 bf16 RoPE dims
FP4_REC = 416      # 256 bytes of E2M1 pairs | 32 UE4M3 scales | 64 bf16 RoPE dims
EPS = float(np.float32(1e-6))
SCALE = D_QK ** -0.5
ROW_BYTES = {"bf16": 1152, "fp8": FP8_REC, "nvfp4": 288, "fp4": FP4_REC}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step of the two-token batch: 128 requests of very different lengths add two tokens each
        dict(name="tables step 128", op="tables", batch=128, lo=1024, hi=16384, new_lo=2, new_hi=2, max_tokens=256, stride=1025, short=False),
        # a large serving batch, some requests idle this step, the token axis padded to a captured size
        dict(name="tables step 4096", op="tables", batch=4096, lo=0, hi=4000, new_lo=0, new_hi=1, max_tokens=4096, stride=65, short=False),
        # mixed chunked prefill whose free list runs out on the way: the last requests are refused
        dict(name="tables prefill 64", op="tables", batch=64, lo=0, hi=6000, new_lo=0, new_hi=2048, max_tokens=131072, stride=256, short=True),
        # the two-token batch's 256 new rows into the 4-bit cache
        dict(name="append fp4 256", op="append", kv="fp4", tokens=256, pad=0, stride=576, norm=True, pages=512),
        # a prefill chunk into the 4-bit cache, rows cut out of a wider projection output
        dict(name="append fp4 32768", op="append", kv="fp4", tokens=32768, pad=37, stride=640, norm=True, pages=1024),
        # a ragged prefill chunk into FP8 records, already normalised
        dict(name="append fp8 5003", op="append", kv="fp8", tokens=5003, pad=117, stride=576, norm=False, pages=300),
        # 512-value NVFP4 rows of six query tokens x 64 requests
        dict(name="append nvfp4 384", op="append", kv="nvfp4", tokens=384, pad=0, stride=512, norm=True, pages=600),
        # two short requests with 16 heads: launch latency
        dict(name="decode 2x16 short", op="decode", batch=2, heads=16, s_q=1, causal=False, lo=70, hi=129, topk=0, sink=False),
        # 128 heads, 64 equal requests of 4096 tokens: the headline batch
        dict(name="decode 64x128 4096", op="decode", batch=64, heads=128, s_q=1, causal=False, lo=4096, hi=4096, topk=0, sink=False),
        # 64 heads, 64 requests of 8192 tokens
        dict(name="decode 64x64 8192", op="decode", batch=64, heads=64, s_q=1, causal=False, lo=8192, hi=8192, topk=0, sink=False),
        # two causal query tokens, 16 heads, ragged lengths, per-head sink
        dict(name="decode 128x16 ragged", op="decode", batch=128, heads=16, s_q=2, causal=True, lo=1024, hi=16384, topk=0, sink=True),
        # token-sparse: 2048 of up to 32768 tokens for each of 32 requests, 128 heads
        dict(name="decode 32x128 topk", op="decode", batch=32, heads=128, s_q=1, causal=False, lo=32768, hi=32768, topk=2048, sink=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "decode"])
    if op == "tables":
        batch = _log_int(rng, 1, 4096)
        hi = _log_int(rng, 64, 16384)
        new_hi = _log_int(rng, 1, max(1, min(8192, 131072 // batch)))
        new_lo = rng.choice([0, 1, new_hi])
        total = batch * (new_lo + new_hi) // 2
        return dict(op=op, batch=batch, lo=rng.choice([0, hi // 2]), hi=hi, new_lo=new_lo, new_hi=new_hi,
                    max_tokens=max(16, min(131072, total + batch + rng.randrange(64))),
                    stride=(hi + new_hi) // PAGE + 1 + rng.randrange(8), short=rng.random() < 0.3)
    if op == "append":
        kv = rng.choice(["fp4", "fp4", "fp8", "nvfp4", "bf16"])
        tokens = _log_int(rng, 1, 32768)
        d = D_LAT if kv == "nvfp4" else D_QK
        return dict(op=op, kv=kv, tokens=tokens, pad=rng.randrange(0, 1 + tokens // 4), stride=d + 8 * rng.choice([0, 0, 1, 8, 192]),
                    norm=rng.random() < 0.7, pages=-(-tokens // PAGE) + rng.randrange(1, 64))
    heads = rng.choice([1, 5, 8, 16, 20, 32, 48, 64, 96, 128])
    s_q = rng.choice([1, 1, 2, 3, 6])
    topk = rng.choice([0, 0, 64 * _log_int(rng, 1, 32)])
    hi = _log_int(rng, 1, 16384)
    batch = max(1, min(_log_int(rng, 1, 128), (1 << 28) // (hi * heads * s_q), 524288 // hi, (1 << 17) // (s_q * max(topk, 64))))
    return dict(op=op, batch=batch, heads=heads, s_q=s_q, causal=topk == 0 and rng.random() < 0.6,
                lo=rng.choice([0, hi // 2, hi]), hi=hi, topk=topk, sink=rng.random() < 0.3)


def _ints(case, what, n, lo, hi):
    """n whole numbers of [lo, hi], the same for every seed of a case; with lo = 0, the first is 0."""
    r = np.random.RandomState((hash_of(what) + 31 * n + 17 * lo + 7 * hi) % (1 << 31))
    v = r.randint(lo, hi + 1, size=n).astype(np.int64)
    if lo == 0 and n > 1:
        v[0] = 0
    return v


def hash_of(text):
    return sum((i + 1) * ord(c) for i, c in enumerate(text))


def _lens(case):
    return _ints(case, "lens", case["batch"], case["lo"], case["hi"])


def _new(case):
    return _ints(case, "new", case["batch"], case["new_lo"], case["new_hi"])


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
_MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)            # between neighbouring E2M1 magnitudes
_MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _fp4_quantise(x):
    """fp32 [..., 16n] -> packed E2M1 bytes [..., 8n], UE4M3 scale bytes [..., n] and the values that they stand for."""
    blk = x.reshape(*x.shape[:-1], -1, 16)
    s8 = (blk.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    q = torch.where(s > 0, blk / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(blk))
    a = q.abs()
    # nearest magnitude, ties to the even code
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8) +
           (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    code = mag | (torch.signbit(q).to(torch.uint8) << 3)
    val = (torch.tensor(_MAGS, device=x.device)[mag.int()] * torch.where(torch.signbit(q), -s, s)).reshape(x.shape)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8), val


def _angles(positions):
    inv = 10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32.0)
    a = positions.double()[:, None] * inv
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "tables":
        return _prepare_tables(case, g, s)
    if case["op"] == "append":
        return _prepare_append(case, g, s)
    return _prepare_decode(case, g, s)


def _prepare_tables(case, g, s):
    B, stride = case["batch"], case["stride"]
    ctx, new = _lens(case), _new(case)
    have = (ctx + PAGE - 1) // PAGE
    need = int(((ctx + new + PAGE - 1) // PAGE - have).sum())
    P = int(have.sum()) + need + 64
    perm = torch.randperm(P, generator=g, device="cuda").int()
    j = torch.arange(stride, device="cuda")[None, :]
    have_t = torch.from_numpy(have).cuda()
    off = torch.cumsum(have_t, 0) - have_t
    at = (off[:, None] + j).clamp(max=P - 1)
    s["block_table"] = torch.where(j < have_t[:, None], perm[at], torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()
    s["free_pages"] = perm[int(have.sum()):].contiguous()
    s["free_range"] = torch.tensor([3, 3 + (need * 2 // 3 if case["short"] else need + 7)], dtype=torch.int32, device="cuda")
    s["context_lens"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
    s["new_lens"] = torch.from_numpy(new.astype(np.int32)).cuda()
    s["num_pages"] = P
    out = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    s["seqlens"], s["token_start"], s["free_next"] = out(B), out(B + 1), out(1)
    s["slots"], s["positions"] = out(case["max_tokens"]), out(case["max_tokens"])
    return s


def _prepare_append(case, g, s):
    T, kv, P = case["tokens"], case["kv"], case["pages"]
    d = D_LAT if kv == "nvfp4" else D_QK
    wide = torch.randn(T, case["stride"], generator=g, device="cuda")
    s["kv"] = (wide * torch.rand(T, 1, generator=g, device="cuda").mul_(3)).bfloat16()[:, :d]
    s["gamma"] = torch.rand(D_LAT, generator=g, device="cuda") + 0.5 if case["norm"] else None
    s["cos"], s["sin"] = _angles(torch.randint(0, 131072, (T,), generator=g, device="cuda"))
    slots = torch.randperm(P * PAGE, generator=g, device="cuda")[:T].int()
    if case["pad"]:
        slots[T - case["pad"]:] = -1
    s["slots"] = slots
    # one page more than the cache has, for the plain form's rows without a slot
    if kv == "bf16":
        s["buffer"] = torch.zeros((P + 1) * PAGE, D_QK, dtype=torch.bfloat16, device="cuda")
        s["cache"], s["cache_scale"] = s["buffer"][:P * PAGE].view(P, PAGE, 1, D_QK), None
    elif kv == "nvfp4":
        s["buffer"] = torch.zeros((P + 1) * PAGE, 256, dtype=torch.uint8, device="cuda")
        s["buffer_scale"] = torch.zeros((P + 1) * PAGE, 32, dtype=torch.uint8, device="cuda")
        s["cache"], s["cache_scale"] = s["buffer"][:P * PAGE].view(P, PAGE, 256), s["buffer_scale"][:P * PAGE].view(P, PAGE, 32)
    else:
        rec = FP4_REC if kv == "fp4" else FP8_REC
        s["buffer"] = torch.zeros((P + 1) * PAGE, rec, dtype=torch.uint8, device="cuda")
        s["cache"], s["cache_scale"] = s["buffer"][:P * PAGE].view(P, PAGE, rec), None
    s["values"] = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_decode(case, g, s):
    B, h, s_q = case["batch"], case["heads"], case["s_q"]
    lens = _lens(case)
    have = (lens + PAGE - 1) // PAGE
    P = int(have.sum()) + 1
    q = torch.randn(B, s_q, h, D_QK, generator=g, device="cuda").bfloat16()
    cache = torch.empty(P, PAGE, FP4_REC, dtype=torch.uint8, device="cuda")
    for p0 in range(0, P, 1024):  # filled by parts: the fp32 source is not held whole
        part = cache[p0:p0 + 1024]
        codes, sc, _ = _fp4_quantise(torch.randn(part.shape[0], PAGE, D_LAT, generator=g, device="cuda").bfloat16().float())
        part[..., :256], part[..., 256:288] = codes, sc
        rope = torch.randn(part.shape[0], PAGE, D_ROPE, generator=g, device="cuda").bfloat16()
        part[..., 288:] = rope.view(torch.uint8)
    perm = torch.randperm(P, generator=g, device="cuda").int()
    stride = max(1, int(have.max()))
    j = torch.arange(stride, device="cuda")[None, :]
    have_t = torch.from_numpy(have).cuda()
    off = torch.cumsum(have_t, 0) - have_t
    bt = torch.where(j < have_t[:, None], perm[(off[:, None] + j).clamp(max=P - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    s["q"], s["cache"], s["block_table"] = q, cache, bt.contiguous()
    s["cache_seqlens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    s["sink"] = torch.randn(h, generator=g, device="cuda") + 1 if case["sink"] else None
    s["indices"] = None
    if case["topk"]:
        u = torch.rand(B, s_q, case["topk"], generator=g, device="cuda")
        idx = (u * s["cache_seqlens"][:, None, None]).int()
        idx = torch.minimum(idx, (s["cache_seqlens"] - 1).clamp(min=0)[:, None, None])
        drop = (torch.rand(B, s_q, case["topk"], generator=g, device="cuda") < 0.05) | (s["cache_seqlens"] == 0)[:, None, None]
        s["indices"] = torch.where(drop, torch.full((), -1, dtype=torch.int32, device="cuda"), idx).contiguous()
    if own:
        import head_latent_attention_get_b200 as M
        s["runner"] = M.DecodeRunner(q, cache, s["block_table"], s["cache_seqlens"], softmax_scale=SCALE, causal=case["causal"],
                                     indices=s["indices"], sink=s["sink"])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if op == "tables":
        return _own_tables(s) if own else _plain_tables(s)
    if op == "append":
        return _own_append(s) if own else _plain_append(s)
    return _own_decode(s) if own else _plain_decode(s)


def _own_tables(s):
    import head_latent_attention_get_b200 as M
    c = s["case"]
    M.mla_extend_tables(s["context_lens"], s["new_lens"], c["batch"], s["free_pages"], s["free_range"], s["num_pages"], s["block_table"],
                        c["stride"], s["seqlens"], s["token_start"], s["slots"], s["positions"], c["max_tokens"], s["free_next"])
    return _tables_out(s)


def _tables_out(s):
    return {k: s[k] for k in ("block_table", "seqlens", "token_start", "slots", "positions", "free_next")}


def _plain_tables(s):
    c = s["case"]
    ctx, new, stride = s["context_lens"].long(), s["new_lens"].long(), c["stride"]
    start = torch.cumsum(new.clamp(min=0), 0) - new.clamp(min=0)
    end = start + new.clamp(min=0)
    ok = (ctx >= 0) & (new >= 0) & (ctx + new <= stride * PAGE) & (end <= c["max_tokens"])
    have = (ctx + PAGE - 1) // PAGE
    need = torch.where(ok, (ctx + new + PAGE - 1) // PAGE - have, torch.zeros_like(ctx))
    upto = torch.cumsum(need, 0)
    first, avail = s["free_range"][0].long(), (s["free_range"][1] - s["free_range"][0]).long()
    ok = ok & ((need == 0) | (upto <= avail))
    base = first + upto - need - have          # free-list place of page j of request b: base[b] + j
    total = torch.where(ok, ctx + new, ctx.clamp(min=0))
    s["seqlens"].copy_(total)
    s["token_start"][:-1].copy_(start)
    s["token_start"][-1:].copy_(end[-1:])
    s["free_next"].copy_((first + torch.where(ok & (need > 0), upto, torch.zeros_like(upto)).max()).reshape(1))
    last = s["free_pages"].numel() - 1
    j = torch.arange(stride, device="cuda")[None, :]
    fresh = ok[:, None] & (j >= have[:, None]) & (j < ((total + PAGE - 1) // PAGE)[:, None])
    s["block_table"].copy_(torch.where(fresh, s["free_pages"][(base[:, None] + j).clamp(0, last)], s["block_table"]))
    t = torch.arange(c["max_tokens"], device="cuda")
    b = torch.searchsorted(end, t, right=True)
    live = b < c["batch"]
    b = b.clamp(max=c["batch"] - 1)
    live = live & ok[b]
    pos = ctx[b] + t - start[b]
    page = s["block_table"][b, (pos // PAGE).clamp(0, stride - 1)]
    s["slots"].copy_(torch.where(live, page * PAGE + (pos % PAGE), torch.full_like(pos, -1)))
    s["positions"].copy_(torch.where(live, pos, torch.full_like(pos, -1)))
    return _tables_out(s)


def _own_append(s):
    import head_latent_attention_get_b200 as M
    c = s["case"]
    fmt = {"bf16": M.MLA_KV_BF16, "fp8": M.MLA_KV_FP8_E4M3, "nvfp4": M.MLA_KV_NVFP4, "fp4": M.MLA_KV_FP4_E2M1}[c["kv"]]
    M.mla_kv_append(s["kv"], c["stride"], c["tokens"], s["kv"].shape[1], s["gamma"], EPS, s["cos"], s["sin"], s["slots"], s["cache"],
                    s["cache_scale"], fmt, c["pages"], s["values"])
    return _append_out(s)


def _append_out(s):
    out = {"values": s["values"], "cache": s["cache"]}
    if s["cache_scale"] is not None:
        out["cache_scale"] = s["cache_scale"]
    return out


def _rotate(x, cos, sin):
    x0, x1 = x[:, 0::2], x[:, 1::2]
    return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).reshape(x.shape)


def _plain_append(s):
    c, kv = s["case"], s["kv"]
    T, fmt = c["tokens"], c["kv"]
    y = kv[:, :D_LAT].float()
    if s["gamma"] is not None:  # the mean of squares in 64 bits: the quantiser's decisions hang on the last bit of its result
        r = (1.0 / torch.sqrt(kv[:, :D_LAT].double().square().sum(-1, keepdim=True) / D_LAT + EPS)).float()
        y = y * r * s["gamma"]
    if fmt == "nvfp4":
        y = torch.cat([y[:, :D_LAT - D_ROPE], _rotate(y[:, D_LAT - D_ROPE:], s["cos"], s["sin"])], 1)
    lat = y.bfloat16()
    slot = s["slots"].long()
    to = torch.where(slot >= 0, slot, c["pages"] * PAGE)
    if fmt == "nvfp4":
        codes, sc, val = _fp4_quantise(lat.float())
        s["buffer"][to], s["buffer_scale"][to] = codes, sc
        row = val.bfloat16()
    else:
        rope = _rotate(kv[:, D_LAT:].float(), s["cos"], s["sin"]).bfloat16()
        if fmt == "bf16":
            row = torch.cat([lat, rope], 1)
            s["buffer"][to] = row
        elif fmt == "fp4":
            codes, sc, val = _fp4_quantise(lat.float())
            s["buffer"][to] = torch.cat([codes, sc, rope.view(torch.uint8)], 1)
            row = torch.cat([val.bfloat16(), rope], 1)
        else:
            t = lat.float().view(T, 4, 128)
            amax = t.abs().amax(-1)
            sc = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
            codes = (t / sc[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            s["buffer"][to] = torch.cat([codes.view(torch.uint8).view(T, D_LAT), sc.view(torch.uint8).view(T, 16), rope.view(torch.uint8)], 1)
            row = torch.cat([(codes.float() * sc[..., None]).view(T, D_LAT).bfloat16(), rope], 1)
    s["values"].copy_(torch.where(slot[:, None] >= 0, row, s["values"]))
    return _append_out(s)


def _own_decode(s):
    s["runner"].plan()
    out, lse = s["runner"].run()
    return {"out": out, "lse": lse}


def _pairs(device):
    """[256, 2]: the two E2M1 values of a byte, low nibble first."""
    v = torch.tensor(_MAGS + tuple(-m for m in _MAGS), device=device)
    b = torch.arange(256, device=device)
    return torch.stack([v[b & 15], v[b >> 4]], -1)


def _rows(s, page, at):
    """fp32 [..., 576] cache rows of (page, token in the page)."""
    rec = s["cache"][page, at]
    codes = _pairs(rec.device)[rec[..., :256].int()].flatten(-2)
    sc = rec[..., 256:288].contiguous().view(torch.float8_e4m3fn).float()
    lat = (codes.unflatten(-1, (32, 16)) * sc[..., None]).flatten(-2)
    return torch.cat([lat, rec[..., 288:].contiguous().view(torch.bfloat16).float()], -1)


def _plain_decode(s):
    c = s["case"]
    B, s_q, h, lens, bt = c["batch"], c["s_q"], c["heads"], s["cache_seqlens"].long(), s["block_table"].long()
    q = s["q"].float()
    if c["topk"]:
        idx = s["indices"].long()
        keep = (idx >= 0) & (idx < lens[:, None, None])
        t = torch.where(keep, idx, torch.zeros_like(idx))
        page = bt[torch.arange(B, device="cuda")[:, None, None], t // PAGE].clamp(min=0)
        k = _rows(s, page, t % PAGE)                                     # [B, s_q, topk, 576]
        sc = torch.matmul(q, k.transpose(-1, -2)) * SCALE                # [B, s_q, h, topk]
        keep = keep[:, :, None, :]
    else:
        n = bt.shape[1] * PAGE
        t = torch.arange(n, device="cuda")
        page = bt[:, t // PAGE].clamp(min=0)
        k = _rows(s, page, (t % PAGE).expand(B, n))[:, None]             # [B, 1, n, 576]
        sc = torch.matmul(q.view(B, 1, s_q * h, D_QK), k.transpose(-1, -2)).view(B, s_q, h, n) * SCALE
        limit = lens[:, None].expand(B, s_q)
        if c["causal"]:
            limit = limit - s_q + torch.arange(1, s_q + 1, device="cuda")
        keep = (t < limit[..., None])[:, :, None, :]
    sc = torch.where(keep, sc, torch.full((), -float("inf"), device="cuda"))
    m = sc.amax(-1, keepdim=True)
    if s["sink"] is not None:
        m = torch.maximum(m, s["sink"][None, None, :, None])
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(sc - m0)
    l = e.sum(-1, keepdim=True)
    if s["sink"] is not None:
        l = l + torch.exp(s["sink"][None, None, :, None] - m0)
    v = k[..., :D_LAT]
    acc = torch.matmul(e, v) if c["topk"] else torch.matmul(e.view(B, 1, s_q * h, -1), v).view(B, s_q, h, D_LAT)
    out = torch.where(l > 0, acc / torch.where(l > 0, l, torch.ones_like(l)), torch.zeros_like(acc))
    return {"out": out.bfloat16(), "lse": (m0 + torch.log(l)).squeeze(-1)}


# --------------------------------------------------------------------------
# the least a pass has to move and compute, and its 64-bit value
# --------------------------------------------------------------------------
def work(case):
    if case["op"] == "tables":
        ctx, new = _lens(case), _new(case)
        fresh = int(((ctx + new + PAGE - 1) // PAGE - (ctx + PAGE - 1) // PAGE).sum())
        if case["short"]:
            fresh = fresh * 2 // 3
        partial = int(((ctx % PAGE > 0) & (new > 0)).sum())   # entries read: the page that a request's first new token goes on in
        return {"bytes": 16 * case["batch"] + 8 * case["max_tokens"] + 8 * fresh + 4 * partial, "flops": 0}
    if case["op"] == "append":
        T, live = case["tokens"], case["tokens"] - case["pad"]
        d = D_LAT if case["kv"] == "nvfp4" else D_QK
        return {"bytes": 4 * T + live * (2 * d + 256 + ROW_BYTES[case["kv"]] + 2 * d) + (4 * D_LAT if case["norm"] else 0), "flops": 0}
    B, h, s_q, lens = case["batch"], case["heads"], case["s_q"], _lens(case)
    if case["topk"]:
        keys = int((lens > 0).sum()) * s_q * 0.95 * case["topk"]
        seen = float(sum(n * (1 - (1 - 1 / n) ** (0.95 * case["topk"] * s_q)) for n in lens.tolist() if n))   # distinct tokens expected
        tables = 4 * B * s_q * case["topk"] + 4 * keys
    else:
        i = np.arange(s_q)
        limit = lens[:, None] - s_q + 1 + i if case["causal"] else np.repeat(lens[:, None], s_q, 1)
        keys = float(np.clip(limit, 0, None).sum())
        seen = float(lens.sum())
        tables = 4 * int(((lens + PAGE - 1) // PAGE).sum())
    rows = B * s_q * h
    return {"bytes": seen * FP4_REC + rows * (2 * D_QK + 2 * D_LAT + 4) + tables + 4 * B, "flops": 2.0 * keys * h * (D_QK + D_LAT)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_decode(s)


def _nearest(x, grid):
    """The nearest of the ascending values `grid`, ties to the one with the even place; 64 bits."""
    g = torch.tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(g, x.contiguous()).clamp(1, len(grid) - 1)
    down, up = x - g[hi - 1], g[hi] - x
    take = torch.where((down < up) | ((down == up) & (hi % 2 == 1)), hi - 1, hi)
    return g[take]


_E4M3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _exact_append(s):
    c, x = s["case"], s["kv"].double()
    fmt = c["kv"]
    lat = x[:, :D_LAT]
    if s["gamma"] is not None:
        lat = lat / torch.sqrt((lat ** 2).mean(1, keepdim=True) + EPS) * s["gamma"].double()
    turn = torch.complex(s["cos"].double(), s["sin"].double())
    old = lat[:, D_LAT - D_ROPE:] if fmt == "nvfp4" else x[:, D_LAT:]
    new = torch.view_as_real(torch.view_as_complex(old.reshape(-1, 32, 2).contiguous()) * turn).reshape(-1, D_ROPE)
    if fmt == "nvfp4":
        lat = torch.cat([lat[:, :D_LAT - D_ROPE], new], 1)
    if fmt != "bf16":  # rows are rounded to bf16 before they are quantised
        lat = lat.bfloat16().double()
    if fmt in ("fp4", "nvfp4"):
        b = lat.view(-1, 32, 16)
        sc = _nearest((b.abs().amax(-1) / 6).clamp(max=448.0), _E4M3)[..., None]
        one = torch.where(sc > 0, sc, torch.ones_like(sc))
        lat = (torch.sign(b) * _nearest((b.abs() / one).clamp(max=6.0), _MAGS) * sc).view(-1, D_LAT)
    elif fmt == "fp8":
        b = lat.view(-1, 4, 128)
        top = b.abs().amax(-1, keepdim=True)
        sc = torch.where(top > 0, (top / 448).float().double(), torch.ones_like(top))
        lat = (torch.sign(b) * _nearest((b.abs() / sc).float().double().clamp(max=448.0), _E4M3) * sc).view(-1, D_LAT)
    row = lat if fmt == "nvfp4" else torch.cat([lat, new], 1)
    out = {"values": torch.where(s["slots"][:, None] >= 0, row, torch.zeros_like(row)), "cache": None}
    if fmt == "nvfp4":
        out["cache_scale"] = None
    return out


def _exact_decode(s):
    c = s["case"]
    mags = torch.tensor(_MAGS, dtype=torch.float64, device="cuda")
    outs, lses = [], []
    for b in range(c["batch"]):
        n = int(s["cache_seqlens"][b])
        pages = s["block_table"][b, :-(-n // PAGE)].long()
        rec = s["cache"][pages].reshape(-1, FP4_REC)[:n]
        by = rec[:, :256].int()
        nib = torch.stack([by & 15, by >> 4], 2).view(n, 512)
        e = torch.tensor(_E4M3 + [float("nan")], dtype=torch.float64, device="cuda")[(rec[:, 256:288] & 127).int()]
        lat = mags[nib & 7] * (1 - 2 * (nib >> 3)).double() * e.repeat_interleave(16, 1)
        keys = torch.cat([lat, rec[:, 288:].contiguous().view(torch.bfloat16).double()], 1)
        for i in range(c["s_q"]):
            if c["topk"]:
                ids = s["indices"][b, i].long()
                k = keys[ids[(ids >= 0) & (ids < n)]]
            else:
                k = keys[:max(0, n - c["s_q"] + i + 1)] if c["causal"] else keys
            sc = s["q"][b, i].double() @ k.T * SCALE
            ext = sc if s["sink"] is None else torch.cat([sc, s["sink"].double()[:, None]], 1)
            if ext.shape[1] == 0:
                outs.append(torch.zeros(c["heads"], D_LAT, dtype=torch.float64, device="cuda"))
                lses.append(torch.full((c["heads"],), -float("inf"), dtype=torch.float64, device="cuda"))
                continue
            lse = torch.logsumexp(ext, 1)
            outs.append(torch.exp(sc - lse[:, None]) @ k[:, :D_LAT])
            lses.append(lse)
    shape = (c["batch"], c["s_q"], c["heads"])
    return {"out": torch.stack(outs).view(*shape, D_LAT), "lse": torch.stack(lses).view(shape)}
