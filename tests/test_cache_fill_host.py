"""Argument checks of mla_extend_tables and mla_kv_append: every call here is
refused before any launch, so none needs a device."""
import ctypes

import numpy as np
import pytest

import head_latent_attention_get_b200 as M

BUF = np.zeros(1 << 16, dtype=np.uint8)
BASE = (BUF.ctypes.data + 1023) // 1024 * 1024


def _tables(**kw):
    names = ["context_lens", "new_lens", "batch", "free_pages", "num_free", "free_range", "num_pages", "block_table",
             "block_table_stride", "seqlens", "token_start", "slots", "positions", "max_tokens", "free_next", "status"]
    a = dict(batch=4, num_free=8, num_pages=16, block_table_stride=3, max_tokens=20, status=None)
    for i, n in enumerate(n for n in names if n not in a):
        a[n] = BASE + 1024 * (i + 1)
    a.update(kw)
    return M.lib().mla_extend_tables(*[a[n] for n in names], None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=-1), dict(num_pages=0), dict(block_table_stride=0), dict(max_tokens=0), dict(num_free=-1),
    dict(context_lens=None), dict(new_lens=None), dict(free_range=None), dict(free_pages=None), dict(block_table=None),
    dict(seqlens=None), dict(token_start=None), dict(slots=None), dict(positions=None), dict(free_next=None),
    dict(slots=BASE + 2), dict(status=BASE + 1)])
def test_tables_invalid(kw):
    assert _tables(**kw) == M.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(num_pages=1 << 25), dict(block_table_stride=1 << 25), dict(max_tokens=(1 << 30) + 1)])
def test_tables_unsupported(kw):
    far = 1 << 40    # far apart, so that the large buffers do not overlap the others
    places = {n: far * (i + 1) for i, n in enumerate(["block_table", "slots", "positions"])}
    assert _tables(**{**places, **kw}) == M.MLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("out,other", [("seqlens", "context_lens"), ("free_next", "free_range"), ("slots", "positions"),
                                       ("token_start", "new_lens"), ("block_table", "free_pages")])
def test_tables_overlap(out, other):
    place = BASE + 20 * 1024
    assert _tables(**{out: place, other: place}) == M.MLA_ERR_INVALID_ARG
    assert _tables(**{out: place, other: place - 4}) == M.MLA_ERR_INVALID_ARG


def _append(**kw):
    names = ["kv", "kv_stride", "tokens", "d_qk", "gamma", "eps", "rope_cos", "rope_sin", "slots", "kcache", "kv_scale",
             "kv_format", "num_pages", "kv_out", "status"]
    a = dict(kv_stride=576, tokens=4, d_qk=576, eps=1e-6, kv_format=M.MLA_KV_FP4_E2M1, num_pages=2, kv_scale=None,
             status=None)
    for i, n in enumerate(n for n in names if n not in a):
        a[n] = BASE + 1024 * (i + 1)
    a.update(kw)
    return M.lib().mla_kv_append(*[ctypes.c_float(a[n]) if n == "eps" else a[n] for n in names], None)


@pytest.mark.parametrize("kw", [
    dict(kv=None), dict(slots=None), dict(kcache=None), dict(tokens=0), dict(tokens=-3), dict(num_pages=0),
    dict(kv_format=4), dict(kv_format=-1), dict(d_qk=512), dict(d_qk=575), dict(kv_stride=575), dict(kv_stride=580),
    dict(kv=BASE + 8), dict(kcache=BASE + 8), dict(kv_out=BASE + 8), dict(gamma=BASE + 8), dict(slots=BASE + 2),
    dict(rope_sin=None), dict(rope_cos=None), dict(eps=-1.0), dict(eps=float("nan")), dict(status=BASE + 2),
    dict(kv_format=M.MLA_KV_NVFP4), dict(kv_format=M.MLA_KV_NVFP4, d_qk=512, kv_stride=512),
    dict(kv_format=M.MLA_KV_NVFP4, d_qk=512, kv_stride=512, kv_scale=BASE + 8)])
def test_append_invalid(kw):
    assert _append(**kw) == M.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(num_pages=1 << 25), dict(tokens=(1 << 30) + 1)])
def test_append_unsupported(kw):
    assert _append(**kw) == M.MLA_ERR_UNSUPPORTED


def test_status_string():
    assert M.mla_status_string(M.MLA_ERR_DEVICE_NO_PAGES) == "MLA_ERR_DEVICE_NO_PAGES"
