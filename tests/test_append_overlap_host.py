"""mla_kv_append refuses buffers that share memory, before any launch: rows are
read and written in no order, so that a result written over another row's input
would depend on the schedule."""
import ctypes

import numpy as np
import pytest

import head_latent_attention_get_b200 as M

BUF = np.zeros(1 << 20, dtype=np.uint8)
BASE = (BUF.ctypes.data + 1023) // 1024 * 1024
STEP = 1 << 16      # apart; no buffer below is larger: 2 pages of bf16 are 147456 bytes and come last
NAMES = ["kv", "gamma", "rope_cos", "rope_sin", "slots", "kv_out", "status", "kv_scale", "kcache"]
PLACE = {n: BASE + STEP * i for i, n in enumerate(NAMES)}
RECORD = {M.MLA_KV_BF16: 1152, M.MLA_KV_FP8_E4M3: 656, M.MLA_KV_NVFP4: 256, M.MLA_KV_FP4_E2M1: 416}


def append(fmt, tokens=4, stride=None, pages=2, **kw):
    d = 512 if fmt == M.MLA_KV_NVFP4 else 576
    a = {**PLACE, **kw}
    return M.lib().mla_kv_append(a["kv"], stride or d, tokens, d, a["gamma"], ctypes.c_float(1e-6), a["rope_cos"], a["rope_sin"],
                                 a["slots"], a["kcache"], a["kv_scale"], fmt, pages, a["kv_out"], a["status"], None)


def bytes_of(fmt, name, tokens=4, stride=None, pages=2):
    d = 512 if fmt == M.MLA_KV_NVFP4 else 576
    return {"kv": ((tokens - 1) * (stride or d) + d) * 2, "gamma": 2048, "rope_cos": tokens * 128, "rope_sin": tokens * 128,
            "slots": 4 * tokens, "kv_out": tokens * d * 2, "status": 4, "kv_scale": pages * 64 * 32, "kcache": pages * 64 * RECORD[fmt]}[name]


@pytest.mark.parametrize("fmt", list(RECORD))
@pytest.mark.parametrize("out", ["kcache", "kv_scale", "kv_out", "status"])
@pytest.mark.parametrize("other", [n for n in NAMES])
def test_overlaps_are_refused(fmt, out, other):
    if out == other or (fmt != M.MLA_KV_NVFP4 and "kv_scale" in (out, other)):
        return
    last = PLACE[other] + (bytes_of(fmt, other) - 1) // 16 * 16        # the last 16 bytes of the other one
    assert append(fmt, **{out: last}) == M.MLA_ERR_INVALID_ARG
    if (out, other) != ("kv_out", "kv"):
        assert append(fmt, **{out: PLACE[other]}) == M.MLA_ERR_INVALID_ARG


def test_values_over_rows_that_are_further_apart():
    assert append(M.MLA_KV_FP4_E2M1, stride=640, kv_out=PLACE["kv"]) == M.MLA_ERR_INVALID_ARG
    assert append(M.MLA_KV_FP4_E2M1, kv_out=PLACE["kv"] + 16) == M.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("fmt", list(RECORD))
def test_neighbours_and_in_place_are_not_overlaps(fmt):
    """Past the checks the launch fails without a device, which is MLA_ERR_CUDA."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("these addresses are the host's")
    assert append(fmt) == M.MLA_ERR_CUDA
    assert append(fmt, kv_out=PLACE["kv"]) == M.MLA_ERR_CUDA
    assert append(fmt, kv_out=PLACE["kv"] + bytes_of(fmt, "kv")) == M.MLA_ERR_CUDA
    assert append(fmt, kv_scale=PLACE["kv"]) == (M.MLA_ERR_INVALID_ARG if fmt == M.MLA_KV_NVFP4 else M.MLA_ERR_CUDA)
