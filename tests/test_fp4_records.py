"""The 416-byte 4-bit token record on the CPU: the oracle's decoding against a
hand-decoded record and against the NVFP4 and bf16 decoders of its parts, the
test quantiser's round trip, and the decode entry points' argument checks."""
import ctypes

import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M
from head_latent_attention_get_b200 import _capi as C
from oracle import mla_oracle as O
from workloads import mla_workloads as W


def test_hand_decoded_record():
    rec = np.zeros((1, 64, 416), dtype=np.uint8)
    rec[0, 3, 0] = 0x5F        # element 0: code F = -6, element 1: code 5 = 3
    rec[0, 3, 255] = 0x1C      # element 510: code C = -2, element 511: code 1 = 0.5
    rec[0, 3, 256] = 0x38      # scale 1.0
    rec[0, 3, 287] = 0xC4      # sign bit ignored: 0x44 = exponent 8, mantissa 4 -> 2 * 1.5 = 3.0
    rec[0, 3, 288:290] = [0x80, 0x3F]   # bf16 1.0
    rec[0, 3, 414:416] = [0x40, 0xC0]   # bf16 -3.0
    row = O.dequant_fp4_records(rec)[0, 3]
    want = np.zeros(576)
    want[[0, 1, 510, 511, 512, 575]] = [-6.0, 3.0, -6.0, 1.5, 1.0, -3.0]
    assert np.array_equal(row, want)


def test_quantiser_round_trip():
    """Half an E2M1 step of the block's scale, at most one eighth of 6 * scale
    plus the scale's own rounding (half an e4m3 step, 2^-4 relative)."""
    rng = np.random.default_rng(1)
    src = torch.from_numpy(rng.standard_normal((2, 64, 576)).astype(np.float32))
    rec = W.quantize_fp4_records(src)
    assert rec.shape == (2, 64, W.FP4_RECORD_BYTES) and W.FP4_RECORD_BYTES == M.FP4_RECORD_BYTES
    rows = O.dequant_fp4_records(rec.numpy())
    blk = src[..., :512].numpy().reshape(2, 64, 32, 16)
    amax = np.abs(blk).max(-1, keepdims=True)
    err = np.abs(rows[..., :512].reshape(blk.shape) - blk)
    assert np.all(err <= amax * (1 / 6 * (1 + 2.0 ** -4) + 2.0 ** -4) + 2.0 ** -10)
    assert np.array_equal(rows[..., 512:], O.torch_bf16_to_f64(src[..., 512:].to(torch.bfloat16)))


def _args(**kw):
    buf = np.zeros(4096, dtype=np.uint8)
    base = (buf.ctypes.data + 255) // 256 * 256
    a = C.MlaDecodeArgs()
    for f in ("q", "kcache", "block_table", "cache_seqlens", "tile_md", "num_splits", "out", "lse", "workspace"):
        setattr(a, f, base)
    a.batch, a.s_q, a.h_q, a.h_kv, a.d_qk, a.d_v, a.page_size = 2, 1, 16, 1, 576, 512, 64
    a.num_pages, a.block_table_stride, a.num_sm_parts, a.softmax_scale = 4, 2, 8, 0.1
    a.kv_format = M.MLA_KV_FP4_E2M1
    a.workspace_bytes = 1 << 30
    a._keep = buf
    for k, v in kw.items():
        setattr(a, k, v)
    return a, base


@pytest.mark.parametrize("kw,code", [
    (dict(d_qk=512), M.MLA_ERR_INVALID_ARG), (dict(kv_format=4), M.MLA_ERR_INVALID_ARG),
    (dict(page_size=32), M.MLA_ERR_INVALID_ARG), (dict(h_kv=2), M.MLA_ERR_UNSUPPORTED),
    (dict(kcache=None), M.MLA_ERR_INVALID_ARG), (dict(workspace_bytes=64), M.MLA_ERR_WORKSPACE_TOO_SMALL),
    (dict(softmax_scale=float("nan")), M.MLA_ERR_INVALID_ARG), (dict(num_pages=1 << 25), M.MLA_ERR_UNSUPPORTED)])
def test_decode_refusals(kw, code):
    a, _ = _args(**kw)
    assert M.lib().mla_decode_paged(ctypes.byref(a), None) == code


def test_decode_refuses_misaligned_cache():
    a, base = _args()
    a.kcache = base + 8
    assert M.lib().mla_decode_paged(ctypes.byref(a), None) == M.MLA_ERR_INVALID_ARG
    a, base = _args(h_q=129)
    assert M.lib().mla_decode_sparse(ctypes.byref(a), base, 64, None) == M.MLA_ERR_UNSUPPORTED
    a, base = _args()
    assert M.lib().mla_decode_sparse(ctypes.byref(a), base, 65, None) == M.MLA_ERR_INVALID_ARG
