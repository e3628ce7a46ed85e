"""The Python calls mla_extend_tables and mla_kv_append refuse tensors that the
library would misread (another element type, gaps), read out of bounds (too
small) or fault on (host memory, another device). Stand-ins report a CUDA device
here; the library below them is replaced by a recorder."""
import pytest
import torch

import head_latent_attention_get_b200 as M
from head_latent_attention_get_b200 import _capi as C


class OnDevice:
    """A host tensor that says it is on a CUDA device."""
    def __init__(self, t, device=0):
        self.t, self.device = t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or 0

    real = C.lib()
    rec = Recorder()
    rec.__dict__["mla_status_string"] = real.mla_status_string
    monkeypatch.setattr(C, "_lib", rec)
    monkeypatch.setattr(C, "_device_calls", (lambda: 0, lambda device: 77))
    return seen


B, STRIDE, AXIS, PAGES = 3, 5, 8, 20
I = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731


def tables(**kw):
    a = dict(context_lens=I(B), new_lens=I(B), free_pages=I(6), free_range=I(2), block_table=I(B, STRIDE), seqlens=I(B), token_start=I(B + 1),
             slots=I(AXIS), positions=I(AXIS), free_next=I(1), status=I(1))
    a.update(kw)
    a = {k: OnDevice(v) if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    M.mla_extend_tables(a["context_lens"], a["new_lens"], B, a["free_pages"], a["free_range"], PAGES, a["block_table"], STRIDE, a["seqlens"],
                        a["token_start"], a["slots"], a["positions"], AXIS, a["free_next"], a["status"])
    return a


def test_tables_pass_what_fits(calls):
    a = tables()
    (name, args), = calls
    ptr = {k: v.data_ptr() for k, v in a.items()}
    assert name == "mla_extend_tables"
    assert args == (ptr["context_lens"], ptr["new_lens"], B, ptr["free_pages"], 6, ptr["free_range"], PAGES, ptr["block_table"], STRIDE,
                    ptr["seqlens"], ptr["token_start"], ptr["slots"], ptr["positions"], AXIS, ptr["free_next"], ptr["status"], 77)


def test_tables_without_a_free_list_or_status(calls):
    tables(free_pages=None, status=None)
    assert calls[0][1][3] is None and calls[0][1][4] == 0 and calls[0][1][15] is None


def test_tables_larger_buffers_and_a_workspace_as_status(calls):
    wide = I(B + 4, STRIDE + 3)
    tables(context_lens=I(B + 9), block_table=wide[:, :STRIDE], status=torch.zeros(256, dtype=torch.uint8))
    assert len(calls) == 1


NAMES = ["context_lens", "new_lens", "free_pages", "free_range", "block_table", "seqlens", "token_start", "slots", "positions", "free_next",
         "status"]


@pytest.mark.parametrize("name", NAMES)
def test_tables_refuse(calls, name):
    good = tables()[name].t
    calls.clear()
    n = good.numel()
    bad = [good.long(), good.float(), OnDevice(good, -1), OnDevice(good, 1), good.numpy(), 12345]
    if name not in ("free_pages",):
        bad.append(good.flatten()[:n - 1].clone())
    if n > 1:
        bad.append(I(*good.shape, 2)[..., 0])               # gaps
    for t in bad:
        with pytest.raises(M.MLAError, match=name) as e:
            tables(**{name: t})
        assert e.value.code == M.MLA_ERR_INVALID_ARG
    assert calls == []


FORMATS = {M.MLA_KV_BF16: (1152, 576), M.MLA_KV_FP8_E4M3: (656, 576), M.MLA_KV_NVFP4: (256, 512), M.MLA_KV_FP4_E2M1: (416, 576)}
T = 6


def append(fmt, stride=None, **kw):
    rec, d = FORMATS[fmt]
    a = dict(kv=torch.zeros(T, d, dtype=torch.bfloat16), gamma=torch.zeros(512), rope_cos=torch.zeros(T, 32), rope_sin=torch.zeros(T, 32),
             slots=I(T), kcache=torch.zeros(2, 64, rec, dtype=torch.uint8), kv_scale=torch.zeros(2, 64, 32, dtype=torch.uint8),
             kv_out=torch.zeros(T, d, dtype=torch.bfloat16), status=I(1))
    a.update(kw)
    a = {k: OnDevice(v) if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    M.mla_kv_append(a["kv"], stride or d, T, d, a["gamma"], 1e-6, a["rope_cos"], a["rope_sin"], a["slots"], a["kcache"], a["kv_scale"], fmt, 2,
                    a["kv_out"], a["status"])
    return a


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_append_passes_what_fits(calls, fmt):
    rec, d = FORMATS[fmt]
    a = append(fmt)
    ptr = {k: v.data_ptr() for k, v in a.items()}
    assert calls[0][0] == "mla_kv_append"
    assert calls[0][1] == (ptr["kv"], d, T, d, ptr["gamma"], 1e-6, ptr["rope_cos"], ptr["rope_sin"], ptr["slots"], ptr["kcache"],
                           ptr["kv_scale"] if fmt == M.MLA_KV_NVFP4 else None, fmt, 2, ptr["kv_out"], ptr["status"], 77)
    append(fmt, stride=640, kv=torch.zeros(T, 640, dtype=torch.bfloat16)[:, :d], gamma=None, rope_cos=None, rope_sin=None, kv_out=None,
           status=None)
    assert calls[1][1][1] == 640 and calls[1][1][4] is None
    append(M.MLA_KV_BF16, kcache=torch.zeros(2, 64, 1, 576, dtype=torch.bfloat16))
    assert len(calls) == 3


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("name", ["kv", "gamma", "rope_cos", "rope_sin", "slots", "kcache", "kv_scale", "kv_out", "status"])
def test_append_refuses(calls, fmt, name):
    if name == "kv_scale" and fmt != M.MLA_KV_NVFP4:
        append(fmt, kv_scale=torch.zeros(1, dtype=torch.float64))      # ignored, as the header says
        return
    good = append(fmt)[name].t
    calls.clear()
    bad = [good.double(), good.to(torch.int64), good.half(), OnDevice(good, -1), OnDevice(good, 1), good.flatten()[:good.numel() - 1].clone(), 7]
    if good.numel() > 1:
        bad.append(torch.zeros(*good.shape, 2, dtype=good.dtype)[..., 0])
    for t in bad:
        with pytest.raises(M.MLAError, match=name) as e:
            append(fmt, **{name: t})
        assert e.value.code == M.MLA_ERR_INVALID_ARG
    assert calls == []


def test_append_refuses_rows_past_the_end(calls):
    wide = torch.zeros(T, 640, dtype=torch.bfloat16)
    append(M.MLA_KV_FP4_E2M1, stride=640, kv=wide[:, 64:])             # its last row ends with the memory
    with pytest.raises(M.MLAError, match="kv"):
        append(M.MLA_KV_FP4_E2M1, stride=640, kv=wide[:, 65:])
    assert len(calls) == 1
