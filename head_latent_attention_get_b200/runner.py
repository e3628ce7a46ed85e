"""Buffer plumbing around the C ABI for one decode problem.

PyTorch only allocates device memory here; the scheduler, decode and combine
all run inside libmla_b200.so. Mirrors the plan-once / run-per-layer shape of
the paged MLA decode APIs (metadata computed once per decode step and reused
by every layer: "Qu'est-ce que FlashMLA ?", section "Exécuter le décodage
MLA").
"""
from __future__ import annotations

import functools

import torch

from . import _capi as C


def _on_its_device(method):
    """The library launches on the current device: it is made the runner's own
    where it is another one."""
    @functools.wraps(method)
    def call(self, stream=None):
        if C._device()[0]() == self.device_index:
            return method(self, stream)
        with torch.cuda.device(self.device_index):
            return method(self, stream)
    return call


class DecodeRunner:
    def __init__(self, q, kcache, block_table, cache_seqlens, *, softmax_scale, causal=False,
                 indices=None, num_sm_parts=None, timeout_ns=0, debug_flags=0, sink=None, q_scale=None,
                 kv_scale=None):
        """q bf16 [B, s_q, h_q, 576] with a bf16 cache or a cache of FP8 (656-byte)
        or 4-bit (416-byte) records, or (NVFP4) packed uint8 [B, s_q, h_q, 256] with q_scale/kv_scale and a packed
        uint8 [pages, 64, 256] cache."""
        dev = q.device
        assert dev.type == "cuda", "the decode path runs on a CUDA device only"
        self.batch, self.s_q, self.h_q, d = q.shape
        self.topk = int(indices.shape[-1]) if indices is not None else 0
        if q.dtype == torch.uint8:
            assert d == 256 and kcache.shape[-1] == 256 and q_scale is not None and kv_scale is not None
            self.kv_format, d_qk = C.MLA_KV_NVFP4, 512
        else:
            assert d == 576
            if kcache.dtype == torch.bfloat16:
                self.kv_format = C.MLA_KV_BF16
            else:
                # the last dimension tells the format, and num_pages is taken from the
                # first: both have to be what the cache's memory holds
                formats = {C.FP8_RECORD_BYTES: C.MLA_KV_FP8_E4M3, C.FP4_RECORD_BYTES: C.MLA_KV_FP4_E2M1}
                assert kcache.element_size() == 1 and kcache.shape[-1] in formats, "records are 656 (FP8) or 416 (4-bit) bytes"
                assert kcache.is_contiguous() and kcache.numel() == kcache.shape[0] * 64 * kcache.shape[-1], \
                    "a cache of records is [pages, 64, record bytes]"
                self.kv_format = formats[kcache.shape[-1]]
            d_qk = 576
        pages, requests = kcache.shape[0], self.batch
        queries = requests * self.s_q * self.h_q
        values = kcache.shape[-1] if kcache.element_size() == 1 else 576
        for name, t, types, count in (
                ("q", q, (torch.bfloat16, torch.uint8), queries * d), ("kcache", kcache, None, pages * 64 * values),
                ("block_table", block_table, (torch.int32,), requests * block_table.shape[-1]),
                ("cache_seqlens", cache_seqlens, (torch.int32,), requests),
                ("indices", indices, (torch.int32,), requests * self.s_q * self.topk),
                ("q_scale", q_scale, (torch.uint8, torch.float8_e4m3fn), queries * 32),
                ("kv_scale", kv_scale, (torch.uint8, torch.float8_e4m3fn), pages * 64 * 32)):
            # the kernels take pointers: what they would misread or fault on is refused here
            if t is not None:
                assert t.device == dev, f"{name} is on {t.device}, q on {dev}"
                assert types is None or t.dtype in types, f"{name} must be {types[0]}, not {t.dtype}"
                assert t.is_contiguous(), f"{name} must be contiguous"
                assert t.numel() >= count, f"{name} has {t.numel()} elements, {count} are used"
        self.device_index = dev.index
        self.q_scale, self.kv_scale = q_scale, kv_scale
        upr, self.rows = C.mla_decode_geometry(self.s_q, self.h_q, 1, self.topk)
        self.units = self.batch * upr
        self.parts = num_sm_parts or C.mla_get_num_sm_parts(dev.index, self.s_q, self.h_q, 1, self.topk)
        self.tile_md = torch.empty(self.parts * C.MLA_TILE_MD_INTS, dtype=torch.int32, device=dev)
        self.num_splits = torch.empty(self.units + 1, dtype=torch.int32, device=dev)
        ws_bytes = C.mla_workspace_size(self.batch, self.s_q, self.h_q, 1, self.topk, self.parts)
        self.workspace = torch.zeros(ws_bytes, dtype=torch.uint8, device=dev)
        self.out = torch.empty(self.batch, self.s_q, self.h_q, 512, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(self.batch, self.s_q, self.h_q, dtype=torch.float32, device=dev)
        self.q, self.kcache, self.block_table, self.cache_seqlens = q, kcache, block_table, cache_seqlens
        self.indices = indices
        if sink is not None:
            assert sink.device == dev and sink.dtype == torch.float32 and sink.shape == (self.h_q,)
            sink = sink.contiguous()
        self.sink = sink
        self.args = C.make_args(
            q=q, kcache=kcache, block_table=block_table, cache_seqlens=cache_seqlens,
            tile_md=self.tile_md, num_splits=self.num_splits, out=self.out, lse=self.lse,
            workspace=self.workspace, batch=self.batch, s_q=self.s_q, h_q=self.h_q, h_kv=1,
            num_pages=kcache.shape[0], num_sm_parts=self.parts, softmax_scale=softmax_scale,
            causal=causal, kv_format=self.kv_format, timeout_ns=timeout_ns, debug_flags=debug_flags,
            sink=sink, d_qk=d_qk, q_scale=q_scale, kv_scale=kv_scale)

    @_on_its_device
    def plan(self, stream=None):
        C.mla_get_metadata(self.cache_seqlens, self.batch, self.s_q, self.h_q, 1, self.topk, self.parts,
                           self.tile_md, self.num_splits, stream)

    @_on_its_device
    def run(self, stream=None):
        if self.topk:
            C.mla_decode_sparse(self.args, self.indices, self.topk, stream)
        else:
            C.mla_decode_paged(self.args, stream)
        return self.out, self.lse

    @_on_its_device
    def status(self, stream=None):
        return C.mla_query_device_status(self.workspace, stream)
