"""DecodeRunner takes the cache's format and its number of pages from the cache's
shape, so it refuses shapes that would make the kernels read past the cache: before
anything is allocated or launched, so these run without a device."""
import types

import pytest
import torch

import head_latent_attention_get_b200 as M


def run(kcache):
    q = types.SimpleNamespace(device=torch.device("cuda", 0), dtype=torch.bfloat16, shape=(2, 1, 16, 576))
    with pytest.raises(AssertionError, match="record"):
        M.DecodeRunner(q, kcache, None, None, softmax_scale=0.1)


@pytest.mark.parametrize("record", [416, 656])
def test_record_caches_of_another_shape(record):
    u8 = dict(dtype=torch.uint8)
    run(torch.zeros(3, 64 * record, **u8))                      # pages as one run of bytes
    run(torch.zeros(3 * 64, record, **u8))                      # tokens in the place of pages
    run(torch.zeros(3, 32, record, **u8))                       # pages of 32
    run(torch.zeros(3, 64, record + 16, **u8))
    run(torch.zeros(3, 64, record + 16, **u8)[..., :record])    # records further apart
    run(torch.zeros(3, 64, record, dtype=torch.float16))


class OnCuda:
    """A host tensor that says it is on a CUDA device."""
    def __init__(self, t, index=0):
        self.t, self.device = t, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.t, name)


def inputs(kv, **kw):
    z = torch.zeros
    a = dict(q=z(2, 1, 4, 576, dtype=torch.bfloat16), kcache=z(3, 64, 1, 576, dtype=torch.bfloat16), block_table=z(2, 5, dtype=torch.int32),
             cache_seqlens=z(2, dtype=torch.int32), indices=z(2, 1, 64, dtype=torch.int32))
    if kv == "fp4":
        a["kcache"] = z(3, 64, 416, dtype=torch.uint8)
    if kv == "nvfp4":
        a.update(q=z(2, 1, 4, 256, dtype=torch.uint8), kcache=z(3, 64, 256, dtype=torch.uint8), q_scale=z(2, 1, 4, 32, dtype=torch.uint8),
                 kv_scale=z(3, 64, 32, dtype=torch.uint8))
        del a["indices"]
    a.update(kw)
    return {k: OnCuda(v) if isinstance(v, torch.Tensor) else v for k, v in a.items()}


def refused(kv, name, t):
    a = inputs(kv, **{name: t})
    with pytest.raises(AssertionError, match=name):
        M.DecodeRunner(a.pop("q"), a.pop("kcache"), a.pop("block_table"), a.pop("cache_seqlens"), softmax_scale=0.1, **a)


@pytest.mark.parametrize("kv", ["bf16", "fp4", "nvfp4"])
@pytest.mark.parametrize("name", ["q", "kcache", "block_table", "cache_seqlens", "indices", "q_scale", "kv_scale"])
def test_inputs_that_would_be_misread(kv, name):
    good = inputs(kv).get(name)
    if good is None:
        return
    good = good.t
    if name in ("block_table", "cache_seqlens", "indices"):
        refused(kv, name, good.long())
    if name in ("q_scale", "kv_scale"):
        refused(kv, name, good.float())
    if name != "q":
        refused(kv, name, OnCuda(good, 1))                       # q says where the others have to be
        refused(kv, name, OnHost(good))
    if name not in ("kcache",) or kv == "bf16":                  # records: the test above
        refused(kv, name, torch.zeros(*good.shape, 2, dtype=good.dtype)[..., 0])
    if name not in ("q", "kcache"):
        refused(kv, name, good[:1].contiguous() if good.dim() > 1 else good[:1])


class OnHost(OnCuda):
    def __init__(self, t):
        self.t, self.device = t, torch.device("cpu")


def test_pages_that_are_not_64_tokens():
    refused("bf16", "kcache", torch.zeros(3, 32, 1, 576, dtype=torch.bfloat16))
