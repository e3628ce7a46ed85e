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
