"""DecodeRunner's calls run on its tensors' device, whichever is current."""
import contextlib

import pytest
import torch

import head_latent_attention_get_b200 as M
from head_latent_attention_get_b200 import _capi as C


@pytest.mark.parametrize("current,own,topk", [(0, 0, 0), (0, 1, 0), (1, 0, 64)])
def test_calls_run_on_the_tensors_device(monkeypatch, current, own, topk):
    now, seen = [current], []

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        yield
        now[0] = before

    monkeypatch.setattr(C, "_device_calls", (lambda: now[0], lambda d: 100 + d))
    monkeypatch.setattr(torch.cuda, "device", device)
    for name in ("mla_get_metadata", "mla_decode_paged", "mla_decode_sparse", "mla_query_device_status"):
        monkeypatch.setattr(C, name, lambda *a, name=name: seen.append((name, now[0], C._stream(a[-1]))))
    r = M.DecodeRunner.__new__(M.DecodeRunner)
    r.__dict__.update(device_index=own, topk=topk, cache_seqlens=None, batch=1, s_q=1, h_q=1, parts=1, tile_md=None, num_splits=None,
                      args=None, indices=None, out=1, lse=2, workspace=None)
    r.plan()
    assert r.run() == (1, 2)
    r.status()
    decode = "mla_decode_sparse" if topk else "mla_decode_paged"
    assert seen == [(n, own, 100 + own) for n in ("mla_get_metadata", decode, "mla_query_device_status")]
    assert now == [current]
    r.run(7)
    assert seen[-1] == (decode, own, 7)
