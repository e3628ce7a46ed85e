"""mla_extend_tables at the ends of its ranges."""
import numpy as np
import pytest
import torch

import head_latent_attention_get_b200 as M

STRIDE = (1 << 25) - 1      # the longest row: 2^31 - 64 tokens


@pytest.mark.gpu
def test_longest_rows():
    """The last tokens of the longest row, behind others on the token axis: context
    plus place on the axis passes 2^31."""
    dev = dict(dtype=torch.int32, device="cuda")
    room = STRIDE * 64
    ctx, new = [0, room - 200, room - 64, room], [2000, 200, 65, 0]
    bt = torch.full((4, STRIDE), -1, **dev)
    bt[1, (room - 200) // 64] = 7                                   # its last page so far
    free = torch.arange(100, 200, **dev)
    out = {k: torch.full((n,), 77, **dev) for k, n in dict(seqlens=4, start=5, slots=2300, pos=2300, nxt=1, st=1).items()}
    out["st"].zero_()
    M.mla_extend_tables(torch.tensor(ctx, **dev), torch.tensor(new, **dev), 4, free, torch.tensor([0, 100], **dev), 200, bt, STRIDE,
                        out["seqlens"], out["start"], out["slots"], out["pos"], 2300, out["nxt"], out["st"])
    got = {k: v.cpu().numpy() for k, v in out.items()}
    assert got["st"][0] == M.MLA_DEVICE_STATUS_BOUNDS               # the third asks for one token too many
    assert got["seqlens"].tolist() == [2000, room, room - 64, room] and got["start"].tolist() == [0, 2000, 2200, 2265, 2265]
    pos = np.concatenate([np.arange(2000), np.arange(room - 200, room), np.full(100, -1)])
    assert np.array_equal(got["pos"], pos)
    page = np.concatenate([100 + np.arange(2000) // 64, np.where(pos[2000:2200] < room - 192, 7, 132 + (pos[2000:2200] - (room - 192)) // 64)])
    want = np.concatenate([page * 64 + pos[:2200] % 64, np.full(100, -1)])
    assert np.array_equal(got["slots"], want)
    assert got["nxt"][0] == 35 and bt[1, STRIDE - 3:].tolist() == [132, 133, 134]

