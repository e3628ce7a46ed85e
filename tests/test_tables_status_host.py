"""mla_extend_tables refuses a status word that lies in another buffer."""
import numpy as np
import pytest

import head_latent_attention_get_b200 as M

BUF = np.zeros(1 << 16, dtype=np.uint8)
BASE = (BUF.ctypes.data + 1023) // 1024 * 1024
NAMES = ["context_lens", "new_lens", "free_pages", "free_range", "block_table", "seqlens", "token_start", "slots", "positions", "free_next"]


@pytest.mark.parametrize("name", NAMES)
def test_status_word_in_another_buffer(name):
    a = {n: BASE + 1024 * (i + 1) for i, n in enumerate(NAMES)}
    assert M.lib().mla_extend_tables(a["context_lens"], a["new_lens"], 4, a["free_pages"], 8, a["free_range"], 16, a["block_table"], 3,
                                     a["seqlens"], a["token_start"], a["slots"], a["positions"], 20, a["free_next"], a[name],
                                     None) == M.MLA_ERR_INVALID_ARG
