"""Edges of the paged cache's operators (gdr_kv_append, gdr_kv_gather, gdr_attn_paged) against
their formulas in 64 bits; bounds in paged_testutil where a test states no other."""
import pytest
import torch

import linear_attention_recurrence_10_b200 as gdr
from paged_testutil import D, NAN, U8, Problem, rope64, status_of

pytestmark = pytest.mark.gpu


# ------------------------------------------------- rows past a sequence's end


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_last_tiles_of_every_length(kind):
    """Chunks that end at every place of a step of the products (16 keys, 32 codes), at either
    half of a tile: what the pages hold behind them (NaN) is cleared before it is multiplied, by
    both blocks of a pair for both, and every call gives the first one's bits."""
    past = [0, 64, 128, 300]
    for i in range(8):
        new = [257 + 5 * i + j for j in range(4)]
        p = Problem(new=new, past=past, page=[16, 64, 128, 256][i % 4], kind=kind, seed=400 + i)
        assert p.rows * 8 >= 256 * p.n_seq  # (pairs, for bf16)
        p.put_plain()
        out, lse, ws = p.attend()
        assert status_of(ws) == 0
        p.check_attend(out, lse, what=i)
        for _ in range(20):
            again, lse2, _ = p.attend(workspace=ws)
            assert torch.equal(out, again) and torch.equal(lse, lse2)
