"""The 4-bit cache on the GPU at the edges of what its calls accept, against the plain restatement
in 64 bits."""
import numpy as np
import pytest
import torch

import nibble_ref as ref
import test_gpu_nibble as base

pytestmark = pytest.mark.gpu

dw = pytest.importorskip("decode_attention_depthweave_b200")

BF, FP = torch.bfloat16, torch.float16
i32, ops = base.i32, base.ops


# ------------------------------------------------------------------------------ tables
@pytest.mark.parametrize("new", [
    [1 << 30, 1 << 30, 1, 1], [1 << 30, 1 << 30, 1 << 30, 1 << 30, 5, 2], [2**31 - 1] * 6 + [3, 0, 2], [4, 1 << 30, 1, (1 << 30) - 1, 2],
    [1] * 40 + [1 << 30] * 4 + [2] * 90, [1 << 30, 0] * 150 + [3]])
def test_totals_of_refused_counts_stay_at_their_cap(new):
    """Counts that no table holds are refused, and so is every row behind them: lengths, pages and slots
    stay as they were, whatever the counts add up to."""
    n, page, pages, width = len(new), 16, 400, 4
    nb = ops(page=page, pages=pages, seqs=n, blocks=width)
    st = dict(seq_lens=[0] * n, block_tables=[[0] * width for _ in range(n)], free_list=list(range(pages)), free_count=[pages])
    base.step(nb, st, new, [0] * n, page, 64)
    with pytest.raises(dw.DwkvError, match="length or count|do not fit"):
        nb.sync()
    # and in a step that releases too
    st = dict(st, seq_lens=[1] * n, block_tables=[[b, 0, 0, 0] for b in range(n)], free_list=list(range(n, pages)) + [0] * n,
              free_count=[pages - n])
    base.step(nb, st, new, [b % 3 == 0 for b in range(n)], page, 64, in_place=False)
    with pytest.raises(dw.DwkvError, match="length or count|do not fit"):
        nb.sync()


# ------------------------------------------------------------------------------ windows
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 16, 2**30, 4096, 1088, 1087, 1086])
@pytest.mark.parametrize("lens,qs", [([2, 1000], [6, 1]), ([2, 0, 700], [3, 2, 1]), ([3, 1000], [200, 60]), ([0, 1, 1087], [40, 90, 1])])
def test_windows_as_long_as_a_request_or_longer(window, lens, qs):
    """Up to the largest that a configuration takes, with rows that stand before the first token."""
    width = 17 - -(-max(lens) // 64)                              # rows of 17 pages: 1088 tokens
    r = base.Requests(61, 8, 2, 128, 64, BF, lens, qs, window, extra_blocks=width)
    assert r.nb.max_blocks == 17
    out, lse = r.run()
    r.nb.sync()
    r.check(out, lse)
