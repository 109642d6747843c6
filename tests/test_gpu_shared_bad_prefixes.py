"""Branches behind prefixes whose length or page is ill-formed, with fewer new tokens than columns: their
rows are NaN and what lies past count[b] stays as it was, whether a prefix is shared or read by each branch."""
import pytest
import torch

import draft_token_verification_11_amd as sv
from tests.test_gpu_attention_shared import _case, _i32, _run

pytestmark = pytest.mark.gpu


# Narrow tables: each branch reads its prefix by itself, (branch, kv head) pairs few, a workgroup for
# each, or many, a wave for each; wide ones: prefixes are shared.
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fan,Hq,H,wide", [(4, 4, 2, 0), (4, 4, 2, 400), (4, 64, 64, 0), (4, 4, 2, 18000), (70, 4, 2, 18000)])
def test_rows_past_count_stay(D, fan, Hq, H, wide):
    T, n = 3, 5
    B = n * fan - 1
    start, count = [(b * 7) % 60 for b in range(B)], [(b + b // fan) % (T + 1) for b in range(B)]
    count[fan + 1], count[3 * fan + 2], count[fan + 3] = T + 1, -1, T + 9
    q, pages, table, ptable = _case(21, B, fan, T, Hq, H, D, start, [130] * n, wide=wide)
    prefix = [130, -1, 64 * ptable.shape[1] + 1, 130, 130]
    ptable[4, 1] = -1
    ill = [not 0 <= count[b] <= T for b in range(B)]
    bad = [b // fan in (1, 2, 4) for b in range(B)]
    out, lse = (x.cpu() for x in _run(q, pages, table, start, ptable, prefix, fan, count))
    for b in range(B):
        new = T if ill[b] else count[b]
        for x in (out[b], lse[b]):
            nan = torch.isnan(x[:new])
            assert nan.all() if ill[b] or bad[b] else not nan.any(), (b, count[b])
            assert (x[new:] == 7).all(), (b, count[b])
