"""Decode over a paged cache at the ends of its values' range: queries, weights and scales far
apart, infinities.  The reference and its tolerances are those of test_gpu_decode_paged.py: the
bounds there are relative to the terms of each sum, so a term that is lost shows wherever the
larger ones are zero."""
import math

import pytest
import torch

from block_sparse_gqa_topk_gb300 import ops
from test_gpu_decode_paged import SLACK, Batch, check_attention, query

pytestmark = pytest.mark.gpu


def both_forms(batch, q, qi, topk, check):
    """check(o, lse, tokens) for the dense call, and for the sparse one with the blocks it took."""
    o, lse = ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)
    check(o, lse, lambda b, g: batch.rows(b, batch.lens[b]))
    sets, o, lse = ops.msa_decode_paged(q, qi, batch.cache, batch.table, batch.lens_t, topk)
    host = sets.cpu()

    def taken(b, g):
        rows = batch.rows(b, batch.lens[b])
        return torch.cat([rows[:0]] + [rows[c * 128:(c + 1) * 128] for c in host[b, g].tolist() if c >= 0])

    check(o, lse, taken)
    assert ops.device_status() == 0


@SLACK
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (64, 12), (128, 9)])
def test_infinite_queries(d, G, fp8, slack):
    """A query with an infinite value has scores of infinities and NaN only: its output is NaN, and
    every other head's is what it was."""
    lens = [300, 129]
    batch = Batch(lens, 16, 2, d, 32, fp8, seed=1, slack=slack)
    q, qi = query(2, 2 * G, d, 2), query(2, 2, 32, 3)
    bad = [(0, 1, math.inf), (1, 2 * G - 1, -math.inf)]
    for b, h, x in bad:
        q[b, h, 5] = x

    def check(o, lse, tokens):
        finite = torch.ones(o.shape[:2], dtype=torch.bool, device="cuda")
        for b, h, _ in bad:
            assert torch.isnan(o[b, h]).all() and not torch.isfinite(lse[b, h])
            finite[b, h] = False
        assert torch.isfinite(o[finite]).all() and torch.isfinite(lse[finite]).all()
        clean = torch.where(finite[..., None], q, 0)
        for b in range(2):
            got, gl = o[b].clone(), lse[b].clone()
            for h in (~finite[b]).nonzero().flatten().tolist():  # a zero query instead: the mean
                rows = tokens(b, h // G)
                got[h] = batch.values("v", rows, h // G).mean(0).bfloat16()
                gl[h] = math.log(len(rows))
            check_attention(batch, b, clean, got[None].expand(2, -1, -1), gl[None].expand(2, -1),
                            lambda g, b=b: tokens(b, g), d ** -0.5)

    both_forms(batch, q, qi, 2, check)
