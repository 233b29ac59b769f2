"""msa_kv8_attn_weights: the sums of long prompts, whose many faint weights stand beside a few large ones."""
import math

import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention
from tests import _kv8_long
from tests.test_gpu_kv8_attn_weights import q64, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,G,qtype", [(2053, 8, "bf16"), (2053, 8, "e4m3"), (300, 64, "bf16"), (9000, 2, "e4m3")])
def test_faint_weights_of_many_rows_are_not_lost(rows, G, qtype):
    """Queries of zeros score 0 everywhere, so each weight is exp(-lse): 1 for the first row's first two queries, 2^-25
    for all others, which one running sum of a token's queries would lose one by one (2^-25 is half of half a step at 1;
    some 2.4e-4 of the token's weight).

    Bound. A thread takes 128 queries a unit in four chains of at most 32 additions, whose sums are added (3 more, 5
    with the chunks of 32); that sum is added to those of the units before, at most `units` of them, and a quad of
    pages that is cut over CTAs joins no more sums than it has units: 2^-24 of the sum for each. An exponential adds
    2^-21 and its rounded argument 2^-22 |lse|."""
    n = rows + 16_000       # (more quads of pages than CTAs: most are summed from end to end by one)
    cache, batch, lens, indptr, table, old = setup([n, 300], [rows, 1], 4, G, qtype, 151)
    batch.q = torch.zeros_like(batch.q)
    lse = torch.full(batch.q.shape[:2], 25 * math.log(2.0), device="cuda")
    lse[0, 0::G] = 0.0
    lse[0, 1::G] = 0.0
    att = KV8Attention(cache, batch, with_weights=True)
    new = torch.zeros_like(old)
    att.add_weights(None, new, lse=lse)
    assert att.errors() == 0
    want = _kv8_long.weights(q64(batch, cache), lse, cache, lens, indptr, table, None, 1.0)
    units = (rows * G + 127) // 128
    for h in range(4):
        w, _ = want[0, h]
        tol = w * ((40 + 2 * units) * 2.0 ** -24 + 2.0 ** -21) + 25 * math.log(2.0) * 2.0 ** -22 * rows * G * 2.0 ** -25
        _kv8_long.close(new[0, h, :n], w, tol, f"head {h}")
