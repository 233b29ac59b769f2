"""msa_kv8_attn_shared: what one member of a group has stays with it, and what the groups' kernel decides."""
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention
from tests import _kv8_long
from tests.test_gpu_kv8_shared import ALL, ints, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -1.0, 1e-40, 2.0 ** 100])
@pytest.mark.parametrize("members,H,G,qtype", [(16, 2, 8, "bf16"), (16, 2, 8, "e4m3"), (8, 2, 8, "bf16"), (4, 2, 8, "e4m3"),
                                               (32, 1, 1, "bf16")])
def test_a_bad_value_scale_stays_with_its_member(members, H, G, qtype, scale):
    """A value scale outside what the cache allows on one member's own page: the other members' rows as if it were
    another, bit for bit. (With 16, 8 and 4 members of 8 queries the tile has 1, 2 and 4 copies of the rows.)"""
    cache, batch, lens, indptr, table, g = setup([(16, [(100 + 7 * i, 1) for i in range(members)])], H, G, qtype, 167)
    att = KV8Attention(cache, batch, max_groups=1)
    bad = 1
    page = int(table[bad, 16])
    want, want_lse = att.attend_shared(ints(g), min_saved=1).clone(), att.lse.clone()
    cache.v_scale[page] = scale
    out, lse = att.attend_shared(ints(g), min_saved=1), att.lse
    others = [r for r in range(members) if r != bad]
    assert torch.isfinite(want).all()
    assert torch.equal(out[others], want[others]) and torch.equal(lse[others], want_lse[others])
    assert att.errors() == 0
    # and those bits are right
    q64 = batch.q.double().view(members, H, G, 128)
    ref, _, tol, _ = _kv8_long.attend(q64, cache, lens, indptr, table, ALL, qtype != "bf16")
    _kv8_long.close(out[others], ref[others], tol[others], "others")
