"""GPU tests of the softmax weights of the 8-bit attention where the exponents of FP16 and FP32
end: long faint tails beside one large key, value scales over their whole range, pages whose
value scale is 0."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache
from tests import _kv8
from tests.test_gpu_kv8 import _assert_attends

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ONE = 0x38          # the E4M3 code of 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _batch(reqs, n, rows, G, q, table=None):
    """`reqs` requests of n tokens on the same pages, `rows` query rows each."""
    need = (n + 127) // 128
    table = np.arange(need) if table is None else np.asarray(table)
    lens = np.full(reqs, n, np.int32)
    indptr = (np.arange(reqs + 1) * rows).astype(np.int32)
    t = np.tile(table.astype(np.int32), (reqs, 1))
    batch = KV8Batch(_cuda(lens), _cuda(indptr), _cuda(t), q, total_rows=reqs * rows, max_rows_per_req=rows)
    return batch, lens, indptr, t


# 1, 8 and 16 rows of 8 queries: four, two and one copy of the query rows in a tile
@pytest.mark.parametrize("rows", [1, 8, 16])
@pytest.mark.parametrize("where", [0, 7000])
def test_a_faint_tail_beside_one_large_key(rows, where):
    """Every key scores 0 but one that scores x (base 2), whose value is 0: the output is the tail's alone,
    2^-x of its values' sum. One weight's FP16 rounding: half a subnormal step, 2^-25, where the row's largest
    weight is kept at 2^7 or more, so 2^-32 of the largest; or 2^-11 of the weight itself. The other
    terms are those of _kv8.attend."""
    xs = torch.tensor([0.0, 10.0, 20.0, 24.0, 26.0, 28.0, 30.0, 30.0])    # exact in E4M3
    n, reqs, G = 16384 + rows, 160, 8
    need = (n + 127) // 128
    g = torch.Generator("cuda").manual_seed(rows)
    cache = KV8Cache.empty(need, 1)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(0.25)
    cache.k_data[where // 128, 0, where % 128, 0] = ONE
    cache.v_data.copy_(torch.randint(0x30, 0x39, cache.v_data.shape, dtype=torch.uint8, device="cuda", generator=g))
    cache.v_data[where // 128, 0, where % 128] = 0
    q = torch.zeros((reqs * rows, G, 128), device="cuda")
    q[:, :, 0] = xs.cuda()
    batch, *_ = _batch(reqs, n, rows, G, q.to(torch.float8_e4m3fn).view(torch.uint8))
    att = KV8Attention(cache, batch, sm_scale=math.log(2.0))
    out = att.attend().double().view(reqs, rows, G, 128)
    assert att.errors() == 0
    codes = torch.from_numpy(_kv8.e4m3_values()).cuda()[cache.v_data.long()].reshape(-1, 128)
    for r in range(rows):
        seen = n - rows + r + 1
        total = codes[:seen].sum(0) * 0.25
        for h in range(G):
            big = 2.0 ** float(xs[h])
            norm = big + seen - 1
            want = total / norm
            d = 2.0 ** -16 * float(xs[h]) * math.log(2.0)
            rel = 2.0 ** -11 + 2.0 ** -18 + math.expm1(2 * d)
            tol = 2.0 ** -8 * want + (rel * want + 2.0 ** -32 * total * big / norm) * (1 + 2.0 ** -8)
            over = (out[:, r, h] - want).abs() - tol
            assert bool((over <= 0).all()), (r, h, float(over.max()), float(out[0, r, h, 0]), float(want[0]))
            lse = att.lse.double().view(reqs, rows, G)[:, r, h]
            assert bool(((lse - math.log(norm)).abs() <= d + 2.0 ** -18 + 2.0 ** -22 * math.log(norm)).all())


@pytest.mark.parametrize("rows", [1, 8, 16])
@pytest.mark.parametrize("reqs", [1, 160])
@pytest.mark.parametrize("x", [3.0, 7.0, 24.0, 40.0])
@pytest.mark.parametrize("span", [60, 40, 33])
@pytest.mark.parametrize("order", [(0, 1), (1, 0), (0, 0, 1, 0), (1, 0, 0, 0, 0, 1, 0)])
def test_value_scales_do_not_weigh_the_sum(rows, reqs, x, span, order):
    """Page 0 has value scale 2^-span, page 1 2^span; every key scores 0 but one of page 1, x (base 2). The
    tokens of both count alike in the sum, whatever their values' scales are."""
    n, G = 128 * len(order) + rows, 8
    cache = KV8Cache.empty(3, 1)
    g = torch.Generator("cuda").manual_seed(3)
    cache.k_scale.fill_(1.0)
    cache.v_data.copy_(torch.randint(0x20, 0x48, cache.v_data.shape, dtype=torch.uint8, device="cuda", generator=g))
    cache.v_scale[0], cache.v_scale[1], cache.v_scale[2] = 2.0 ** -span, 2.0 ** span, 1.0
    cache.k_data[1, 0, 17, 0] = ONE
    q = torch.zeros((reqs * rows, G, 128), device="cuda")
    q[:, :, 0] = x
    batch, lens, indptr, table = _batch(reqs, n, rows, G, q.to(torch.float8_e4m3fn).view(torch.uint8), list(order) + [2])
    att = KV8Attention(cache, batch, sm_scale=math.log(2.0))
    out = att.attend()
    assert att.errors() == 0
    qv = batch.q.view(torch.float8_e4m3fn).double().view(-1, 1, G, 128)
    one = _kv8.attend(qv[:rows], cache, lens[:1], indptr[:2], table[:1], sm_scale=math.log(2.0))
    _assert_attends(out, att.lse, [t.repeat(reqs, *[1] * (t.dim() - 1)) for t in one])


@pytest.mark.parametrize("rows", [1, 8, 16])
@pytest.mark.parametrize("zero", [[0], [5], [0, 1, 2, 9], list(range(10))])
@pytest.mark.parametrize("reqs", [1, 40])
@pytest.mark.parametrize("level", [-18, 20])
def test_pages_of_scale_zero(rows, zero, reqs, level):
    """A page whose value scale is 0 counts in the sum alone; the weights of the others keep their bits
    however small or large their values' scale is."""
    n, G = 1280 + rows, 8
    kd, ks = _kv8.fill(11, 1, 5)
    vd, vs = _kv8.fill(11, 1, 6)
    vs *= 2.0 ** level
    vs[zero] = 0.0
    cache = KV8Cache(kd, ks, vd, vs)
    g = torch.Generator("cuda").manual_seed(rows)
    q = torch.randn((reqs * rows, G, 128), device="cuda", generator=g).to(torch.bfloat16)
    batch, lens, indptr, table = _batch(reqs, n, rows, G, q)
    att = KV8Attention(cache, batch)
    out = att.attend()
    assert att.errors() == 0
    _assert_attends(out, att.lse, _kv8.attend(q.double().view(-1, 1, G, 128), cache, lens, indptr, table))


@pytest.mark.parametrize("rows", [1, 8, 16])
def test_small_elements_of_a_bf16_query(rows):
    """A row with one large element and 127 small ones, each at the worst place of the split into two E4M3
    rows: half their smallest step, 2^-10 with the largest element at 225, at most 2^-17.8 of the
    largest. Keys see the small ones alone, so that a score is off by up to 127 times that; the
    rest of its error is that of _kv8.attend."""
    n, G = 128 + rows, 8
    cache = KV8Cache.empty(2, 1)
    g = torch.Generator("cuda").manual_seed(rows)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    cache.v_data.copy_(torch.randint(0x30, 0x39, cache.v_data.shape, dtype=torch.uint8, device="cuda", generator=g))
    cache.k_data[:, :, ::2, 1:] = ONE                         # every other key sums the small elements up
    small = 0.125 * (1 + 2.0 ** -7) * torch.exp2(-torch.arange(G, device="cuda").float())
    q = small[None, :, None].repeat(rows, 1, 128)
    q[:, :, 0] = 225.0
    q = q.to(torch.bfloat16)
    batch, lens, indptr, table = _batch(1, n, rows, G, q)
    att = KV8Attention(cache, batch, sm_scale=1.0)
    out = att.attend()
    assert att.errors() == 0
    want, lse, _, _ = _kv8.attend(q.double().view(rows, 1, G, 128), cache, lens, indptr, table, sm_scale=1.0)
    d = 127 * 225 * 2.0 ** -17.8 + 2.0 ** -16 * 127 * 0.126
    assert bool(((att.lse.double() - lse).abs() <= d + 2.0 ** -18 + 2.0 ** -22 * lse.abs()).all())
    rel = 2.0 ** -11 + 2.0 ** -18 + math.expm1(2 * d)         # the values are positive: sum p |v| is the output
    assert bool(((out.double() - want).abs() <= (2.0 ** -8 + rel * (1 + 2.0 ** -8)) * want + 2.0 ** -20).all())
