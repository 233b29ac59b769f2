"""Measured cases of the operators for long sequences over the 8-bit paged cache.

Kinds of case:
  window    attention to the last `window` tokens and to the first `sinks` ones, for single tokens,
            speculative rows and prompts
  shared    attention of requests whose block tables begin with the same pages, those pages read
            once for all of a group's rows
  weights   the attention weight that every cached token gets, added to what it got before
  evict     sequences cut to their heaviest tokens, moved to pages of their own

`run` computes a case in its plain form, or with the package's own calls where `own` is true.
"""
import math
import random

import torch

own = False

DIM = 128      # head dim
BLOCK = 128    # tokens in a page
E4M3_MAX = 448.0
SCALE = 1.0 / math.sqrt(DIM)
FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------- the cases
def listed():
    heads = dict(kv_heads=4, q_per_kv=8)
    return [
        # one user's next token far into a long context: latency counts
        dict(name="window_token_32k", kind="window", reqs=1, min_len=32768, max_len=32768, rows=1, q="e4m3", window=4096,
             sinks=4, shape=1, **heads),
        # a serving step: ragged contexts, shorter and longer than the window, one to eight speculative rows
        dict(name="window_ragged_64", kind="window", reqs=64, min_len=512, max_len=65536, rows=8, q="bf16", window=4096,
             sinks=4, shape=2, **heads),
        # a chunk of a long prompt at odd sizes: matrix products bound it
        dict(name="window_prompt_2k_of_16k", kind="window", reqs=1, min_len=16421, max_len=16421, rows=2053, q="bf16",
             window=4096, sinks=4, shape=3, **heads),
        # four samples of one prompt, some tokens each
        dict(name="shared_samples_4", kind="shared", groups=1, members=4, min_prefix=4000, max_prefix=4100, min_own=1,
             max_own=200, rows=1, q="e4m3", shape=4, **heads),
        # many beams of one long prompt
        dict(name="shared_beams_64", kind="shared", groups=1, members=64, min_prefix=16384, max_prefix=16384, min_own=1,
             max_own=256, rows=1, q="bf16", shape=5, **heads),
        # users of four long system prompts, each with a conversation of its own and speculative rows
        dict(name="shared_prompts_4x16", kind="shared", groups=4, members=16, min_prefix=8192, max_prefix=32768,
             min_own=64, max_own=4096, rows=8, q="bf16", shape=6, **heads),
        # one user's next token: latency counts
        dict(name="weights_token_4k", kind="weights", reqs=1, min_len=4096, max_len=4096, rows=1, q="e4m3", shape=7,
             **heads),
        # a serving step of ragged contexts: the keys' bytes bound it
        dict(name="weights_ragged_64", kind="weights", reqs=64, min_len=512, max_len=65536, rows=8, q="bf16", shape=8,
             **heads),
        # a chunk of a long prompt: matrix products and exponentials bound it
        dict(name="weights_prompt_2k_of_16k", kind="weights", reqs=1, min_len=16421, max_len=16421, rows=2053, q="bf16",
             shape=9, **heads),
        # one sequence that has reached its limit: latency counts
        dict(name="evict_one_5k", kind="evict", parents=1, min_len=5000, max_len=5000, keep=2048, sinks=4, recent=256,
             kv_heads=4, shape=10),
        # a few sequences at odd lengths, eight KV heads
        dict(name="evict_heads_8", kind="evict", parents=6, min_len=4000, max_len=12000, keep=1999, sinks=1, recent=333,
             kv_heads=8, shape=11),
        # a server's long sequences cut down together
        dict(name="evict_ragged_32", kind="evict", parents=32, min_len=12288, max_len=65536, keep=8192, sinks=4,
             recent=1024, kv_heads=4, shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["window", "shared", "weights", "evict"])
    shape = rng.randrange(1 << 20)
    if kind == "evict":
        parents = _log_int(rng, 1, 24)
        max_len = _log_int(rng, 2, 32768)
        keep = _log_int(rng, 1, max(1, min(8192, max_len)))
        sinks = min(keep, rng.choice([0, 1, 4, 130]))
        return dict(kind=kind, parents=parents, min_len=max(1, max_len // rng.choice([1, 2, 16])), max_len=max_len,
                    keep=keep, sinks=sinks, recent=rng.randint(0, keep - sinks), kv_heads=rng.choice([1, 2, 4, 4, 8]),
                    shape=shape)
    kv_heads, q_per_kv = rng.choice([(4, 8), (4, 8), (8, 4), (2, 16), (1, 8), (8, 1), (3, 5), (5, 7)])
    common = dict(kind=kind, kv_heads=kv_heads, q_per_kv=q_per_kv, q=rng.choice(["e4m3", "bf16"]), shape=shape)
    if kind == "shared":
        groups, members = rng.randint(1, 4), _log_int(rng, 2, 32)
        max_prefix = _log_int(rng, 128, 16384)
        return dict(groups=groups, members=members, min_prefix=max(1, max_prefix // rng.choice([1, 2, 8])),
                    max_prefix=max_prefix, min_own=1, max_own=_log_int(rng, 1, 1500), rows=rng.choice([1, 1, 2, 3, 8]),
                    **common)
    if kind == "window":
        common.update(window=_log_int(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 64, 130]))
    if rng.random() < 0.3:        # prompts
        max_len = _log_int(rng, 16, 12000)
        return dict(reqs=rng.randint(1, 3), min_len=max(1, max_len // 2), max_len=max_len,
                    rows=min(max_len, _log_int(rng, 9, 1500)), **common)
    least = 2 if kind == "weights" else 1          # (a single token gets all the weight there is)
    max_len = _log_int(rng, least, 32768)
    reqs = max(1, min(_log_int(rng, 1, 64), (1 << 20) // (max_len * kv_heads) + 1))
    return dict(reqs=reqs, min_len=max(least, max_len // rng.choice([1, 2, 64])), max_len=max_len,
                rows=rng.choice([1, 1, 2, 3, 4, 8]), **common)


def _pages_of(n):
    return (n + BLOCK - 1) // BLOCK


def _lengths(case):
    """(context length, rows) of each request, a function of the case alone."""
    rng = random.Random(case["shape"])
    got = []
    for _ in range(case["reqs"]):
        n = _log_int(rng, case["min_len"], case["max_len"])
        most = min(n, case["rows"])
        if case["rows"] > 8:       # prompts: most of what is not in the cache yet
            r = rng.randint(max(1, most // 2), most) if case["reqs"] > 1 else most
        else:
            r = rng.randint(1, most) if case["rows"] == 8 else most
        got.append((n, r))
    return got


def _groups(case):
    """[(shared pages, [(context length, rows) of each member])], a function of the case alone."""
    rng = random.Random(case["shape"])
    got = []
    for _ in range(case["groups"]):
        pages = _log_int(rng, case["min_prefix"], case["max_prefix"]) // BLOCK
        members = []
        for _ in range(case["members"]):
            r = rng.randint(1, case["rows"]) if case["rows"] == 8 else case["rows"]
            members.append((pages * BLOCK + max(r, _log_int(rng, case["min_own"], case["max_own"])), r))
        got.append((pages, members))
    return got


def _parents(case):
    rng = random.Random(case["shape"])
    return [_log_int(rng, case["min_len"], case["max_len"]) for _ in range(case["parents"])]


# ------------------------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _plane(pages, heads, gen, outliers):
    """Codes and scales of a filled 8-bit plane, as the append leaves them: normal values, a few strong
    channels for keys, the level changing from page to page; the scale a power of two."""
    codes = torch.empty((pages, heads, BLOCK, DIM), dtype=torch.uint8, device="cuda")
    scale = torch.empty((pages, heads), dtype=torch.float32, device="cuda")
    for p0 in range(0, pages, 2048):
        n = min(2048, pages - p0)
        x = torch.randn((n, heads, BLOCK, DIM), device="cuda", generator=gen)
        x *= torch.exp2(torch.rand((n, heads, 1, 1), device="cuda", generator=gen) - 0.5)
        if outliers:
            x[..., 5::31] *= 3.0
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / E4M3_MAX)))
        codes[p0:p0 + n] = (x / s[:, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(FP8).view(torch.uint8)
        scale[p0:p0 + n] = s
    return codes, scale


def _cache_planes(pages, heads, gen):
    k, ks = _plane(pages, heads, gen, True)
    v, vs = _plane(pages, heads, gen, False)
    return {"k_data": k, "k_scale": ks, "v_data": v, "v_scale": vs}


def _tables(counts, width, total, seed):
    """A block table int32 [B, width] over a shuffled pool of `total` pages (counts[b] pages each)."""
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, perm, at


def _prepare_batch(case, st, seed, gen):
    """Requests, their queries, and where each row sits among them."""
    shared = case["kind"] == "shared"
    if shared:
        groups = _groups(case)
        lens, rows = zip(*[m for _, members in groups for m in members])
        counts = [_pages_of(n) - p for p, members in groups for n, _ in members] + [p for p, _ in groups]
    else:
        lens, rows = zip(*_lengths(case))
        counts = [_pages_of(n) for n in lens]
    width = max(_pages_of(n) for n in lens)
    table, perm, pages = _tables(counts, width, sum(counts), seed)
    if shared:                    # a member's row: its group's pages, then its own
        m, every = case["members"], table
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        for b in range(len(lens)):
            g, p = b // m, groups[b // m][0]
            table[b, :p] = every[len(lens) + g, :p]
            table[b, p:_pages_of(lens[b])] = every[b, :_pages_of(lens[b]) - p]
        st["prefix"] = [p for p, _ in groups]
        st["group_indptr"] = _ints([g * m for g in range(len(groups) + 1)])
    indptr = [0]
    for r in rows:
        indptr.append(indptr[-1] + r)
    total, heads = indptr[-1], case["kv_heads"]
    st.update(lens=lens, rows=rows, indptr=indptr, table=table.cuda(), context_lens=_ints(lens), q_indptr=_ints(indptr))
    st["row_req"] = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(rows)).cuda()
    st["row_at"] = (torch.arange(total, device="cuda") - st["q_indptr"].long()[st["row_req"]])
    st["planes"] = _cache_planes(pages, heads, gen)
    q = torch.randn((total, heads * case["q_per_kv"], DIM), device="cuda", generator=gen) * 1.5
    st["q"] = q.to(FP8).view(torch.uint8) if case["q"] == "e4m3" else q.to(torch.bfloat16)


def prepare(case, seed):
    gen = _gen(seed)
    kind = case["kind"]
    st = {"case": case}
    if kind == "evict":
        lens, heads = _parents(case), case["kv_heads"]
        n = len(lens)
        counts = [_pages_of(m) for m in lens]
        spare = sum(_pages_of(min(m, case["keep"])) for m in lens) + 3
        width = max(counts)
        total = sum(counts) + spare
        table, perm, at = _tables(counts + [0] * n, width, total, seed)
        refs = torch.zeros(total, dtype=torch.int32)
        refs[perm[:at].long()] = 1
        st["planes"] = _cache_planes(total, heads, gen)
        st["table"], st["refs"], st["seq_lens"] = table.cuda(), refs.cuda(), _ints(lens + [0] * n)
        st["parents"], st["children"] = _ints(list(range(n))), _ints(list(range(n, 2 * n)))
        # a few tokens have most of the weight, a few have none at all
        w = torch.exp(torch.randn((2 * n, heads, width * BLOCK), device="cuda", generator=gen) * 2.5)
        w *= torch.rand((2 * n, heads, width * BLOCK), device="cuda", generator=gen) > 0.1
        st["weights"] = w
        st["lens"] = lens
    else:
        _prepare_batch(case, st, seed, gen)
        if kind == "weights":
            shape = (len(st["lens"]), case["kv_heads"], st["table"].shape[1] * BLOCK)
            st["old"] = torch.exp(torch.randn(shape, device="cuda", generator=gen))
            st["new"] = torch.zeros(shape, device="cuda")
            st["lse"] = _lse(st)      # what the attention of the same step returned
    if own:
        import block_sparse_attention_nvfp4_gb300 as msa
        st["cache"] = msa.KV8Cache(**st["planes"])
        if kind == "evict":
            st["pool"] = msa.PagePool([st["cache"]], st["seq_lens"], st["table"], st["refs"])
        else:
            st["batch"] = msa.KV8Batch(st["context_lens"], st["q_indptr"], st["table"], st["q"],
                                       total_rows=st["indptr"][-1], max_rows_per_req=max(st["rows"]))
            st["attention"] = msa.KV8Attention(st["cache"], st["batch"], with_weights=kind == "weights",
                                               max_groups=case["groups"] if kind == "shared" else 0)
    return st


# ------------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "window":
        if own:
            out = st["attention"].attend(window=case["window"], sinks=case["sinks"])
            return {"out": out, "lse": st["attention"].lse}
        return _window(st)
    if kind == "shared":
        if own:
            out = st["attention"].attend_shared(st["group_indptr"])
            return {"out": out, "lse": st["attention"].lse}
        return _shared(st)
    if kind == "weights":
        if own:
            st["attention"].add_weights(st["old"], st["new"], lse=st["lse"])
        else:
            _weights(st)
        return st["new"]
    if own:
        st["pool"].evict(st["parents"], st["children"], st["weights"], keep=case["keep"], sinks=case["sinks"],
                         recent=case["recent"])
        st["pool"].free(st["children"])
    else:
        _evict(st)
    p = st["planes"]
    return {"k": p["k_data"].view(FP8), "k_scale": p["k_scale"], "v": p["v_data"].view(FP8), "v_scale": p["v_scale"],
            "weights": st["weights"], "table": st["table"], "refs": st["refs"], "seq_lens": st["seq_lens"]}


def _queries(st):
    """Queries padded to [B, KV heads, queries a head, most rows, 128]."""
    case = st["case"]
    H, G = case["kv_heads"], case["q_per_kv"]
    q = (st["q"].view(FP8) if case["q"] == "e4m3" else st["q"]).float()
    padded = q.new_zeros((len(st["lens"]), max(st["rows"]), H, G, DIM))
    padded[st["row_req"], st["row_at"]] = q.view(-1, H, G, DIM)
    return padded.permute(0, 2, 3, 1, 4)


def _rows(st, x):
    """[B, H, G, most rows, ..] back to [rows, H G, ..]."""
    x = x.permute(0, 3, 1, 2, *range(4, x.dim()))[st["row_req"], st["row_at"]]
    return x.flatten(1, 2)


def _gather(st, name, table, pos):
    """Values of the tokens at positions pos [B, n] of the rows of `table`: [B, H, n, 128]."""
    page = torch.gather(table.long(), 1, pos // BLOCK)
    x = st["planes"][name + "_data"].view(FP8)[page, :, pos % BLOCK].float()
    x *= st["planes"][name + "_scale"][page][..., None]
    return x.transpose(1, 2)


def _row_pos(st):
    """Positions of the padded rows [B, most rows]."""
    n, r = st["context_lens"].long(), (st["q_indptr"][1:] - st["q_indptr"][:-1]).long()
    return (n - r)[:, None] + torch.arange(max(st["rows"]), device="cuda")


def _scores(st, q, k):
    """sm_scale q k: [B, H, G, rows, keys]."""
    B, H, G, R, _ = q.shape
    return torch.matmul(q.reshape(B, H, G * R, DIM), k.transpose(2, 3)).mul_(SCALE).view(B, H, G, R, k.shape[2])


def _finish(st, s, values):
    """Softmax of s over its last axis, and its products with the values' parts [(first key, last key, v)]."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    e = s.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    B, H, G, R, _ = e.shape
    o = sum(torch.matmul(e[..., a:b].reshape(B, H, G * R, b - a), v).view(B, H, G, R, DIM) for a, b, v in values) / l
    return {"out": _rows(st, o).to(torch.bfloat16), "lse": _rows(st, m + l.log()).squeeze(-1)}


def _window(st):
    case = st["case"]
    W, S = case["window"], case["sinks"]
    n, pos_r = st["context_lens"].long(), _row_pos(st)
    # the first tokens, and those of the windows of a request's rows
    first = (pos_r[:, :1] - W + 1).clamp(min=S)
    most = max(m - max(S, m - r - W + 1) for m, r in zip(st["lens"], st["rows"]))
    sinks = torch.arange(min(S, max(st["lens"])), device="cuda").expand(len(st["lens"]), -1)
    pos = torch.cat([sinks, first + torch.arange(max(0, most), device="cuda")], 1)
    held = pos < n[:, None]
    pos = torch.where(held, pos, 0)
    k, v = _gather(st, "k", st["table"], pos), _gather(st, "v", st["table"], pos)
    see = held[:, None] & (pos[:, None] <= pos_r[..., None]) & ((pos[:, None] > pos_r[..., None] - W) | (pos[:, None] < S))
    s = _scores(st, _queries(st), k).masked_fill_(~see[:, None, None], -math.inf)
    return _finish(st, s, [(0, pos.shape[1], v)])


def _shared(st):
    case = st["case"]
    m, H, G = case["members"], case["kv_heads"], case["q_per_kv"]
    n, pos_r, q = st["context_lens"].long(), _row_pos(st), _queries(st)
    pages = torch.tensor(st["prefix"], device="cuda")
    B, R, N = q.shape[0], q.shape[3], len(st["prefix"])
    # the groups' first pages, for all rows of a group at once
    pos = torch.arange(max(st["prefix"]) * BLOCK, device="cuda").expand(N, -1)
    held = pos < pages[:, None] * BLOCK
    pos = torch.where(held, pos, 0)
    front = st["table"][::m]
    k, v = _gather(st, "k", front, pos), _gather(st, "v", front, pos)
    qg = q.reshape(N, m, H, G, R, DIM).permute(0, 2, 3, 1, 4, 5).reshape(N, H, G, m * R, DIM)
    s0 = _scores(st, qg, k).masked_fill_(~held[:, None, None, None], -math.inf)
    s0 = s0.view(N, H, G, m, R, s0.shape[-1]).permute(0, 3, 1, 2, 4, 5).reshape(B, H, G, R, s0.shape[-1])
    # every member's own tokens
    first = pages.repeat_interleave(m) * BLOCK
    most = max(x - p * BLOCK for x, p in zip(st["lens"], [p for p in st["prefix"] for _ in range(m)]))
    own_pos = first[:, None] + torch.arange(most, device="cuda")
    held = own_pos < n[:, None]
    own_pos = torch.where(held, own_pos, 0)
    k1, v1 = _gather(st, "k", st["table"], own_pos), _gather(st, "v", st["table"], own_pos)
    see = held[:, None] & (own_pos[:, None] <= pos_r[..., None])
    s1 = _scores(st, q, k1).masked_fill_(~see[:, None, None], -math.inf)
    # one softmax over both parts; the weights of the first meet the group's values
    top = torch.maximum(s0.amax(-1, keepdim=True) if s0.shape[-1] else s1.amax(-1, keepdim=True), s1.amax(-1, keepdim=True))
    top = torch.where(top > -math.inf, top, 0.0)
    e0, e1 = s0.sub_(top).exp_(), s1.sub_(top).exp_()
    l = e0.sum(-1, keepdim=True) + e1.sum(-1, keepdim=True)
    o = torch.matmul(e1.view(B, H, G * R, -1), v1).view(B, H, G, R, DIM)
    e0 = e0.view(N, m, H, G, R, e0.shape[-1]).permute(0, 2, 1, 3, 4, 5).reshape(N, H, m * G * R, e0.shape[-1])
    o0 = torch.matmul(e0, v).view(N, H, m, G, R, DIM).permute(0, 2, 1, 3, 4, 5).reshape(B, H, G, R, DIM)
    return {"out": _rows(st, (o + o0) / l).to(torch.bfloat16), "lse": _rows(st, top + l.log()).squeeze(-1)}


def _all_scores(st):
    """Scores of the padded rows against all tokens, -inf where a row does not see one."""
    n, pos_r = st["context_lens"].long(), _row_pos(st)
    pos = torch.arange(max(st["lens"]), device="cuda").expand(len(st["lens"]), -1)
    held = pos < n[:, None]
    k = _gather(st, "k", st["table"], torch.where(held, pos, 0))
    see = held[:, None] & (pos[:, None] <= pos_r[..., None])
    return _scores(st, _queries(st), k).masked_fill_(~see[:, None, None], -math.inf)


def _lse(st):
    return _rows(st, torch.logsumexp(_all_scores(st), -1)).contiguous()


def _weights(st):
    case = st["case"]
    H, G = case["kv_heads"], case["q_per_kv"]
    s = _all_scores(st)
    lse = s.new_full((s.shape[0], s.shape[3], H, G), math.inf)     # rows that are not there add nothing
    lse[st["row_req"], st["row_at"]] = st["lse"].view(-1, H, G)
    w = s.sub_(lse.permute(0, 2, 3, 1)[..., None]).exp_().sum((2, 3))
    N = s.shape[-1]
    n, r = st["context_lens"].long(), (st["q_indptr"][1:] - st["q_indptr"][:-1]).long()
    pos = torch.arange(N, device="cuda")
    old = torch.where((pos < (n - r)[:, None])[:, None], st["old"][..., :N], 0.0)
    st["new"][..., :N] = torch.where((pos < n[:, None])[:, None], old + w, st["new"][..., :N])


def _evict(st):
    case = st["case"]
    keep, S, recent = case["keep"], case["sinks"], case["recent"]
    lens, table, refs, weights = st["seq_lens"], st["table"], st["refs"], st["weights"]
    par, child = st["parents"].long(), st["children"].long()
    n = lens[par].long()
    kept = n.clamp(max=keep)
    most = max(min(m, keep) for m in st["lens"])
    # the tokens in the order of their claims: first and last ones, then by weight, ties to the lower position
    N = max(st["lens"])
    pos = torch.arange(N, device="cuda")
    w = weights[par][..., :N]
    must = (pos < S) | (pos >= (n - recent)[:, None])
    rank = torch.where(must[:, None], math.inf, w).masked_fill_((pos >= n[:, None])[:, None], -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :most]
    at = torch.arange(most, device="cuda")
    here = at < kept[:, None]                                            # [n, most]
    src = torch.where(here[:, None], order, N).sort(-1).values           # in the order of their positions
    src = torch.where(here[:, None], src, 0)                             # [n, H, most]
    # pages of their own, the lowest free ones in list order
    need = (kept + BLOCK - 1) // BLOCK
    col = torch.arange(table.shape[1], device="cuda")
    fresh = col < need[:, None]
    free = (refs == 0).nonzero().squeeze(1)[:int(need.sum())]
    rows = table[child]
    rows[fresh] = free.to(torch.int32)
    table[child] = rows
    # what moves
    H = weights.shape[1]
    heads = torch.arange(H, device="cuda")[:, None]
    page = torch.gather(table[par].long()[:, None].expand(-1, H, -1), 2, src // BLOCK)
    pad = -most % BLOCK
    to = torch.where(fresh, rows.long(), 0)[:, :(most + pad) // BLOCK]   # [n, new pages]
    there = fresh[:, :(most + pad) // BLOCK]
    for name in ("k", "v"):
        data, scale = st["planes"][name + "_data"], st["planes"][name + "_scale"]
        old = torch.where(here[:, None], scale[page, heads], 0.0)        # [n, H, most]
        new = torch.nn.functional.pad(old, (0, pad)).view(*old.shape[:2], -1, BLOCK).amax(-1)
        ratio = old / new.repeat_interleave(BLOCK, -1)[..., :most]
        codes = (data.view(FP8)[page, heads, src % BLOCK].float() * ratio[..., None]).to(FP8).view(torch.uint8)
        entry, head, slot = (here[:, None].expand(-1, H, -1)).nonzero(as_tuple=True)
        data[to[entry, slot // BLOCK], head, slot % BLOCK] = codes[entry, head, slot]
        scale[to[there]] = new.permute(0, 2, 1)[there]
    moved = torch.gather(w, 2, src)
    weights[child, :, :most] = torch.where(here[:, None], moved, weights[child, :, :most])
    # (the children have ended again: their pages' counts and their lengths are what they were)


# ------------------------------------------------------------------------------- floors
def work(case):
    kind = case["kind"]
    H = case["kv_heads"]
    if kind == "evict":
        lens = _parents(case)
        kept = [min(n, case["keep"]) for n in lens]
        per = H * 2 * DIM * 2 + H * 4                   # a token's codes read and written, its weight written
        pages = sum(_pages_of(k) for k in kept)
        return {"bytes": sum(lens) * H * 4 + sum(kept) * per + pages * (H * 16 + 8) + sum(4 * _pages_of(n) for n in lens),
                "flops": sum(kept) * H * 2 * DIM}
    G, size = case["q_per_kv"], 1 if case["q"] == "e4m3" else 2
    if kind == "shared":
        tokens = pairs = rows = 0
        for p, members in _groups(case):
            tokens += p * BLOCK + sum(n - p * BLOCK for n, _ in members)
            rows += sum(r for _, r in members)
            pairs += sum(n * r - r * (r - 1) // 2 for n, r in members)
        return {"bytes": tokens * H * 2 * DIM + rows * H * G * (DIM * (size + 2) + 4), "flops": 4 * DIM * pairs * H * G}
    tokens = pairs = rows = 0
    for n, r in _lengths(case):
        rows += r
        if kind == "weights":
            tokens += n
            pairs += n * r - r * (r - 1) // 2
        else:
            S, W = case["sinks"], case["window"]
            lo = max(0, n - r - W + 1)
            tokens += n - lo + min(S, lo)
            pairs += sum(p + 1 if p + 1 <= W else W + min(S, p + 1 - W) for p in range(n - r, n))
    if kind == "weights":
        return {"bytes": tokens * H * (DIM + 8) + rows * H * G * (DIM * size + 4), "flops": 2 * DIM * pairs * H * G}
    return {"bytes": tokens * H * 2 * DIM + rows * H * G * (DIM * (size + 2) + 4), "flops": 4 * DIM * pairs * H * G}


# ------------------------------------------------------------------------------- 64 bits
def _e4m3_values():
    """The 256 values of E4M3 from their bits."""
    got = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if (c & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        got.append(-v if c & 128 else v)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _round_e4m3(x):
    """The E4M3 value nearest to x, ties to the even code, saturating (64 bits)."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=E4M3_MAX), x)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _exact_evict(case, st) if case["kind"] == "evict" else _exact_rows(case, st)


def _exact_rows(case, st):
    """Every request and head by itself, over the keys that any of its rows sees."""
    value = _e4m3_values()
    H, G, p = case["kv_heads"], case["q_per_kv"], st["planes"]
    q = value[st["q"].long()] if case["q"] == "e4m3" else st["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    new = st["new"].double() if case["kind"] == "weights" else None
    for b, (n, r) in enumerate(zip(st["lens"], st["rows"])):
        r0 = st["indptr"][b]
        t = torch.arange(n, device="cuda")
        if case["kind"] == "window":
            t = t[(t < case["sinks"]) | (t > n - r - case["window"])]
        page, slot = st["table"][b].long()[t // BLOCK], t % BLOCK
        for h in range(H):
            k = value[p["k_data"][page, h, slot].long()] * p["k_scale"][page, h].double()[:, None]
            v = value[p["v_data"][page, h, slot].long()] * p["v_scale"][page, h].double()[:, None]
            for a in range(0, r, 512):
                at = torch.arange(n - r + a, min(n, n - r + a + 512), device="cuda")[:, None]
                rows = slice(r0 + a, r0 + a + at.shape[0])
                see = t <= at
                if case["kind"] == "window":
                    see &= (t > at - case["window"]) | (t < case["sinks"])
                for g in range(h * G, (h + 1) * G):
                    z = torch.where(see, (q[rows, g] @ k.T) / math.sqrt(DIM), -math.inf)
                    if new is None:
                        y = torch.logsumexp(z, 1)
                        lse[rows, g] = y
                        out[rows, g] = torch.exp(z - y[:, None]) @ v
                    else:
                        if a == 0 and g == h * G:
                            new[b, h, :n] = torch.where(t < n - r, st["old"][b, h, :n].double(), 0.0)
                        new[b, h, :n] += torch.exp(z - st["lse"][rows, g].double()[:, None]).sum(0)
    return new if new is not None else {"out": out, "lse": lse}


def _exact_evict(case, st):
    value = _e4m3_values()
    planes = {n: (value[st["planes"][n + "_data"].long()], st["planes"][n + "_scale"].double()) for n in ("k", "v")}
    weights = st["weights"].double()
    free = [i for i, r in enumerate(st["refs"].tolist()) if r == 0]
    n_par = len(st["lens"])
    for b, n in enumerate(st["lens"]):
        keep = min(n, case["keep"])
        ids, free = free[:_pages_of(keep)], free[_pages_of(keep):]
        for h in range(case["kv_heads"]):
            t = torch.arange(n, device="cuda")
            if n > keep:
                must = (t < case["sinks"]) | (t >= n - case["recent"])
                w = st["weights"][b, h, :n]
                rest = t[~must]
                # by weight, then by position (weights are single precision: a pair is one number of 64 bits)
                key = w[rest].view(torch.int32).long() * (1 << 20) + ((1 << 20) - 1 - rest)
                m = keep - int(must.sum())
                t = torch.cat([t[must], rest[key.topk(m).indices] if m else rest[:0]]).sort().values
            weights[n_par + b, h, :keep] = st["weights"][b, h, t].double()
            for vals, scale in planes.values():
                page = st["table"][b].long()[t // BLOCK]
                x, s = vals[page, h, t % BLOCK], scale[page, h]
                for i, p in enumerate(ids):
                    part = slice(i * BLOCK, min(keep, (i + 1) * BLOCK))
                    top = s[part].max()
                    m = part.stop - part.start
                    vals[p, h, :m] = _round_e4m3(x[part] * (s[part] / top)[:, None])
                    scale[p, h] = top
    return {"k": planes["k"][0], "k_scale": planes["k"][1], "v": planes["v"][0], "v_scale": planes["v"][1],
            "weights": weights, "table": None, "refs": None, "seq_lens": None}
