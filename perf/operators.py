"""Measured cases of the 8-bit cache operators and of the page operators.

Kinds of case:
  attend    attention over the paged 8-bit cache (E4M3 codes, one FP32 scale for each page and KV
            head): single tokens, speculative rows, chosen blocks, prompts
  append    new tokens' K and V quantised into their pages of the 8-bit cache
  copy      pages, or their first tokens, copied within the caches
  fork      sequences forked, grown by some tokens, and freed again
  compact   live pages moved to the front of the pool, block tables rewritten

`run` computes a case in its plain form, or with the package's own calls where `own` is true.
"""
import math
import random

import torch

own = False

DIM = 128      # head dim
BLOCK = 128    # tokens in a page
E4M3_MAX = 448.0
MIN_EXP = -60  # smallest exponent of an appended page's scale
FP8 = torch.float8_e4m3fn

# page planes of the NVFP4 cache: (strips, bytes of a token in a strip)
NVFP4_PLANES = (("k_data", 4, 64), ("k_scale", 4, 8), ("v_data", 4, 64), ("v_scale", 4, 8),
                ("ki_data", 1, 64), ("ki_scale", 1, 8))


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one user's next token at the smallest context of the repository's workloads: latency counts
        dict(name="attend_token_4k", kind="attend", reqs=1, min_len=4096, max_len=4096, rows=1, kv_heads=4, q_per_kv=8,
             q="e4m3", blocks=0, shape=1),
        # a serving step: ragged contexts, one to eight speculative rows each, BF16 queries
        dict(name="attend_ragged_64", kind="attend", reqs=64, min_len=512, max_len=65536, rows=8, kv_heads=4, q_per_kv=8,
             q="bf16", blocks=0, shape=4),
        # the sparse step: the 16 blocks that the indexer chose for each group, 8 speculative rows
        dict(name="attend_blocks_16x32k", kind="attend", reqs=16, min_len=32768, max_len=32768, rows=8, kv_heads=4,
             q_per_kv=8, q="e4m3", blocks=16, shape=2),
        # a chunk of a long prompt at odd sizes: matrix products bound it
        dict(name="attend_prompt_2k_of_16k", kind="attend", reqs=1, min_len=16421, max_len=16421, rows=2053, kv_heads=4,
             q_per_kv=8, q="bf16", blocks=0, shape=3),
        # one new token for each sequence of a large batch
        dict(name="append_step_256", kind="append", reqs=256, min_len=1, max_len=512, rows=1, kv_heads=4, src="bf16",
             shape=5),
        # ragged prompts, the first page of each partly filled
        dict(name="append_prompts_8", kind="append", reqs=8, min_len=4000, max_len=12000, rows=12000, kv_heads=4,
             src="bf16", shape=6),
        # copy-on-write of a few tails
        dict(name="copy_tails_8", kind="copy", pages=64, pairs=8, cache="nvfp4", kv_heads=4, partial=True, shape=7),
        # a large part of the cache duplicated
        dict(name="copy_pages_1024", kind="copy", pages=4096, pairs=1024, cache="kv8", kv_heads=4, partial=False,
             shape=8),
        # four samples of one prompt
        dict(name="fork_samples_4", kind="fork", pages=512, parents=1, children=4, min_len=4000, max_len=4100, grow=8,
             cache="nvfp4", kv_heads=4, shape=9),
        # many beams of several long prompts
        dict(name="fork_beams_256", kind="fork", pages=4096, parents=16, children=256, min_len=8000, max_len=24000,
             grow=200, cache="kv8", kv_heads=4, shape=10),
        # a small pool after a few requests ended
        dict(name="compact_256", kind="compact", pages=256, seqs=16, live=60, cache="nvfp4", kv_heads=4, shape=11),
        # a large pool, half of it live
        dict(name="compact_4096", kind="compact", pages=4096, seqs=96, live=50, cache="kv8", kv_heads=4, shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "append", "copy", "fork", "compact"])
    shape = rng.randrange(1 << 20)
    if kind == "attend":
        kv_heads, q_per_kv = rng.choice([(4, 8), (4, 8), (8, 4), (2, 16), (1, 8), (8, 1), (3, 5), (5, 7)])
        q = rng.choice(["e4m3", "bf16"])
        form = rng.choice(["decode", "decode", "blocks", "prompt"])
        if form == "prompt":
            max_len = _log_int(rng, 16, 12000)
            return dict(kind=kind, reqs=rng.randint(1, 3), min_len=max(1, max_len // 2), max_len=max_len,
                        rows=min(max_len, _log_int(rng, 9, 1500)), kv_heads=kv_heads, q_per_kv=q_per_kv, q=q, blocks=0,
                        shape=shape)
        max_len = _log_int(rng, 1, 32768)
        reqs = max(1, min(_log_int(rng, 1, 64), (1 << 20) // (max_len * kv_heads) + 1))
        return dict(kind=kind, reqs=reqs, min_len=max(1, max_len // rng.choice([1, 2, 64])), max_len=max_len,
                    rows=rng.choice([1, 1, 2, 3, 4, 8]), kv_heads=kv_heads, q_per_kv=q_per_kv, q=q,
                    blocks=rng.choice([4, 16, 32]) if form == "blocks" else 0, shape=shape)
    if kind == "append":
        rows = rng.choice([1, 1, 3, 8, _log_int(rng, 9, 8000)])
        reqs = _log_int(rng, 1, 200) if rows <= 8 else rng.randint(1, 6)
        return dict(kind=kind, reqs=reqs, min_len=1, max_len=max(rows, _log_int(rng, 64, 600)), rows=rows,
                    kv_heads=rng.choice([1, 2, 4, 4, 5, 8]), src=rng.choice(["bf16", "fp16", "fp32"]), shape=shape)
    cache = rng.choice(["nvfp4", "kv8"])
    kv_heads = 4 if cache == "nvfp4" else rng.choice([1, 4, 8])
    if kind == "copy":
        pages = _log_int(rng, 16, 2000)
        return dict(kind=kind, pages=pages, pairs=rng.randint(1, pages // 3), cache=cache, kv_heads=kv_heads,
                    partial=rng.random() < 0.5, shape=shape)
    if kind == "fork":
        parents = rng.randint(1, 8)
        max_len = _log_int(rng, 2, 16000)
        return dict(kind=kind, pages=2048, parents=parents, children=_log_int(rng, 1, 128), min_len=max(1, max_len // 2),
                    max_len=max_len, grow=rng.choice([1, 8, 130, 300]), cache=cache, kv_heads=kv_heads, shape=shape)
    return dict(kind=kind, pages=_log_int(rng, 16, 2000), seqs=_log_int(rng, 1, 64), live=rng.randint(5, 95),
                cache=cache, kv_heads=kv_heads, shape=shape)


def _lengths(case):
    """(context length, rows) of each request, a function of the case alone."""
    rng = random.Random(case["shape"])
    got = []
    for _ in range(case["reqs"]):
        n = _log_int(rng, case["min_len"], case["max_len"])
        most = min(n, case["rows"])
        if case["rows"] > 8:       # prompts: most of what is not in the cache yet
            r = rng.randint(max(1, most // 2), most) if case["reqs"] > 1 else most
        elif case["kind"] == "attend" and case["rows"] == 8 and not case["blocks"]:
            r = rng.randint(1, most)
        else:
            r = most
        got.append((n, r))
    return got


def _parent_lengths(case):
    rng = random.Random(case["shape"])
    return [rng.randint(case["min_len"], case["max_len"]) for _ in range(case["parents"])]


def _pages_of(n):
    return (n + BLOCK - 1) // BLOCK


def _pairs(case):
    """(source page, target page, tokens) of each copy: targets distinct, and none of them a source."""
    rng = random.Random(case["shape"])
    perm = list(range(case["pages"]))
    rng.shuffle(perm)
    n = case["pairs"]
    return [(perm[rng.randrange(n, len(perm))], perm[i], rng.randint(1, BLOCK) if case["partial"] else BLOCK)
            for i in range(n)]


def _page_tables(case):
    """Page lists of a pool's sequences after some have ended: (lengths, lists)."""
    rng = random.Random(case["shape"])
    perm = list(range(case["pages"]))
    rng.shuffle(perm)
    n = max(1, case["pages"] * case["live"] // 100)
    held = perm[:n]
    seqs = min(case["seqs"], n)
    cuts = sorted(rng.sample(range(1, n), seqs - 1)) if seqs > 1 else []
    lists = [held[a:b] for a, b in zip([0] + cuts, cuts + [n])]
    for i in range(1, seqs):       # some share a prefix with the first
        if rng.random() < 0.25:
            lists[i] = lists[0][:rng.randint(1, len(lists[0]))] + lists[i]
    lens = [len(p) * BLOCK - rng.randrange(BLOCK) for p in lists]
    return lens, lists


def _token_bytes(case):
    """Bytes of one token in all planes of a page cache, and bytes kept once for a page."""
    if case["cache"] == "nvfp4":
        return sum(s * b for _, s, b in NVFP4_PLANES), 0
    return 2 * case["kv_heads"] * DIM, 2 * case["kv_heads"] * 4


# ------------------------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tables(lens, seed, spare=0):
    """A shuffled block table over just enough pages: (table int32 [B, M], pages)."""
    need = [_pages_of(n) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.cuda(), total


def _kv8_plane(pages, heads, gen, outliers):
    """Codes and scales of a filled 8-bit plane: normal values, a few strong channels for keys, the
    level changing from page to page; scale = largest magnitude / 448."""
    codes = torch.empty((pages, heads, BLOCK, DIM), dtype=torch.uint8, device="cuda")
    scale = torch.empty((pages, heads), dtype=torch.float32, device="cuda")
    for p0 in range(0, pages, 2048):
        n = min(2048, pages - p0)
        x = torch.randn((n, heads, BLOCK, DIM), device="cuda", generator=gen)
        x *= torch.exp2(torch.rand((n, heads, 1, 1), device="cuda", generator=gen) - 0.5)
        if outliers:
            x[..., 5::31] *= 3.0
        s = x.abs().amax((2, 3)) / E4M3_MAX
        codes[p0:p0 + n] = (x / s[:, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(FP8).view(torch.uint8)
        scale[p0:p0 + n] = s
    return codes, scale


def _random_bytes(shape, gen):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=gen)


def _planes(case, pages, gen):
    """The planes of a page cache by name, filled."""
    if case["cache"] == "nvfp4":
        return {n: _random_bytes((pages, s, BLOCK, b) if s > 1 else (pages, BLOCK, b), gen) for n, s, b in NVFP4_PLANES}
    heads = case["kv_heads"]
    planes = {}
    for n in ("k", "v"):
        planes[n + "_data"] = _random_bytes((pages, heads, BLOCK, DIM), gen) & 0xBF   # finite codes
        planes[n + "_scale"] = torch.rand((pages, heads), device="cuda", generator=gen) + 0.5
    return planes


def _cache_object(case, planes):
    from block_sparse_attention_nvfp4_gb300 import KV8Cache, KVCache
    return KVCache(**planes) if case.get("cache") == "nvfp4" else KV8Cache(**planes)


def prepare(case, seed):
    gen = _gen(seed)
    kind = case["kind"]
    st = {"case": case}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if kind in ("attend", "append"):
        lens, rows = zip(*_lengths(case))
        st["lens"], st["rows"] = lens, rows
        indptr = [0]
        for r in rows:
            indptr.append(indptr[-1] + r)
        st["indptr"] = indptr
        st["table"], pages = _tables(lens, seed)
        st["context_lens"], st["q_indptr"] = ints(lens), ints(indptr)
        heads = case["kv_heads"]
        planes = {}
        planes["k_data"], planes["k_scale"] = _kv8_plane(pages, heads, gen, True)
        planes["v_data"], planes["v_scale"] = _kv8_plane(pages, heads, gen, False)
        st["planes"] = planes
        total = indptr[-1]
        if kind == "attend":
            q = torch.randn((total, heads * case["q_per_kv"], DIM), device="cuda", generator=gen) * 1.5
            st["q"] = q.to(FP8).view(torch.uint8) if case["q"] == "e4m3" else q.to(torch.bfloat16)
            st["ids"] = None
            if case["blocks"]:
                ids = torch.full((len(lens), heads, case["blocks"]), -1, dtype=torch.int32)
                pick = random.Random(seed)
                for b, n in enumerate(lens):
                    nb = _pages_of(n)
                    for h in range(heads):
                        some = sorted(pick.sample(range(nb - 1), min(nb, case["blocks"]) - 1)) + [nb - 1]
                        ids[b, h, :len(some)] = torch.tensor(some, dtype=torch.int32)
                st["ids"] = ids.cuda()
        else:
            dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["src"]]
            level = torch.exp2(torch.rand((total, heads, 1), device="cuda", generator=gen))
            st["k"] = (torch.randn((total, heads, DIM), device="cuda", generator=gen) * level).to(dt)
            st["v"] = (torch.randn((total, heads, DIM), device="cuda", generator=gen) * level).to(dt)
            # pages that are partly filled already carry scales as this operator leaves them
            for n in ("k_scale", "v_scale"):
                planes[n] = torch.exp2(torch.ceil(torch.log2(planes[n])))
    elif kind == "copy":
        st["planes"] = _planes(case, case["pages"], gen)
        src, dst, tokens = zip(*_pairs(case))
        st["src"], st["dst"] = ints(src), ints(dst)
        st["tokens"] = ints(tokens) if case["partial"] else None
        seqs = 1
        st["seq_lens"], st["table"] = ints([0] * seqs), ints([[-1]] * seqs)
        st["refs"] = ints([0] * case["pages"])
    elif kind == "fork":
        lens = _parent_lengths(case)
        P, n, c = case["parents"], case["pages"], case["children"]
        rng = random.Random(case["shape"] + 1)
        of = [rng.randrange(P) for _ in range(c)]
        grown = [lens[p] + case["grow"] for p in of]
        perm = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table = torch.full((P + c, _pages_of(max(lens) + case["grow"])), -1, dtype=torch.int32)
        refs = torch.zeros(n, dtype=torch.int32)
        at = 0
        for b, m in enumerate(lens):
            table[b, :_pages_of(m)] = perm[at:at + _pages_of(m)]
            at += _pages_of(m)
        refs[perm[:at].long()] = 1
        st["planes"] = _planes(case, n, gen)
        st["table"], st["refs"] = table.cuda(), refs.cuda()
        st["seq_lens"] = ints(list(lens) + [0] * c)
        st["parents"], st["children"], st["grown"] = ints(of), ints(list(range(P, P + c))), ints(grown)
    elif kind == "compact":
        lens, lists = _page_tables(case)
        n = case["pages"]
        rng = random.Random(seed)
        names = list(range(n))
        rng.shuffle(names)         # other inputs, other page names
        table = torch.full((len(lists), max(len(p) for p in lists)), -1, dtype=torch.int32)
        refs = [0] * n
        for b, p in enumerate(lists):
            table[b, :len(p)] = torch.tensor([names[x] for x in p], dtype=torch.int32)
            for x in p:
                refs[names[x]] += 1
        st["planes"] = _planes(case, n, gen)
        st["table"], st["refs"], st["seq_lens"] = table.cuda(), ints(refs), ints(lens)
        st["new_table"], st["new_refs"] = st["table"].clone(), st["refs"].clone()
    if own:
        import block_sparse_attention_nvfp4_gb300 as msa
        st["cache"] = _cache_object(case, st["planes"])
        if kind in ("attend", "append"):
            st["batch"] = msa.KV8Batch(st["context_lens"], st["q_indptr"], st["table"], st.get("q"),
                                       total_rows=st["indptr"][-1], max_rows_per_req=max(st["rows"]))
            if kind == "attend":
                st["attention"] = msa.KV8Attention(st["cache"], st["batch"])
            else:
                st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        else:
            st["pool"] = msa.PagePool([st["cache"]], st["seq_lens"], st["table"], st["refs"])
    return st


# ------------------------------------------------------------------------------- one pass
def run(st):
    kind = st["case"]["kind"]
    if kind == "attend":
        if own:
            out = st["attention"].attend(st["ids"])
            return {"out": out, "lse": st["attention"].lse}
        return _attend(st)
    if kind == "append":
        if own:
            st["cache"].append(st["batch"], st["k"], st["v"], st["ws"])
        else:
            for n in ("k", "v"):
                _append(st, st[n], st["planes"][n + "_data"], st["planes"][n + "_scale"])
        p = st["planes"]
        return {"k": p["k_data"].view(FP8), "k_scale": p["k_scale"], "v": p["v_data"].view(FP8), "v_scale": p["v_scale"]}
    if kind == "copy":
        if own:
            st["pool"].copy(st["src"], st["dst"], st["tokens"])
        else:
            _copy(st["planes"], st["src"].long(), st["dst"].long(), st["tokens"])
        return _plane_values(st)
    if kind == "fork":
        if own:
            st["pool"].fork(st["parents"], st["children"])
            st["pool"].reserve(st["children"], st["grown"])
            st["pool"].free(st["children"])
        else:
            _fork(st)
            _reserve(st)
            _free(st)
        return {"table": st["table"], "refs": st["refs"], "seq_lens": st["seq_lens"], "planes": _plane_values(st)}
    if own:
        st["pool"].compact(st["new_table"], st["new_refs"])
    else:
        _compact(st)
    return {"table": st["new_table"], "refs": st["new_refs"], "planes": _plane_values(st)}


def _plane_values(st):
    """The planes as what they hold: E4M3 values and scales, or the NVFP4 bytes."""
    kv8 = st["case"]["cache"] == "kv8"
    return {n: t.view(FP8) if kv8 and t.dtype == torch.uint8 else t for n, t in st["planes"].items()}


def _attend(st):
    case, p = st["case"], st["planes"]
    H, G = case["kv_heads"], case["q_per_kv"]
    total = st["indptr"][-1]
    q = (st["q"].view(FP8) if case["q"] == "e4m3" else st["q"]).float()
    out = torch.empty((total, H * G, DIM), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((total, H * G), dtype=torch.float32, device="cuda")
    heads = torch.arange(H, device="cuda")[:, None]
    for b, (n, r) in enumerate(zip(st["lens"], st["rows"])):
        r0 = st["indptr"][b]
        nb = _pages_of(n)
        blocks = torch.arange(nb, device="cuda").expand(H, nb) if st["ids"] is None else st["ids"][b].long()
        phys = st["table"][b].long()[blocks.clamp(min=0)]                                # [H, blocks]
        k = p["k_data"].view(FP8)[phys, heads].float() * p["k_scale"][phys, heads][..., None, None]
        v = p["v_data"].view(FP8)[phys, heads].float() * p["v_scale"][phys, heads][..., None, None]
        k, v = k.flatten(1, 2), v.flatten(1, 2)                                          # [H, keys, 128]
        pos = blocks[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
        pos = torch.where(blocks[..., None] >= 0, pos, n).flatten(1, 2)                  # [H, keys]
        row_pos = n - r + torch.arange(r, device="cuda")
        v = torch.where((pos < n)[..., None], v, 0.0)
        s = torch.matmul(q[r0:r0 + r].view(r, H, G, DIM).permute(1, 2, 0, 3).reshape(H, G * r, DIM), k.transpose(1, 2))
        s *= 1.0 / math.sqrt(DIM)
        s = s.view(H, G, r, -1).masked_fill_(pos[:, None, None, :] > row_pos[:, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        e = s.sub_(m).exp_()
        l = e.sum(-1, keepdim=True)
        o = torch.matmul(e.view(H, G * r, -1), v).view(H, G, r, DIM) / l
        out[r0:r0 + r] = o.permute(2, 0, 1, 3).reshape(r, H * G, DIM).to(torch.bfloat16)
        lse[r0:r0 + r] = (m + l.log()).squeeze(-1).permute(2, 0, 1).reshape(r, H * G)
    return {"out": out, "lse": lse}


def _pow2_at_least(x):
    """The smallest power of two that is not below x (64 bits; 0 for 0)."""
    m, e = torch.frexp(x)
    return torch.where(x > 0, torch.ldexp(torch.ones_like(x), torch.where(m == 0.5, e - 1, e)), 0.0)


def _append(st, x, data, scale):
    n, r = st["context_lens"].long(), (st["q_indptr"][1:] - st["q_indptr"][:-1]).long()
    total = x.shape[0]
    req = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), r, output_size=total)
    pos = n[req] - r[req] + torch.arange(total, device="cuda") - st["q_indptr"].long()[req]
    phys = st["table"].long()[req, pos // BLOCK]
    xf = x.float()
    amax = torch.zeros_like(scale).index_reduce_(0, phys, xf.abs().amax(-1), "amax")
    need = _pow2_at_least(amax.double() / E4M3_MAX).clamp_(min=2.0 ** MIN_EXP)
    first = n - r                                       # the request's first new position
    live = r > 0
    page0 = st["table"].long()[torch.arange(n.numel(), device="cuda"), first.clamp(max=st["table"].shape[1] * BLOCK - 1) // BLOCK]
    page0, f = page0[live], (first % BLOCK)[live]       # each request's first touched page, its first new slot
    old = torch.zeros_like(need)
    old[page0] = torch.where((f > 0)[:, None], scale[page0].double(), 0.0)
    new = torch.maximum(need, _pow2_at_least(old))
    ratio = (old / new).float()[page0][:, :, None, None]
    slots = torch.arange(BLOCK, device="cuda")[None, None, :, None]
    codes = data.view(FP8)[page0].float()
    data[page0] = torch.where((slots < f[:, None, None, None]), (codes * ratio).to(FP8).view(torch.uint8), data[page0])
    data[phys, :, pos % BLOCK] = (xf / new.float()[phys][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(FP8).view(torch.uint8)
    scale[phys] = new.float()[phys]


def _copy(planes, src, dst, tokens):
    for t in planes.values():
        if tokens is None or t.dim() == 2:              # whole pages, and what a page keeps once
            t[dst] = t[src]
        else:
            keep = torch.arange(BLOCK, device="cuda")[:, None] < tokens.view(-1, *[1] * (t.dim() - 1))
            t[dst] = torch.where(keep, t[src], t[dst])


def _fork(st):
    lens, table, refs = st["seq_lens"], st["table"], st["refs"]
    par, child = st["parents"].long(), st["children"].long()
    n = lens[par].long()
    full, tail = n // BLOCK, n % BLOCK
    free = (refs == 0).nonzero().squeeze(1)
    needs = (tail > 0)
    page = free[(needs.cumsum(0) - 1).clamp(min=0)]
    col = torch.arange(table.shape[1], device="cuda")
    shared = col < full[:, None]
    table[child] = torch.where(shared, table[par], table[child])
    refs.index_add_(0, table[par][shared].long(), torch.ones_like(table[par][shared]))
    child_t, page_t, full_t = child[needs], page[needs], full[needs]
    old = table[par[needs], full_t].long()
    table[child_t, full_t] = page_t.to(torch.int32)
    refs[page_t] = 1
    lens[child] = lens[par]
    _copy(st["planes"], old, page_t, tail[needs])


def _reserve(st):
    lens, table, refs = st["seq_lens"], st["table"], st["refs"]
    rows, to = st["children"].long(), st["grown"].long()
    have, want = (lens[rows].long() + BLOCK - 1) // BLOCK, (to + BLOCK - 1) // BLOCK
    col = torch.arange(table.shape[1], device="cuda")
    fresh = (col >= have[:, None]) & (col < want[:, None])
    free = (refs == 0).nonzero().squeeze(1)[:int(fresh.sum())]
    t = table[rows]
    t[fresh] = free.to(torch.int32)
    table[rows] = t
    refs[free] = 1
    lens[rows] = st["grown"]


def _free(st):
    lens, table, refs = st["seq_lens"], st["table"], st["refs"]
    rows = st["children"].long()
    held = torch.arange(table.shape[1], device="cuda") < ((lens[rows].long() + BLOCK - 1) // BLOCK)[:, None]
    pages = table[rows][held].long()
    refs.index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    lens[rows] = 0


def _compact(st):
    refs, table = st["refs"], st["table"]
    live = refs > 0
    ids = torch.arange(refs.numel(), device="cuda")
    front = ids < live.sum()
    movers, holes = (live & ~front).nonzero().squeeze(1), (~live & front).nonzero().squeeze(1)
    to = ids.clone()
    to[movers] = holes
    held = torch.arange(table.shape[1], device="cuda") < ((st["seq_lens"].long() + BLOCK - 1) // BLOCK)[:, None]
    st["new_table"].copy_(torch.where(held, to[table.clamp(min=0).long()].to(torch.int32), table))
    st["new_refs"].copy_(torch.where(front, torch.where(live, refs, 0), 0))
    st["new_refs"][holes] = refs[movers]
    for t in st["planes"].values():
        t[holes] = t[movers]


# ------------------------------------------------------------------------------- floors
def work(case):
    kind = case["kind"]
    if kind == "attend":
        H, G = case["kv_heads"], case["q_per_kv"]
        pairs = tokens = meta = 0
        rows = 0
        for n, r in _lengths(case):
            nb = _pages_of(n)
            rows += r
            if case["blocks"] and nb > case["blocks"]:
                last = n - (nb - 1) * BLOCK
                keys = (case["blocks"] - 1) * BLOCK + last
                tokens += keys
                # the recent block's and the row's own later keys are what a row may not see
                pairs += keys * r - r * (r - 1) // 2
                meta += 4 * H * case["blocks"]
            else:
                tokens += n
                pairs += n * r - r * (r - 1) // 2
                meta += 4 * nb
        q_bytes = 1 if case["q"] == "e4m3" else 2
        return {"bytes": tokens * H * 2 * DIM + rows * H * G * (DIM * (q_bytes + 2) + 4) + meta,
                "flops": 4 * DIM * pairs * H * G}
    if kind == "append":
        rows = sum(r for _, r in _lengths(case))
        size = 4 if case["src"] == "fp32" else 2
        values = rows * case["kv_heads"] * DIM * 2
        return {"bytes": values * (size + 1) + 8 * case["kv_heads"] * sum(_pages_of(r) for _, r in _lengths(case)),
                "flops": 2 * values}
    per_token, per_page = _token_bytes(case)
    if kind == "copy":
        pairs = _pairs(case)
        return {"bytes": sum(2 * (t * per_token + per_page) + 12 for _, _, t in pairs), "flops": 0}
    if kind == "fork":
        lens = _parent_lengths(case)
        rng = random.Random(case["shape"] + 1)
        total = 0
        for _ in range(case["children"]):
            n = lens[rng.randrange(case["parents"])]
            total += 2 * ((n % BLOCK) * per_token + (per_page if n % BLOCK else 0))
            total += 4 * (2 * _pages_of(n) + 2 * _pages_of(n + case["grow"])) + 24    # rows and counts
        return {"bytes": total, "flops": 0}
    lens, lists = _page_tables(case)
    live = set(x for p in lists for x in p)
    holes = len(live) * (case["pages"] - len(live)) // case["pages"]   # what a shuffled pool has on average
    return {"bytes": 2 * holes * (BLOCK * per_token + per_page) + 8 * case["pages"] + 8 * sum(len(p) for p in lists),
            "flops": 0}


# ------------------------------------------------------------------------------- 64 bits
def _e4m3_values():
    """The 256 values of E4M3 from their bits."""
    got = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if (c & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        got.append(-v if c & 128 else v)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def exact(case, seed):
    if case["kind"] == "attend":
        return _exact_attend(case, prepare_plain(case, seed))
    if case["kind"] == "append":
        return _exact_append(case, prepare_plain(case, seed))
    return None      # copied bytes and page numbers: nothing is computed in floating point


def prepare_plain(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_attend(case, st):
    value = _e4m3_values()
    H, G, p = case["kv_heads"], case["q_per_kv"], st["planes"]
    q = value[st["q"].long()] if case["q"] == "e4m3" else st["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    for b, (n, r) in enumerate(zip(st["lens"], st["rows"])):
        rows = slice(st["indptr"][b], st["indptr"][b] + r)
        at = torch.arange(n - r, n, device="cuda")
        for h in range(H):
            which = range(_pages_of(n)) if st["ids"] is None else [i for i in st["ids"][b, h].tolist() if i >= 0]
            which = torch.tensor(list(which), device="cuda")
            page = st["table"][b, which].long()
            t = (which[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(-1)
            seen = t < n
            k = (value[p["k_data"][page, h].long()] * p["k_scale"][page, h].double()[:, None, None]).reshape(-1, DIM)[seen]
            v = (value[p["v_data"][page, h].long()] * p["v_scale"][page, h].double()[:, None, None]).reshape(-1, DIM)[seen]
            for g in range(h * G, (h + 1) * G):
                z = (q[rows, g] @ k.T) / math.sqrt(DIM)
                z = z + torch.where(t[seen][None, :] <= at[:, None], 0.0, -math.inf)
                y = torch.logsumexp(z, 1)
                lse[rows, g] = y
                out[rows, g] = torch.exp(z - y[:, None]) @ v
    return {"out": out, "lse": lse}


def _round_e4m3(x):
    """The E4M3 value nearest to x, ties to the even code, saturating (64 bits)."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=E4M3_MAX), x)


def _exact_append(case, st):
    value = _e4m3_values()
    got = {}
    for name in ("k", "v"):
        x, codes = st[name].double(), st["planes"][name + "_data"]
        scale = st["planes"][name + "_scale"].double()
        vals = value[codes.long()]
        for b, (n, r) in enumerate(zip(st["lens"], st["rows"])):
            t = n - r
            while t < n:                 # page by page
                page, f = int(st["table"][b, t // BLOCK]), t % BLOCK
                m = min(BLOCK - f, n - t)
                i = st["indptr"][b] + t - (n - r)
                new = x[i:i + m].transpose(0, 1)                     # [H, m, 128]
                want = new.abs().amax((1, 2)) / E4M3_MAX
                e = torch.ceil(torch.log2(want.clamp(min=2.0 ** -200))).clamp(min=MIN_EXP)
                s = torch.exp2(e)
                s = torch.where(want > s, 2 * s, s)                  # the logarithm's own rounding
                s = torch.where((want <= s / 2) & (e > MIN_EXP), s / 2, s)
                if f:
                    s = torch.maximum(s, scale[page])
                    vals[page, :, :f] = _round_e4m3(vals[page, :, :f] * (scale[page] / s)[:, None, None])
                vals[page, :, f:f + m] = _round_e4m3(new / s[:, None, None])
                scale[page] = s
                t += m
        got[name], got[name + "_scale"] = vals, scale
    return got
