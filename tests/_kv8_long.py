"""Plain 64-bit forms of the operators for long sequences over the 8-bit cache (window, shared pages, weights,
eviction), for the tests."""
import math

import numpy as np
import torch

from tests._kv8 import BLOCK, DIM, e4m3_codes, e4m3_values


def tokens(cache, table_row, h, t):
    """(page, K values, V codes' values, V scales) of the tokens t of a request, float64; page -1: outside the pool."""
    val = torch.from_numpy(e4m3_values()).cuda()
    page = torch.as_tensor(np.asarray(table_row, np.int64), device="cuda")[t // BLOCK]
    good = (page >= 0) & (page < cache.num_pages)
    p, s = page.clamp(0, cache.num_pages - 1), t % BLOCK
    k = val[cache.k_data[p, h, s].long()] * cache.k_scale[p, h].double()[:, None]
    return good, k, val[cache.v_data[p, h, s].long()], cache.v_scale[p, h].double()


def attend(q, cache, lens, indptr, table, sees, exact_q=True, sm_scale=1.0 / math.sqrt(DIM)):
    """Attention in 64 bits where a row at position p sees the tokens t with sees(t, p) (and t <= p), and how far a
    kernel may be off it: out, lse, their bounds. q float64 [rows, H, G, 128].

    The bounds add up the kernel's roundings, half a step each (p the softmax weights, A = sum p |v|): a weight's
    FP16 rounding 2^-11, its FP32 exponential and argument 2^-18 together; a score's error d (128 FP32 sums of
    magnitude at most S, 2^-16 S; the part of a BF16 query that its two E4M3 rows do not hold, 2^-17.8 of its largest
    element at most, unless q is exact), by which a weight moves by e^(2 d) at most; FP16 weights below 2^-14 of
    the reference, 2^-24 of the largest; the output's BF16 rounding, 2^-8 of the value (halves that are joined add FP32
    roundings of 2^-22 of A)."""
    rows, H, G = q.shape[:3]
    out = torch.zeros((rows, H, G, DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, H, G), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        n, r0, r = int(n), int(indptr[b]), int(indptr[b + 1] - indptr[b])
        for r1 in range(0, r, 256):
            p = torch.arange(n - r + r1, min(n, n - r + r1 + 256), device="cuda")
            t = torch.arange(n, device="cuda")
            see = (t[None] <= p[:, None]) & sees(t[None], p[:, None])
            use = see.any(0)
            t, see = t[use], see[:, use]
            sl = slice(r0 + r1, r0 + r1 + len(p))
            for h in range(H):
                good, k, vc, vs = tokens(cache, table[b], h, t)
                seen = (see & good[None])[:, None]                              # [rows, 1, t]
                qq = q[sl, h]
                s = torch.where(seen, torch.einsum("rgd,td->rgt", qq, k) * sm_scale, -math.inf)
                y = torch.logsumexp(s, -1)
                w = torch.where(seen & (y != -math.inf)[..., None], torch.exp(s - y[..., None]), 0.0)   # (a NaN score: a NaN row)
                v = vc * vs[:, None]
                if torch.isnan(v).any():        # a NaN reaches the rows that see it, and no others
                    clean = torch.nan_to_num(v)
                    o = torch.einsum("rgt,td->rgd", w, clean)
                    hit = torch.einsum("rt,td->rd", seen[:, 0].double(), torch.isnan(v).double()) > 0
                    o = torch.where(hit[:, None], math.nan, o)
                    v = clean
                else:
                    o = torch.einsum("rgt,td->rgd", w, v)
                mag = torch.where(seen, torch.einsum("rgd,td->rgt", qq.abs(), k.abs()) * sm_scale, 0.0).amax(-1)
                low = 0.0 if exact_q else torch.where(seen, k.abs().sum(1) * sm_scale, 0.0).amax(-1) * qq.abs().amax(-1) * 2.0 ** -17.8
                d = 2.0 ** -16 * mag + low
                A = torch.einsum("rgt,td->rgd", w, v.abs())
                sub = 2.0 ** -24 * torch.nan_to_num(vc).abs().sum(0) * (w * vs).amax(-1)[..., None]
                rel = 2.0 ** -11 + 2.0 ** -18 + 2.0 ** -20 + torch.expm1(2 * d)[..., None]
                out[sl, h], lse[sl, h] = o, y
                tol[sl, h] = 2.0 ** -8 * o.abs() + (rel * A + sub) * (1 + 2.0 ** -8) + 1e-30
                tol_lse[sl, h] = d + 2.0 ** -18 + 2.0 ** -22 * y.abs().nan_to_num(posinf=0.0)
    f = lambda x: x.reshape(rows, H * G, *x.shape[3:])  # noqa: E731
    return f(out), f(lse), f(tol), f(tol_lse)


def close(got, want, tol, what=""):
    """got within tol of want, NaN and infinities where want has them."""
    got = got.double()
    same = (torch.isnan(got) & torch.isnan(want)) | (got == want)
    bad = ~same & ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i].item()}, "
                             f"want {want[i].item()} +- {tol[i].item()}")


def weights(q, lse, cache, lens, indptr, table, old, keep, exact_q=True, sm_scale=1.0 / math.sqrt(DIM)):
    """{(b, h): (new weights of tokens 0 .. N - 1, their bounds)} in 64 bits. lse: what the kernel was given.

    The bounds: with a score's error d (as in attend) and its argument s log2 e - lse log2 e rounded three times in
    FP32 (2^-23 of the larger of |s|, |lse|, times ln 2 / ln 2), a weight w moves by w (e^d' - 1); the exponential adds 2^-21;
    n FP32 sums of non-negative numbers add n 2^-24 of the sum, of which the kernel's two chains see half each."""
    rows, H, G = q.shape[:3]
    lse = lse.double().view(rows, H, G)
    got = {}
    for b, n in enumerate(lens):
        n, r0, r = int(n), int(indptr[b]), int(indptr[b + 1] - indptr[b])
        t = torch.arange(n, device="cuda")
        for h in range(H):
            good, k, _, _ = tokens(cache, table[b], h, t)
            dead = torch.isnan(k).any(1)
            k = torch.nan_to_num(k)
            w = torch.zeros(n, dtype=torch.float64, device="cuda")
            tol = torch.zeros_like(w)
            for r1 in range(0, r, 256):
                p = torch.arange(n - r + r1, min(n, n - r + r1 + 256), device="cuda")
                sl = slice(r0 + r1, r0 + r1 + len(p))
                qq, y = q[sl, h], lse[sl, h]
                use = torch.isfinite(y) & torch.isfinite(qq).all(-1)
                qq = torch.nan_to_num(qq, posinf=0.0, neginf=0.0)
                s = torch.einsum("rgd,td->rgt", qq, k) * sm_scale
                seen = (t[None] <= p[:, None])[:, None] & use[..., None] & (good & ~dead)[None, None]
                x = torch.where(seen, torch.exp(s - torch.where(use, y, 0.0)[..., None]), 0.0)
                mag = torch.einsum("rgd,td->rgt", qq.abs(), k.abs()) * sm_scale
                low = 0.0 if exact_q else (k.abs().sum(1) * sm_scale)[None, None] * qq.abs().amax(-1)[..., None] * 2.0 ** -17.8
                d = 2.0 ** -16 * mag + low + 2.0 ** -22 * (s.abs() + torch.where(use, y, 0.0).abs()[..., None])
                w += x.sum((0, 1))
                tol += torch.where(seen, x * (torch.expm1(d) + 2.0 ** -21), 0.0).sum((0, 1))
            first = torch.where(t < n - r, keep * old[b, h, :n].double(), 0.0) if old is not None else torch.zeros_like(w)
            got[b, h] = first + w, tol + (r * G + 4) * 2.0 ** -24 * (w + first.abs()) + 1e-37
    return got


def kept(w, n, keep, sinks, recent):
    """Positions that a head keeps of n tokens with weights w (float32 numpy), in order."""
    if n <= keep:
        return np.arange(n)
    t = np.arange(n)
    must = (t < sinks) | (t >= n - recent)
    key = np.where(w[:n] > 0, w[:n], np.float32(0.0))          # negative and NaN: 0
    rest = t[~must]
    order = rest[np.lexsort((rest, -key[rest].astype(np.float64)))]
    return np.sort(np.concatenate([t[must], order[:keep - sinks - recent]]))


def evict(state, caches, weights, parents, children, keep, sinks, recent):
    """msa_pages_evict on numpy state, in place: state = (lens, table, refs); caches: dicts of k_data, k_scale, v_data,
    v_scale; weights: one [S, H, L] for each. Entries that do nothing are left out."""
    val = e4m3_values()
    lens, table, refs = state
    old_lens, old_table = lens.copy(), table.copy()
    old = [{n: a.copy() for n, a in c.items()} for c in caches]
    old_w = [w.copy() for w in weights]
    free = [p for p in range(len(refs)) if refs[p] == 0]
    inplace = {p for p, c in zip(parents, children) if p == c}
    seen, out = set(), False
    for par, ch in zip(parents, children):
        if not (0 <= par < len(lens) and 0 <= ch < len(lens)):
            continue
        first, _ = ch not in seen, seen.add(ch)
        if not first or (par != ch and (old_lens[ch] != 0 or par in inplace)):
            continue
        n = int(old_lens[par])
        m = min(n, keep)
        if n == 0 or (par == ch and n <= keep):
            continue
        need = (m + BLOCK - 1) // BLOCK
        if out or need > len(free):      # (this entry and all later ones that need pages)
            out = True
            continue
        ids, free = free[:need], free[need:]
        for c, o, w, ow in zip(caches, old, weights, old_w):
            for h in range(w.shape[1]):
                t = kept(ow[par, h], n, keep, sinks, recent)
                w[ch, h, :m] = ow[par, h, t]
                page = old_table[par, t // BLOCK]
                good = (page >= 0) & (page < len(refs))
                pg = np.where(good, page, 0)
                for k in ("k", "v"):
                    s = o[k + "_scale"][pg, h].astype(np.float32)
                    s = np.where(good & (s > 0) & np.isfinite(s), s, np.float32(0))
                    codes = np.where(good[:, None], o[k + "_data"][pg, h, t % BLOCK], 0).astype(np.uint8)
                    for i, p in enumerate(ids):
                        a, b = i * BLOCK, min(m, (i + 1) * BLOCK)
                        top = s[a:b].max()
                        ratio = (s[a:b] / top if top > 0 else np.zeros(b - a, np.float32)).astype(np.float32)
                        x = (val[codes[a:b]].astype(np.float32) * ratio[:, None]).astype(np.float64)
                        c[k + "_data"][p, h, :b - a] = np.where((ratio == 1)[:, None], codes[a:b], e4m3_codes(x))
                        c[k + "_scale"][p, h] = top
        for p in ids:
            refs[p] = 1
        if par == ch:
            for x in old_table[par, :(n + BLOCK - 1) // BLOCK]:
                if 0 <= x < len(refs):
                    refs[x] = max(0, refs[x] - 1)
        table[ch, :need] = ids
        lens[ch] = m
