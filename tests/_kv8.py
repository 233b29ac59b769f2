"""Plain 64-bit forms of the 8-bit cache operators and of the page operators, for the tests."""
import math

import numpy as np
import torch

DIM, BLOCK = 128, 128
FP8 = torch.float8_e4m3fn


def e4m3_values():
    """The 256 E4M3 values from their bits (float64)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def e4m3_codes(x):
    """E4M3 codes of float64 values: nearest, ties to the even code, saturating; NaN -> 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = np.exp2(e - 3)
    q = np.rint(a / step) * step            # exact: at most 4 significant bits more than a step
    q = np.minimum(q, 448.0)
    _, ex = np.frexp(np.maximum(q, 2.0 ** -6))
    ex = ex - 1
    code = np.where(q < 2.0 ** -6, np.rint(q * 2.0 ** 9),
                    ((ex + 7) * 8 + np.rint((q / np.exp2(ex.astype(np.float64)) - 1) * 8))).astype(np.int64)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def pow2_at_least(x):
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.where(x > 0, np.ldexp(1.0, np.where(m == 0.5, e - 1, e)), 0.0)


def append_plane(x, lens, indptr, table, data, scale):
    """The append rule on one plane, page by page, in place (numpy: x [T, H, 128] float64)."""
    val = e4m3_values()
    for b, n in enumerate(lens):
        r = int(indptr[b + 1] - indptr[b])
        t = n - r
        while t < n:
            f = t % BLOCK
            m = min(BLOCK - f, n - t)
            page = int(table[b, t // BLOCK])
            new = x[indptr[b] + t - (n - r):][:m].transpose(1, 0, 2)      # [H, m, 128]
            for h in range(new.shape[0]):
                fin = new[h][np.isfinite(new[h])]
                amax = np.abs(fin).max() if fin.size else 0.0
                s = max(float(pow2_at_least(amax / 448.0)), 2.0 ** -60)
                if f:
                    old = float(scale[page, h])
                    old = old if old > 0 and math.isfinite(old) else 0.0
                    s = max(s, float(pow2_at_least(old)))
                    if old != s:
                        data[page, h, :f] = e4m3_codes(val[data[page, h, :f]] * (old / s))
                data[page, h, f:f + m] = e4m3_codes(new[h] / s)
                scale[page, h] = s
            t += m


def fill(pages, heads, seed, level=1.0):
    """A filled plane on the GPU: codes and scales (float32, not powers of two)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((pages, heads, BLOCK, DIM), device="cuda", generator=g) * level
    x *= torch.exp2(torch.rand((pages, heads, 1, 1), device="cuda", generator=g) * 3 - 1.5)
    s = x.abs().amax((2, 3)) / 448.0
    return (x / s[:, :, None, None]).clamp_(-448, 448).to(FP8).view(torch.uint8), s


def batch_of(lens, rows, seed, spare=3):
    """(context_lens, q_indptr, block_table, pages): a shuffled table over all pages plus spare ones."""
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
    perm = np.random.default_rng(seed).permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), max(1, max(need, default=1))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    indptr = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    return np.asarray(lens, np.int32), indptr, table, len(perm)


def attend(q, cache, lens, indptr, table, ids=None, sm_scale=1.0 / math.sqrt(DIM)):
    """Attention in 64 bits on the GPU, and how far a kernel may be off it.

    q float64 [rows, H, G, 128] as the values that the codes or BF16 stand for. Returns out, lse and
    their bounds. With p the softmax weights, A = sum p |v|, and one rounding half a step:
      * a weight's FP16 rounding 2^-11, its FP32 exponential and its argument's rounding 2^-18 together,
      * a score's error d: FP32 sums of 128 products (each sum 2^-23, the sum of magnitudes at most S,
        so 128 2^-23 S = 2^-16 S) and, for BF16 queries, the part of q below 2^-18 of its
        largest element; a weight moves by a factor within e^(2 d) (its own score and the sum's),
      * FP16 weights below 2^-14 of the reference have a step of 2^-24: 2^-24 sum |code| max p v_scale,
      * the output's BF16 rounding 2^-8 of the value."""
    val = torch.from_numpy(e4m3_values()).cuda()
    rows, H, G = q.shape[:3]
    out = torch.zeros((rows, H, G, DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, H, G), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        n, r0, r = int(n), int(indptr[b]), int(indptr[b + 1] - indptr[b])
        if r == 0:
            continue
        nb = (n + BLOCK - 1) // BLOCK
        pos_r = torch.arange(n - r, n, device="cuda")
        for h in range(H):
            use = list(range(nb)) if ids is None else list(dict.fromkeys(int(c) for c in ids[b, h] if 0 <= c < nb))
            use = [c for c in use if 0 <= int(table[b, c]) < cache.num_pages]
            if not use:
                continue
            page = torch.tensor([int(table[b, c]) for c in use], device="cuda")
            t = (torch.tensor(use, device="cuda")[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(-1)
            vs = cache.v_scale[page, h].double().repeat_interleave(BLOCK)
            k = val[cache.k_data[page, h].long()].reshape(-1, DIM) * cache.k_scale[page, h].double().repeat_interleave(BLOCK)[:, None]
            vc = val[cache.v_data[page, h].long()].reshape(-1, DIM)
            keep = t < n
            t, k, vc, vs = t[keep], k[keep], vc[keep], vs[keep]
            for r1 in range(0, r, 256):
                qq = q[r0 + r1:min(r0 + r, r0 + r1 + 256), h]                     # [rows, G, 128]
                see = t[None, None, :] <= pos_r[r1:r1 + 256][:, None, None]
                s = torch.where(see, torch.einsum("rgd,td->rgt", qq, k) * sm_scale, -math.inf)
                mag = torch.where(see, torch.einsum("rgd,td->rgt", qq.abs(), k.abs()) * sm_scale, 0.0).amax(-1)
                low = torch.where(see, (k.abs().sum(1) * sm_scale)[None, None, :], 0.0).amax(-1) * qq.abs().amax(-1) * 2.0 ** -18
                d = 2.0 ** -16 * mag + low
                y = torch.logsumexp(s, -1)
                p = torch.where(see & (y > -math.inf)[..., None], torch.exp(s - y[..., None]), 0.0)
                p = torch.nan_to_num(p, nan=math.nan)
                v = vc * vs[:, None]
                vis = torch.where(see.any(1)[:, :, None], vc[None], 0.0)           # codes a row may see
                o = torch.einsum("rgt,rtd->rgd", p, vis * vs[None, :, None]) if torch.isnan(v).any() else torch.einsum("rgt,td->rgd", p, v)
                A = torch.einsum("rgt,td->rgd", p, torch.nan_to_num(v).abs())
                sub = 2.0 ** -24 * torch.nan_to_num(vc).abs().sum(0) * (p * vs).amax(-1)[..., None]
                sl = slice(r0 + r1, r0 + r1 + qq.shape[0])
                out[sl, h], lse[sl, h] = o, y
                rel = 2.0 ** -11 + 2.0 ** -18 + torch.expm1(2 * d)[..., None]
                tol[sl, h] = 2.0 ** -8 * o.abs() + (rel * A + sub) * (1 + 2.0 ** -8) + 1e-30
                tol_lse[sl, h] = d + 2.0 ** -18 + 2.0 ** -22 * y.abs().nan_to_num(posinf=0.0)
    return out.reshape(rows, H * G, DIM), lse.reshape(rows, H * G), tol.reshape(rows, H * G, DIM), tol_lse.reshape(rows, H * G)


class Pool:
    """The page operators in plain Python over numpy state."""

    def __init__(self, lens, table, refs, planes):
        self.lens, self.table, self.refs = lens.copy(), table.copy(), refs.copy()
        self.planes = {n: a.copy() for n, a in planes.items()}    # [P, ..., 128, bytes] or [P, k]

    def copy(self, src, dst, tokens=None):
        for i, (a, b) in enumerate(zip(src, dst)):
            if a < 0 or b < 0 or a == b:
                continue
            t = BLOCK if tokens is None else tokens[i]
            for x in self.planes.values():
                if x.ndim == 2:
                    x[b] = x[a]
                else:
                    x[b, ..., :t, :] = x[a, ..., :t, :]

    def _free_pages(self):
        return [p for p in range(len(self.refs)) if self.refs[p] == 0]

    def fork(self, parents, children):
        lens, table = self.lens.copy(), self.table.copy()
        free, done, short = self._free_pages(), set(), False
        for p, c in zip(parents, children):
            if not (0 <= p < len(lens) and 0 <= c < len(lens)) or c in done or lens[c] != 0 or p == c:
                if 0 <= c < len(lens):
                    done.add(c)
                continue
            done.add(c)
            n = int(lens[p])
            full, tail = n // BLOCK, n % BLOCK
            if tail:
                if not free:
                    continue
                page = free.pop(0)
                self.copy([table[p, full]], [page], [tail])
                self.table[c, full], self.refs[page] = page, 1
            self.table[c, :full] = table[p, :full]
            for x in table[p, :full]:
                self.refs[x] += 1
            self.lens[c] = n

    def reserve(self, seqs, new_lens):
        free, done, asked = self._free_pages(), set(), 0
        have = len(free)
        for s, n in zip(seqs, new_lens):
            if not 0 <= s < len(self.lens) or s in done:
                continue
            done.add(s)
            if n > self.table.shape[1] * BLOCK or n <= self.lens[s]:
                continue
            c0, c1 = (self.lens[s] + BLOCK - 1) // BLOCK, (n + BLOCK - 1) // BLOCK
            asked += c1 - c0
            if asked > have and c1 > c0:
                continue
            for c in range(c0, c1):
                page = free.pop(0)
                self.table[s, c], self.refs[page] = page, 1
            self.lens[s] = n

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.lens):
                for c in range((self.lens[s] + BLOCK - 1) // BLOCK):
                    self.refs[self.table[s, c]] -= 1
                self.lens[s] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = np.arange(len(self.refs))
        for m, h in zip(movers, holes):
            to[m] = h
            self.refs[h], self.refs[m] = self.refs[m], 0
        self.copy(movers, holes)
        for s in range(len(self.lens)):
            for c in range((self.lens[s] + BLOCK - 1) // BLOCK):
                self.table[s, c] = to[self.table[s, c]]
        return live
