"""Binary64 statements of the paged INT4 KV cache's operators, for the tests: attention over
block tables, and the pool's reserve, fork and free as loops over rows."""
import math

import torch

CODES = ("k_cache", "v_cache")
STEPS = ("k_scale", "k_zero", "v_scale", "v_zero")


def random_pages(pages, hkv, page, seed, device="cuda"):
    """Random codes, scales near those of normal data and whole zeros."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    c = {n: torch.randint(0, 256, (pages, hkv, page, 64), generator=g, dtype=torch.uint8) for n in CODES}
    for n in ("k_scale", "v_scale"):
        c[n] = (0.05 + 0.4 * torch.rand((pages, hkv, page), generator=g)).half()
    for n in ("k_zero", "v_zero"):
        c[n] = torch.randint(0, 16, (pages, hkv, page), generator=g).half()
    return {n: t.to(device) for n, t in c.items()}


def attention(q, cache, table, lens, cu, scale=None, window=0, sinks=0):
    """(out, size, score size, floor, score rms): the result in binary64; per element the sum of p_j |vhat_j|,
    the terms a kernel adds; the largest sum of a score's terms (those of q.c and of z sum(q)); per
    element max s_j sum |c_j - z_j| of the values. Rows outside the sequences are NaN."""
    q, table = q.double().cpu(), table.cpu()
    cache = {n: t.cpu() for n, t in cache.items()}
    tokens, hq, d = q.shape
    pages, hkv, page, _ = cache["k_cache"].shape
    group = hq // hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.full((tokens, hq, d), math.nan, dtype=torch.float64)
    size, floor = torch.zeros_like(out), torch.zeros_like(out)
    score_size, score_rms = 0.0, 0.0
    for b, n in enumerate(lens):
        n = min(max(n, 0), table.shape[1] * page)
        nq = cu[b + 1] - cu[b]
        slots = torch.arange(n)
        ids = table[b, slots // page].long()
        there = (ids >= 0) & (ids < pages)
        ids = ids.clamp(0, pages - 1)

        def rows(name):
            codes = cache[name + "_cache"][ids, :, slots % page]  # [n, hkv, 64]
            u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
            s = cache[name + "_scale"][ids, :, slots % page].double()[..., None]
            z = cache[name + "_zero"][ids, :, slots % page].double()[..., None]
            return u, s, z

        (ku, ks, kz), (vu, vs, vz) = rows("k"), rows("v")
        for i in range(nq):
            p = n - nq + i
            seen = there & (slots <= p)
            if window:
                seen &= (slots > p - window) | (slots < sinks)
            t = cu[b] + i
            out[t] = 0
            at = seen.nonzero()[:, 0]
            if not len(at):
                continue
            for g in range(hkv):
                k, v = (ku[at, g] - kz[at, g]) * ks[at, g], (vu[at, g] - vz[at, g]) * vs[at, g]
                rows_q = q[t, g * group:(g + 1) * group]
                w = torch.softmax(rows_q @ k.T * scale, 1)
                out[t, g * group:(g + 1) * group] = w @ v
                size[t, g * group:(g + 1) * group] = w @ v.abs()
                floor[t, g * group:(g + 1) * group] = vs[at, g].max() * (vu[at, g] - vz[at, g]).abs().sum(0)
                terms = (rows_q.abs() @ ku[at, g].T + rows_q.sum(1).abs()[:, None] * kz[at, g].T.abs()) * ks[at, g].T * scale
                score_size = max(score_size, float(terms.max()))
                score_rms = max(score_rms, float((rows_q ** 2 @ (k ** 2).T).max()) ** 0.5 * scale)
    return out, size, score_size, floor, score_rms


def check_attention(got, ref, what=""):
    """|got - out| <= eps * size, and for bf16 results half a step, 2^-8, of the value.

    A score is a sum of exact products in fp32 and its zero's term. The tensor cores add sixteen
    products at a time and truncate (2^-23 of the size S of the terms each, eight steps); the zero's
    term, the scale and the row's factor are five roundings of 2^-24: 11 * 2^-23 S at most. A weight
    is off by that, relatively, and by ex2's 2^-22; both enter the numerator and the sum of weights.
    For fp32 results a weight is two fp16 terms, 2^-22 of it at most; for bf16 results one, half a
    step of fp16: 2^-11. The sums: truncated chains of at most 32 products (fp32 results) or of one
    warp's run (bf16 results; at most 2000 slots here, two terms per 16: 250) of 2^-23 each, and
    rounded sums of 2^-24 per join: 2^-17 covers both with a value sum of up to 64 such steps, and
    2^-14 the long chain. A weight's fp16 terms end at steps of 2^-24: with the row's reference such
    that the largest weight of its block's largest value scale is 2^8 or more, half of that is 2^-33
    of the largest weight, for each slot: 2^-33 * floor.

    The kernel for chunks of prompts ("prefill", bf16 results) rounds (c - z) s of the keys to fp16:
    128 independent errors of at most half a step, 2^-11, so a score is off by a sum of standard
    deviation 2^-11 / sqrt(3) times the root of its squared terms; eight of those, twice as above."""
    out, size, s, floor, s2 = ref
    got = got.double().cpu()
    bf16 = what in ("bf16", "prefill")
    eps = 2 * (11 * 2 ** -23 * s + 2 ** -22) + (2 ** -11 + 2 ** -14 if bf16 else 2 ** -22 + 2 ** -17)
    if what == "prefill":
        eps += 2 * 8 * 2 ** -11 / 3 ** 0.5 * s2
    rows = ~torch.isnan(out[:, 0, 0])
    tol = eps * size + 2 ** -33 * floor + (2 ** -8 * out.abs() if bf16 else 0)
    bad = ((got - out).abs() > tol + 1e-30)[rows]
    assert torch.isfinite(got[rows]).all()
    assert not bad.any(), f"{int(bad.sum())} elements off, worst {float(((got - out).abs() / (tol + 1e-30))[rows].max()):.3g} x"


class Pool:
    """The pool's rules, one row after another."""

    def __init__(self, pages, page, table, lens, refs, stack):
        self.pages, self.page = pages, page
        self.table, self.lens, self.refs, self.stack = table, lens, refs, stack  # lists

    def reserve(self, add):
        status, free, asked = [], len(self.stack), 0
        cols = len(self.table[0])
        for b, n in enumerate(add):
            length = self.lens[b]
            if n < 0 or length < 0 or length > cols * self.page or -(-(length + n) // self.page) > cols:
                status.append(2)
                continue
            have = -(-length // self.page)
            want = -(-(length + n) // self.page) - have
            asked += want
            if want and asked > free:
                status.append(1)
                continue
            for j in range(want):
                page = self.stack.pop()
                self.table[b][have + j] = page
                self.refs[page] = 1
            self.lens[b] = length + n
            status.append(0)
        return status

    def fork(self, parents, children):
        """(status, [(source page, new page, slots)])"""
        status, copies, free, asked = [], [], len(self.stack), 0
        lens = list(self.lens)
        taken = set()
        rows, cols = len(self.table), len(self.table[0])
        for p, c in zip(parents, children):
            if not (0 <= p < rows and 0 <= c < rows) or p == c or lens[c] != 0 or c in taken or lens[p] < 0 \
                    or lens[p] > cols * self.page:
                status.append(2)
                continue
            taken.add(c)
            full, tail = divmod(lens[p], self.page)
            asked += tail > 0
            if tail and asked > free:
                status.append(1)
                continue
            row = [-1] * cols
            for j in range(full):
                row[j] = self.table[p][j]
                if 0 <= row[j] < self.pages:
                    self.refs[row[j]] += 1
            if tail:
                row[full] = self.stack.pop()
                self.refs[row[full]] = 1
                copies.append((self.table[p][full], row[full], tail))
            self.table[c], self.lens[c] = row, lens[p]
            status.append(0)
        return status, copies

    def free(self, rows):
        gone = []
        for r in rows:
            if not 0 <= r < len(self.table):
                continue
            if self.lens[r] <= 0:
                self.lens[r] = 0
                continue
            for j in range(min(-(-self.lens[r] // self.page), len(self.table[r]))):
                page = self.table[r][j]
                if 0 <= page < self.pages and self.refs[page] > 0:
                    self.refs[page] -= 1
                    if self.refs[page] == 0:
                        gone.append(page)
            self.table[r] = [-1] * len(self.table[r])
            self.lens[r] = 0
        self.stack += sorted(gone)
