"""The paged INT4 KV cache's operators as measurable cases: attention that reads pages,
copies of pages and of slots, and the page table's fork, reserve and free.

A case is a dict of plain values. `prepare` builds what a serving program holds before the
call (the page pool, block tables, queries), `run` makes one pass through the operator: in
plain 32-bit torch operations, or through the package's entry points when `own` is set.
`exact` gives attention's result in binary64, `work` what a pass has to move and compute.
"""
import math
import random

import torch

own = False

D = 128                 # head_dim of the cache
CODES = ("k_cache", "v_cache")
STEPS = ("k_scale", "k_zero", "v_scale", "v_zero")
SLOT_BYTES = 2 * (D // 2 + 4)  # one slot of one kv head: K and V codes, fp16 scales and zeros


# ---------------------------------------------------------------- cases
def listed():
    att = dict(op="attention", seqs=1, len_min=1, len_max=1, q_min=1, q_max=1, hq=32, hkv=8, page=64, window=0,
               sinks=0, f32=False, mix=0)
    return [
        # one chat turn of a single user: every microsecond of latency counts
        dict(att, name="decode_one", len_min=257, len_max=257, page=16),
        # a serving batch of ragged conversations, one token each
        dict(att, name="decode_batch", seqs=32, len_max=4096, mix=1),
        # few very long documents, fp32 out for a caller that merges results itself
        dict(att, name="decode_long_f32", seqs=4, len_min=40001, len_max=65537, page=128, f32=True, mix=2),
        # four drafted tokens per sequence checked at once, sliding window with sink tokens
        dict(att, name="draft_window", seqs=16, len_min=900, len_max=32768, q_min=4, q_max=4, hq=64, page=32,
             window=4096, sinks=4, mix=3),
        # a chunk of prompt over a cached prefix, ragged
        dict(att, name="prefill_chunk", seqs=3, len_min=2100, len_max=4096, q_min=1027, q_max=2048, mix=4),
        # a handful of pages moved between users' tables (8 heads, 16 slots each)
        dict(op="copy_pages", name="copy_pages_few", pages=8, pool=64, hkv=8, page=16),
        # a pool being defragmented: 4096 pages of 64 slots, 285 MB read and written
        dict(op="copy_pages", name="copy_pages_many", pages=4096, pool=8448, hkv=8, page=64),
        # accepted draft tokens pulled together after a verification step
        dict(op="copy_slots", name="keep_draft", seqs=32, len_max=8, keep_max=5, hkv=8, page=16, dst_page=64, mix=5),
        # long sequences cut down to the slots an eviction policy kept
        dict(op="copy_slots", name="keep_window", seqs=8, len_max=32768, keep_max=20011, hkv=8, page=64, dst_page=64,
             mix=6),
        # one request branching into a few beams
        dict(op="beam_step", name="beam_few", parents=1, beams=4, len_min=700, len_max=700, hkv=8, page=64, mix=7),
        # a large batch branching: 1024 children of 256 sequences, most pages shared
        dict(op="beam_step", name="beam_many", parents=256, beams=4, len_min=33, len_max=2048, hkv=8, page=64, mix=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "copy_pages", "copy_slots", "beam_step"])
    page = rng.choice([16, 32, 64, 128])
    if op == "attention":
        hq, hkv = rng.choice([(32, 8), (8, 8), (64, 8), (16, 8), (8, 4), (32, 4), (12, 4)])
        window = rng.choice([0, 0, _log(rng, 16, 8192)])
        c = dict(op=op, hq=hq, hkv=hkv, page=page, window=window, sinks=rng.choice([0, 1, 4, 37]) if window else 0,
                 f32=rng.random() < 0.3, mix=rng.randrange(1000))
        if rng.random() < 0.3:  # prompts in chunks
            q_max = _log(rng, 17, 1500)
            len_max = q_max + _log(rng, 1, 2000)
            return dict(c, seqs=rng.randint(1, 3), len_min=len_max - len_max // 3, len_max=len_max,
                        q_min=max(1, q_max // 2), q_max=q_max)
        seqs = _log(rng, 1, 64)
        len_max = _log(rng, 8, 65536 * 4 // max(4, seqs))
        q_max = rng.choice([1, 1, 1, 2, 5, 8])
        return dict(c, seqs=seqs, len_min=rng.randint(1, len_max), len_max=len_max, q_min=rng.randint(1, q_max),
                    q_max=q_max)
    hkv = rng.choice([1, 2, 4, 8])
    if op == "copy_pages":
        pages = _log(rng, 1, 4096 * 64 // page // 2)
        return dict(op=op, pages=pages, pool=2 * pages + rng.randint(1, 40), hkv=hkv, page=page)
    if op == "copy_slots":
        seqs = _log(rng, 1, 64)
        len_max = _log(rng, 4, 32768 * 8 // max(8, seqs))
        return dict(op=op, seqs=seqs, len_max=len_max, keep_max=rng.randint(1, len_max), hkv=hkv, page=page,
                    dst_page=rng.choice([16, 32, 64]), mix=rng.randrange(1000))
    len_max = _log(rng, 5, 2048)
    return dict(op=op, parents=_log(rng, 1, 250), beams=rng.randint(1, 4), len_min=rng.randint(1, len_max),
                len_max=len_max, hkv=hkv, page=page, mix=rng.randrange(1000))


def _ragged(n, lo, hi, mix):
    """n whole numbers spread over lo .. hi, the last one hi, the same for every seed."""
    r = random.Random(mix)
    return [r.randint(lo, hi) for _ in range(n - 1)] + [hi]


def _lens(c):
    lens = _ragged(c["seqs"], c["len_min"], c["len_max"], c["mix"])
    nq = _ragged(c["seqs"], c["q_min"], c["q_max"], c["mix"] + 1)
    return [max(a, b) for a, b in zip(lens, nq)], nq  # the new tokens are in the cache already


def _keeps(c):
    lens = _ragged(c["seqs"], 1, c["len_max"], c["mix"])
    return lens, [min(a, b) for a, b in zip(lens, _ragged(c["seqs"], 0, c["keep_max"], c["mix"] + 1))]


# ---------------------------------------------------------------- inputs
def _quantise(x):
    """[..., 128] values -> packed codes, scale, zero by the cache's asymmetric rule (clip 0.95)."""
    lo = (x.amin(-1) * 0.95).clamp(max=0)
    hi = (x.amax(-1) * 0.95).clamp(min=0)
    scale = ((hi - lo) / 15).half()
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    zero = (-lo / scale.float()).round().clamp(0, 15)
    u = ((x / scale.float()[..., None]).round() + zero[..., None]).clamp(0, 15).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), scale, zero.half()


def _values(g, pages, hkv, page):
    """A pool written by the R3 kernel in earnest: rotated keys are near Gaussian, values
    keep two outlier dims per head."""
    k = torch.randn((pages, hkv, page, D), generator=g, device="cuda")
    kc, ks, kz = _quantise(k)
    del k
    v = torch.randn((pages, hkv, page, D), generator=g, device="cuda")
    v[..., torch.randint(0, D, (2,), generator=g, device="cuda")] *= 50
    vc, vs, vz = _quantise(v)
    return dict(k_cache=kc, v_cache=vc, k_scale=ks, k_zero=kz, v_scale=vs, v_zero=vz)


def _bytes(g, pages, hkv, page):
    """A pool of arbitrary contents, for operators that only move them."""
    c = {n: torch.randint(0, 256, (pages, hkv, page, D // 2), generator=g, device="cuda", dtype=torch.uint8)
         for n in CODES}
    c.update({n: torch.rand((pages, hkv, page), generator=g, device="cuda").half() for n in STEPS})
    return c


def _dev(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(perm, lens, page, cols):
    """Block tables [seqs, cols] that hand out the pages of `perm` in order, -1 behind a
    sequence's last page, and how many pages they took."""
    held = torch.tensor([-(-n // page) for n in lens], device="cuda")
    col = torch.arange(cols, device="cuda")
    place = (held.cumsum(0) - held)[:, None] + col
    used = sum(-(-n // page) for n in lens)
    return torch.where(col < held[:, None], perm[place.clamp(max=perm.numel() - 1)], -1).int(), used


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "attention":
        lens, nq = _lens(c)
        pages = sum(-(-n // c["page"]) for n in lens) + 3
        cache = _values(g, pages, c["hkv"], c["page"])
        table, _ = _tables(torch.randperm(pages, generator=g, device="cuda"), lens, c["page"],
                           -(-max(lens) // c["page"]))
        q = torch.randn((sum(nq), c["hq"], D), generator=g, device="cuda").bfloat16()
        cu = [0]
        for n in nq:
            cu.append(cu[-1] + n)
        return dict(case=c, q=q, cache=cache, table=table, lens=_dev(lens), cu_q=_dev(cu), max_q=max(nq))
    if c["op"] == "copy_pages":
        perm = torch.randperm(c["pool"], generator=g, device="cuda").int()
        return dict(case=c, cache=_bytes(g, c["pool"], c["hkv"], c["page"]), src=perm[:c["pages"]].contiguous(),
                    dst=perm[c["pages"]:2 * c["pages"]].contiguous())
    if c["op"] == "copy_slots":
        lens, keeps = _keeps(c)
        n_src = sum(-(-n // c["page"]) for n in lens)
        n_dst = sum(-(-n // c["dst_page"]) for n in keeps) + 1
        src_table, _ = _tables(torch.randperm(n_src, generator=g, device="cuda"), lens, c["page"],
                               -(-max(lens) // c["page"]))
        dst_table, _ = _tables(torch.randperm(n_dst, generator=g, device="cuda"), keeps, c["dst_page"],
                               max(1, -(-max(keeps) // c["dst_page"])))
        keep = [torch.randperm(a, generator=g, device="cuda")[:b].sort()[0] for a, b in zip(lens, keeps)]
        cu = [0]
        for n in keeps:
            cu.append(cu[-1] + n)
        return dict(case=c, cache=_bytes(g, n_src, c["hkv"], c["page"]), src_table=src_table,
                    dst=_bytes(g, n_dst, c["hkv"], c["dst_page"]), dst_table=dst_table,
                    keep=torch.cat(keep).int(), cu_keep=_dev(cu))
    # parents hold their pages, the children's rows are empty; each pass lets the children of
    # the pass before go, branches again and makes room for a token per child
    n, kids = c["parents"], c["parents"] * c["beams"]
    lens = _ragged(n, c["len_min"], c["len_max"], c["mix"])
    used = sum(-(-x // c["page"]) for x in lens)
    pool = used + 2 * kids + 5
    perm = torch.randperm(pool, generator=g, device="cuda")
    cols = -(-(max(lens) + 1) // c["page"])
    table, _ = _tables(perm, lens, c["page"], cols)
    cache = _bytes(g, pool, c["hkv"], c["page"])
    cache["refs"] = torch.zeros(pool, dtype=torch.int32, device="cuda")
    cache["refs"][perm[:used]] = 1
    cache["free_pages"] = torch.cat([perm[used:], torch.zeros_like(perm[:used])]).int()
    cache["free_count"] = _dev([pool - used])
    children = torch.arange(n, n + kids, device="cuda").int()
    return dict(case=c, pool=cache, table=torch.cat([table, table.new_full((kids, cols), -1)]),
                lens=torch.cat([_dev(lens), _dev([0] * kids)]),
                parents=torch.randint(0, n, (kids,), generator=g, device="cuda").int(), children=children,
                add=torch.cat([_dev([0] * n), _dev([1] * kids)]))


# ---------------------------------------------------------------- plain forms
def _plain_rows(cache, name, table):
    """Dequantised K or V of every table row as [seqs, hkv, slots, 128] fp32."""
    at = table.clamp(min=0).long()
    codes = cache[name + "_cache"][at]  # [seqs, cols, hkv, page, 64]
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    x = (u - cache[name + "_zero"][at].float()[..., None]) * cache[name + "_scale"][at].float()[..., None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attention(s):
    c, q, cu = s["case"], s["q"], s["cu_q"].long()
    tokens, hq, _ = q.shape
    seqs, hkv, mq = s["lens"].numel(), c["hkv"], s["max_q"]
    k, v = _plain_rows(s["cache"], "k", s["table"]), _plain_rows(s["cache"], "v", s["table"])
    i = torch.arange(mq, device=q.device)
    nq = cu[1:] - cu[:-1]
    rows = q[(cu[:-1, None] + i).clamp(max=tokens - 1)].float()  # [seqs, mq, hq, 128]
    rows = rows.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = torch.matmul(rows, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    score = score.unflatten(2, (hq // hkv, mq))
    pos = s["lens"].long()[:, None] - nq[:, None] + i  # [seqs, mq]
    j = torch.arange(k.shape[2], device=q.device)
    seen = (j <= pos[..., None]) & (pos[..., None] >= 0)
    if c["window"]:
        seen &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    seen = seen[:, None, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.clamp(min=-3e38))
    out = torch.matmul((p / p.sum(-1, keepdim=True).clamp(min=1e-30)).flatten(2, 3), v)
    out = out.unflatten(2, (hq // hkv, mq)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [seqs, mq, hq, 128]
    t = torch.arange(tokens, device=q.device)
    b = torch.bucketize(t, cu[1:], right=True)
    out = out[b, t - cu[b]]
    return out if c["f32"] else out.bfloat16()


def _plain_copy_slots(s):
    cu, e = s["cu_keep"].long(), torch.arange(s["keep"].numel(), device="cuda")
    row = torch.bucketize(e, cu[1:], right=True)
    src, dst = s["keep"].long(), e - cu[row]
    a, b = s["case"]["page"], s["case"]["dst_page"]
    sp, dp = s["src_table"][row, src // a].long(), s["dst_table"][row, dst // b].long()
    for name in CODES + STEPS:
        s["dst"][name][dp, :, dst % b] = s["cache"][name][sp, :, src % a]
    return s["dst"]


def _plain_free(pool, table, lens, rows, page):
    held = table[rows].long()
    inside = torch.arange(table.shape[1], device="cuda") < ((lens[rows] + page - 1) // page)[:, None]
    refs = pool["refs"]
    drop = torch.zeros(refs.numel() + 1, dtype=torch.int32, device="cuda")
    drop.index_add_(0, torch.where(inside, held, refs.numel()).flatten(),
                    torch.ones(held.numel(), dtype=torch.int32, device="cuda"))
    refs -= drop[:-1]
    gone = ((drop[:-1] > 0) & (refs == 0)).nonzero()[:, 0]
    count = pool["free_count"]
    pool["free_pages"][count + torch.arange(gone.numel(), device="cuda")] = gone.int()
    count += gone.numel()
    table[rows] = -1
    lens[rows] = 0


def _plain_fork(pool, table, lens, parents, children, page):
    n = lens[parents].long()
    full, tail = n // page, n % page
    need = tail > 0
    total = need.long().cumsum(0)
    fits = ~need | (total <= pool["free_count"])
    new = pool["free_pages"][(pool["free_count"] - total).clamp(min=0)]
    col = torch.arange(table.shape[1], device="cuda")
    shared = col < full[:, None]
    rows = torch.where(shared, table[parents], torch.where((col == full[:, None]) & need[:, None], new[:, None], -1))
    table[children] = torch.where(fits[:, None], rows, table[children])
    lens[children] = torch.where(fits, n.int(), lens[children])
    at = (shared & fits[:, None]).flatten().nonzero()[:, 0]
    at = rows.flatten()[at]
    pool["refs"].index_add_(0, at, torch.ones_like(at))
    copied = (need & fits).nonzero()[:, 0]
    src, dst = table[parents[copied], full[copied]].long(), new[copied].long()
    pool["refs"][dst] = 1
    inside = torch.arange(page, device="cuda") < tail[copied][:, None, None]
    for name in STEPS:
        pool[name][dst] = torch.where(inside, pool[name][src], pool[name][dst])
    for name in CODES:
        pool[name][dst] = torch.where(inside[..., None], pool[name][src], pool[name][dst])
    pool["free_count"] -= (total * fits).amax()
    return (~fits).int()


def _plain_reserve(pool, table, lens, add, page):
    have, want = (lens + page - 1) // page, (lens + add + page - 1) // page
    total = (want - have).long().cumsum(0)
    fits = (total <= pool["free_count"]) | (want == have)
    col = torch.arange(table.shape[1], device="cuda")
    new = (col >= have[:, None]) & (col < want[:, None]) & fits[:, None]
    place = pool["free_count"] - 1 - (total - want + have)[:, None] - (col - have[:, None])
    pages = pool["free_pages"][place.clamp(0, pool["free_pages"].numel() - 1)]
    table.copy_(torch.where(new, pages, table))
    at = new.flatten().nonzero()[:, 0]
    pool["refs"][pages.flatten()[at].long()] = 1
    lens += add * fits
    pool["free_count"] -= (total * fits).amax()
    return (~fits).int()


def run(state):
    s = state
    c = s["case"]
    if own:
        import online_hadamard_rotation_b200 as spin
    if c["op"] == "attention":
        if own:
            return spin.paged_attention_int4kv(s["q"], s["cache"], s["table"], s["lens"], s["cu_q"], s["max_q"],
                                               window=c["window"], sinks=c["sinks"],
                                               out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
        return _plain_attention(s)
    if c["op"] == "copy_pages":
        if own:
            spin.copy_kv_pages(s["cache"], s["src"], s["dst"])
        else:
            src, dst = s["src"].long(), s["dst"].long()
            for name in CODES + STEPS:
                s["cache"][name][dst] = s["cache"][name][src]
        return s["cache"]
    if c["op"] == "copy_slots":
        if own:
            spin.copy_kv_slots(s["cache"], s["src_table"], s["keep"], s["cu_keep"], s["dst"], s["dst_table"])
            return s["dst"]
        return _plain_copy_slots(s)
    pool, table, lens = s["pool"], s["table"], s["lens"]
    if own:
        spin.free_kv_pages(pool, table, lens, s["children"])
        forked = spin.fork_kv_pages(pool, table, lens, s["parents"], s["children"])
        grown = spin.reserve_kv_pages(pool, table, lens, s["add"])
    else:
        _plain_free(pool, table, lens, s["children"], c["page"])
        forked = _plain_fork(pool, table, lens, s["parents"], s["children"], c["page"])
        grown = _plain_reserve(pool, table, lens, s["add"], c["page"])
    return dict(pool, table=table, lens=lens, forked=forked, grown=grown)


# ---------------------------------------------------------------- what a pass needs
def _seen(c, length, nq):
    """(cache slots that any of the nq last tokens sees, visible (token, slot) pairs)."""
    if not c["window"]:
        return length, nq * length - nq * (nq - 1) // 2
    first = max(0, length - nq - c["window"] + 1)  # oldest slot in a window
    slots = min(c["sinks"], first) + length - first
    pairs = sum(min(p + 1, c["window"]) + min(c["sinks"], max(0, p + 1 - c["window"]))
                for p in range(length - nq, length))
    return slots, pairs


def work(case):
    c = case
    if c["op"] == "attention":
        lens, nq = _lens(c)
        seen = [_seen(c, a, b) for a, b in zip(lens, nq)]
        rows = sum(nq) * c["hq"] * D
        table = sum(-(-a // c["page"]) for a, _ in seen) * 4
        return dict(bytes=sum(a for a, _ in seen) * c["hkv"] * SLOT_BYTES + rows * (2 + (4 if c["f32"] else 2)) + table,
                    flops=sum(b for _, b in seen) * c["hq"] * 4 * D)
    if c["op"] == "copy_pages":
        return dict(bytes=c["pages"] * (2 * c["page"] * c["hkv"] * SLOT_BYTES + 8), flops=0)
    if c["op"] == "copy_slots":
        n = sum(_keeps(c)[1])
        return dict(bytes=n * (2 * c["hkv"] * SLOT_BYTES + 4), flops=0)
    # the tails of the children's sequences are copied, their tables read and written
    lens = _ragged(c["parents"], c["len_min"], c["len_max"], c["mix"])
    tail = sum(n % c["page"] for n in lens) / len(lens)
    cols = sum(-(-n // c["page"]) for n in lens) / len(lens)
    kids = c["parents"] * c["beams"]
    return dict(bytes=kids * (2 * tail * c["hkv"] * SLOT_BYTES + 5 * 4 * cols), flops=0)


def exact(case, seed):
    if case["op"] != "attention":
        return None  # bytes and whole numbers are moved, nothing is computed
    s = prepare(case, seed)
    cache, page, hkv = s["cache"], case["page"], case["hkv"]
    lens, nq = _lens(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["hq"] // hkv
    at = 0
    for b, (n, m) in enumerate(zip(lens, nq)):
        pages = s["table"][b, :-(-n // page)].long()

        def rows(name, h):
            packed = cache[name + "_cache"][pages, h].reshape(-1, D // 2)[:n].to(torch.int64)
            code = torch.empty((n, D), dtype=torch.float64, device="cuda")
            code[:, 0::2] = (packed % 16).double()
            code[:, 1::2] = (packed // 16).double()
            step, zero = (cache[name + e][pages, h].reshape(-1)[:n, None].double() for e in ("_scale", "_zero"))
            return step * (code - zero)

        place = torch.arange(n - m, n, device="cuda")[:, None]
        slot = torch.arange(n, device="cuda")[None]
        hidden = slot > place
        if case["window"]:
            hidden |= (place - slot >= case["window"]) & (slot >= case["sinks"])
        for h in range(hkv):
            key, value = rows("k", h), rows("v", h)
            for e in range(h * group, (h + 1) * group):
                logit = s["q"][at:at + m, e].double() @ key.T / math.sqrt(D)
                out[at:at + m, e] = torch.softmax(logit.masked_fill(hidden, -math.inf), 1) @ value
        at += m
    return out
