"""Attention over the INT4 KV cache in pages where numbers leave the usual range: NaN queries,
scales and zeros that are not finite and are seen by some rows of a tile only, scales far apart,
large scores, long sequences. Against the binary64 statement."""
import functools
import math

import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged_attn import make, run

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# (lens, nq, hq, hkv): one warp writes the row; warps of a block join it; blocks join it; several
# tokens; the kernel for chunks of prompts, in the first half of a block and in the second
SHAPES = {"short": ([50, 40], [1, 1], 8, 2), "joined in a block": ([460], [1], 8, 2),
          "joined by blocks": ([40000, 300], [1, 1], 8, 2), "drafts": ([3000, 70], [4, 2], 64, 8),
          "chunk": ([900, 333], [500, 300], 32, 8), "chunk, one head": ([1700], [1700], 8, 8)}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_nan_queries_give_nan(spin_gpu, shape, dtype):
    """A NaN (or an infinite) query row is not hidden behind a 0, and no other row knows of it."""
    lens, nq, hq, hkv = SHAPES[shape]
    q, cache, table, cu = make(lens, nq, hq, hkv, 64, seed=1)
    tokens = q.shape[0]
    bad = sorted({0, tokens // 3, tokens - 1})
    for t in bad:
        q[t] = math.nan
    inf = tokens // 2 if tokens > 4 else None
    if inf is not None:
        q[inf, :, 5] = math.inf
    q[bad[0], 1] = 0.5  # a head of the same token that is fine
    got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=dtype)
    want = ref.attention(torch.nan_to_num(q, 1.0, 1.0, 1.0), cache, table, lens, cu)
    for t in bad:
        whole = torch.ones(hq, dtype=torch.bool, device="cuda")
        whole[1] = t != bad[0]
        assert torch.isnan(got[t, whole]).all(), t
    assert torch.isfinite(got[bad[0], 1]).all()
    rows = [t for t in range(tokens) if t not in bad[1:] and t != inf]
    if inf is not None:
        assert not torch.isfinite(got[inf]).any()
    fine = torch.zeros(tokens, hq, dtype=torch.bool)
    fine[rows] = True
    fine[bad[0]] = False
    fine[bad[0], 1] = True
    got = torch.where(fine[..., None].cuda(), got, want[0].to(got.dtype).cuda())
    what = "" if dtype == F32 else "prefill" if shape.startswith("chunk") else "bf16"
    ref.check_attention(got, want, what)


def sees(lens, nq, slot, window=0, sinks=0):
    """Which tokens of the first sequence see its slot `slot`, as a mask over all tokens."""
    p = torch.arange(lens[0] - nq[0], lens[0])
    m = torch.zeros(sum(nq), dtype=torch.bool)
    m[:nq[0]] = (slot <= p) & ((p - slot < window) | (slot < sinks) if window else torch.ones_like(p, dtype=torch.bool))
    return m


def poison(cache, table, page, slot, **steps):
    for name, value in steps.items():
        cache[name][table[0, slot // page].item(), :, slot % page] = value


# several tokens: tiles of 8 and 16 rows, chunks; a slot in the middle of the new ones; windows that leave it
SOME = {"two heads": ([300, 40], [5, 1], 2, 2, {}), "drafts": ([3000, 70], [4, 2], 64, 8, {}),
        "drafts, window": ([1000, 70], [6, 2], 32, 8, dict(window=3)), "chunk": ([900, 333], [500, 300], 32, 8, {}),
        "chunk, window": ([900, 333], [500, 300], 32, 8, dict(window=100, sinks=3))}


def some(shape, seed):
    lens, nq, hq, hkv, kw = SOME[shape]
    q, cache, table, cu = make(lens, nq, hq, hkv, 32, seed=seed)
    slot = lens[0] - nq[0] + nq[0] // 2
    assert 0 < sees(lens, nq, slot, **kw).sum() < nq[0]
    return lens, nq, q, cache, table, cu, kw, slot, sees(lens, nq, slot, **kw)


@functools.lru_cache(maxsize=None)
def without(shape, seed):
    """The statement of some(shape, seed) as it is, for the rows that do not see what a test changes."""
    lens, nq, q, cache, table, cu, kw, _, _ = some(shape, seed)
    return ref.attention(q, cache, table, lens, cu, **kw)


def check_unseen(got, want, mask, what):
    """The rows that do not see the slot, against the statement without it."""
    got = torch.where(mask[:, None, None].cuda(), want[0].to(got.dtype).cuda(), got)
    ref.check_attention(got, want, what)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [dict(k_scale=math.nan), dict(k_scale=math.inf), dict(k_scale=-math.inf),
                                 dict(k_zero=math.nan), dict(k_zero=-math.inf), dict(k_scale=math.inf, k_zero=0)])
@pytest.mark.parametrize("shape", SOME)
def test_key_scales_that_are_not_finite(spin_gpu, shape, bad, dtype):
    """The rows that see the slot are NaN, the others do not know of it, in the same tile too."""
    lens, nq, q, cache, table, cu, kw, slot, mask = some(shape, 2)
    want = without(shape, 2)
    poison(cache, table, 32, slot, **bad)
    got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=dtype, **kw)
    assert torch.isnan(got[mask]).all()
    check_unseen(got, want, mask, "bf16" if dtype == BF16 else "")


@pytest.mark.parametrize("scale", [60000.0, -60000.0, 2.0 ** -24, 0.0])
@pytest.mark.parametrize("shape", SOME)
def test_key_scales_far_apart(spin_gpu, shape, scale):
    """One slot's key scale is far from the others': the rows that do not see it are as exact as ever,
    and so are those that do."""
    lens, nq, q, cache, table, cu, kw, slot, mask = some(shape, 3)
    cache["k_scale"] *= 0.02
    poison(cache, table, 32, slot, k_scale=scale)
    kw = dict(kw, scale=2.5)
    want = ref.attention(q, cache, table, lens, cu, **kw)
    alone = dict(cache, k_scale=cache["k_scale"].clone())
    poison(alone, table, 32, slot, k_scale=0.0)
    s = ref.attention(q, alone, table, lens, cu, **kw)[2]  # size of the scores the unseeing rows meet
    kw["softmax_scale"] = kw.pop("scale")
    got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=BF16, **kw)
    check_unseen(got, (want[0], want[1], s, *want[3:]), mask, "bf16")
    ref.check_attention(got, want, "bf16")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("most", [20, 57])
@pytest.mark.parametrize("shape", ["drafts", "chunk", "chunk, window"])
def test_large_scores(spin_gpu, shape, most, dtype):
    """Queries that follow keys, whose elements are of one size: an error in a key's factor would be one
    in every product of its score."""
    lens, nq, q, cache, table, cu, kw, _, _ = some(shape, 4)
    g = torch.Generator().manual_seed(5)
    signs = torch.randint(0, 2, (64,), generator=g) * 12 + (torch.randint(0, 2, (64,), generator=g) * 12 << 4)
    cache["k_cache"][:] = signs.to(torch.uint8).cuda()  # codes 0 and 12 about a zero of 6
    cache["k_zero"].fill_(6)
    cache["k_scale"] = (0.2 + 0.002 * torch.rand(cache["k_scale"].shape, generator=g)).half().cuda()
    q[:] = torch.stack([signs & 15, signs >> 4], -1).flatten().cuda() / 6 - 1
    scale = most / (6 * 0.201 * 128)
    want = ref.attention(q, cache, table, lens, cu, scale=scale, **kw)
    got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=dtype, softmax_scale=scale, **kw)
    ref.check_attention(got, want, "bf16" if dtype == BF16 else "")


@pytest.mark.parametrize("shape", ["drafts", "chunk"])
def test_query_rows_of_all_sizes(spin_gpu, shape):
    """Rows of one tile from 2^-60 to 2^40 with a softmax scale for each, rows of zeros, and keys whose
    scales keep the largest scores near 10."""
    lens, nq, q, cache, table, cu, kw, _, _ = some(shape, 6)
    g = torch.Generator().manual_seed(7)
    for top in (0, 40):
        e = torch.randint(-60, 1, q.shape[:2], generator=g).float() + top
        e[::3] = top
        rows = (torch.randn(q.shape, generator=g) * torch.exp2(e)[..., None]).bfloat16()
        rows[1] = 0
        rows = rows.cuda()
        want = ref.attention(rows, cache, table, lens, cu, scale=2.0 ** -top / 10, **kw)
        got = run(spin_gpu, rows, cache, table, lens, cu, out_dtype=BF16, softmax_scale=2.0 ** -top / 10, **kw)
        ref.check_attention(got, want, "bf16")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [dict(v_scale=math.nan), dict(v_scale=math.inf), dict(v_scale=-math.inf),
                                 dict(v_zero=math.nan), dict(v_zero=math.inf), dict(v_zero=-math.inf, v_scale=0)])
@pytest.mark.parametrize("shape", SOME)
def test_value_scales_that_are_not_finite(spin_gpu, shape, bad, dtype):
    """As for keys: a weight of 0 leaves nothing of such a value in the rows that do not see it."""
    lens, nq, q, cache, table, cu, kw, slot, mask = some(shape, 8)
    want = without(shape, 8)
    poison(cache, table, 32, slot, **bad)
    got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=dtype, **kw)
    assert torch.isnan(got[mask]).all()
    check_unseen(got, want, mask, "bf16" if dtype == BF16 else "")


def test_value_scales_that_are_not_finite_among_zeros_between_the_codes(spin_gpu):
    from tests.test_gpu_paged_attn import odd_zeros
    for shape in SOME:
        lens, nq, q, cache, table, cu, kw, slot, mask = some(shape, 9)
        want = odd_zeros(q, cache, table, lens, cu, 10, **kw)
        poison(cache, table, 32, slot, v_zero=math.nan)
        poison(cache, table, 32, slot + 1, v_scale=math.inf)
        for dtype in (F32, BF16):
            got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=dtype, **kw)
            seen = mask | sees(lens, nq, slot + 1, **kw)
            assert torch.isnan(got[seen]).all()
            check_unseen(got, want, seen, "prefill" if dtype == BF16 else "")


def weight_floor(q, cache, table, lens, cu, page, scale, window=0, sinks=0):
    """Per element max_j p_j |s_j| times sum_j |c_j - z_j|: a weight p_j s_j ends at steps of 2^-24 where a
    row's largest is 2^8 or more, so half a step is 2^-33 of that for each slot; 2^3 and 2^-28 in the
    kernel for chunks."""
    tokens, hq, _ = q.shape
    hkv, out = cache["k_cache"].shape[1], torch.zeros(q.shape, dtype=torch.float64)
    for b, n in enumerate(lens):
        slots = torch.arange(n)
        ids = table[b].cpu()[slots // page].long()

        def rows(name):
            x = cache[name + "_cache"].cpu()[ids, :, slots % page]
            z, s = (cache[name + e].cpu()[ids, :, slots % page].double()[..., None] for e in ("_zero", "_scale"))
            return torch.stack([x & 15, x >> 4], -1).flatten(-2).double() - z, s  # [n, hkv, 128]

        (k, ks), (v, vs) = rows("k"), rows("v")
        p = torch.arange(n - (cu[b + 1] - cu[b]), n)[:, None]
        hidden = (slots > p) | ((p - slots >= window) & (slots >= sinks) if window else torch.zeros(()).bool())
        for h in range(hq):
            g = h * hkv // hq
            score = q[cu[b]:cu[b + 1], h].double().cpu() @ (k * ks)[:, g].T * scale
            w = torch.softmax(score.masked_fill(hidden, -math.inf), 1) * vs[:, g, 0].abs()
            out[cu[b]:cu[b + 1], h] = w.amax(1, keepdim=True) * ((~hidden).double() @ v[:, g].abs())
    return out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("small", [2.0 ** -16, 2.0 ** -9])
@pytest.mark.parametrize("shape", SOME)
def test_value_scales_far_apart(spin_gpu, shape, small, dtype):
    """One slot has a value scale of 60000 and scores below the others' by about 25, the others have scales
    of 2^-16 or 2^-9: neither its scale nor its tile's largest one may cost the others their bits, in the
    rows that see it and in those that do not."""
    lens, nq, q, cache, table, cu, kw, slot, mask = some(shape, 11)
    g = torch.Generator().manual_seed(12)
    q += 1
    cache["v_scale"] = (small * (1 + torch.rand(cache["v_scale"].shape, generator=g))).half().cuda()
    cache["k_scale"] *= 0.1
    poison(cache, table, 32, slot, v_scale=60000.0, k_scale=0.28, k_zero=8)
    cache["k_cache"][table[0, slot // 32].item(), :, slot % 32] = 0
    want = ref.attention(q, cache, table, lens, cu, **kw)
    floor = weight_floor(q, cache, table, lens, cu, 32, 128 ** -0.5, **kw)
    if dtype == BF16 and shape.startswith("chunk"):
        floor = 32 * floor
    got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=dtype, **kw)
    ref.check_attention(got, (*want[:3], floor, want[4]), "bf16" if dtype == BF16 else "")


@pytest.mark.parametrize("most,dtype", [(4096, BF16), (1, BF16), (1, F32), (4, F32)])
def test_long_sums_are_not_too_small(spin_gpu, most, dtype):
    """262144 slots of positive values: tensor cores truncate as they add, which a long chain of sums
    shows as results that are too small on average. Chains of at most 256 products of 2^-23 each, 2^-15
    together, for bf16 results; of 16 for fp32 ones, 2^-19, whose other errors (sums of at most 2^12
    rounded terms, 2^-24 each and of either sign; weights of 2^-22) stay below 2^-17 on average. Results
    differ by several bf16 steps (a row's weight lies on some 1000 slots), so their 8192 roundings of at
    most 2^-8 are of either sign: their mean is below 2^-13, four standard deviations of
    2^-8 / sqrt(3 * 8192) < 2^-15."""
    n, nq, hq, page = 1 << 18, 4096, 4, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = spin_gpu.alloc_kv_cache(n // page, 1, page)
    for name in ref.CODES:
        cache[name].copy_(torch.randint(0, 256, cache[name].shape, generator=g, device="cuda", dtype=torch.uint8))
    cache["k_scale"].fill_(0.5)
    cache["k_zero"].fill_(7)
    cache["v_scale"].copy_(0.05 + 0.4 * torch.rand(cache["v_scale"].shape, generator=g, device="cuda"))
    q = torch.randn((nq, hq, 128), generator=g, device="cuda").bfloat16()
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None].contiguous()
    got = run(spin_gpu, q, cache, table, [n], [0, nq], max_q_len=most, out_dtype=dtype)

    def rows(name):
        x = cache[name + "_cache"][:, 0].reshape(n, 64)
        z, s = (cache[name + e].reshape(n, 1).double() for e in ("_zero", "_scale"))
        return (torch.stack([x & 15, x >> 4], -1).flatten(1).double() - z) * s

    k, v = rows("k"), rows("v")
    tokens = torch.arange(0, nq, nq // 16, device="cuda")
    off = []
    for h in range(hq):
        score = q[tokens, h].double() @ k.T / math.sqrt(128)
        score.masked_fill_(torch.arange(n, device="cuda") > n - nq + tokens[:, None], -math.inf)
        want = torch.softmax(score, 1) @ v
        off.append((got[tokens, h].double() - want) / want)
    mean = float(torch.stack(off).mean())
    assert abs(mean) < (2 ** -15 + 2 ** -13 if dtype == BF16 else 2 ** -17), mean


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", ["drafts", "chunk"])
def test_infinite_queries_among_tiny_ones(spin_gpu, shape, dtype):
    """An infinite query whose scores are all +inf gives NaN, whatever the sizes of the rows beside it."""
    lens, nq, q, cache, table, cu, kw, _, _ = some(shape, 13)
    for name in ("k_cache", "k_zero"):
        cache[name].fill_(0 if name == "k_zero" else 0x33)
    q *= 2.0 ** -50
    q[nq[0] // 2] = 1
    q[nq[0] // 2, :, 7] = math.inf
    got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=dtype, **kw)
    rows = torch.ones(q.shape[0], dtype=torch.bool)
    rows[nq[0] // 2] = False
    assert torch.isnan(got[~rows]).all() and torch.isfinite(got[rows]).all()
    q[nq[0] // 2] = 0
    want = ref.attention(q, cache, table, lens, cu, **kw)
    check_unseen(got, want, ~rows, "bf16" if dtype == BF16 else "")
