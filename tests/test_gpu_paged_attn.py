"""Attention over the INT4 KV cache in pages (spin_paged_attention_int4kv) against its
binary64 statement: head groupings, lengths from none to many blocks, several new tokens per
sequence, windows with sinks, page sizes, masked garbage, and how it is called (streams,
graphs, outputs with rows of their own)."""
import math

import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


def make(lens, nq, hq, hkv, page, seed, spare=3, cols=None):
    """Queries, a pool whose pages are dealt out in random order, table (garbage behind a
    sequence's last page), lens, cu."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-max(n, 0) // page) for n in lens]
    pages = sum(held) + spare
    cache = ref.random_pages(pages, hkv, page, seed + 1)
    perm = torch.randperm(pages, generator=g)
    cols = cols or max(1, max(held) + 1)
    table = torch.randint(-5, 2 * pages, (len(lens), cols), generator=g, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = perm[at:at + n].int()
        at += n
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], hq, 128), generator=g).bfloat16().cuda()
    return q, cache, table.cuda(), cu


def run(spin, q, cache, table, lens, cu, **kw):
    most = max([b - a for a, b in zip(cu, cu[1:])] + [1])
    return spin.paged_attention_int4kv(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                       torch.tensor(cu, dtype=torch.int32, device="cuda"), kw.pop("max_q_len", most),
                                       **kw)


def both(spin, lens, nq, hq, hkv, page, seed, **kw):
    q, cache, table, cu = make(lens, nq, hq, hkv, page, seed)
    want = ref.attention(q, cache, table, lens, cu, **kw)
    ref.check_attention(run(spin, q, cache, table, lens, cu, **kw), want)
    ref.check_attention(run(spin, q, cache, table, lens, cu, out_dtype=torch.bfloat16, **kw), want, "bf16")


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [63, 64, 65], [0, 257, 31], [700]])
def test_decode_lengths_and_pages(spin_gpu, lens, page):
    both(spin_gpu, lens, [1] * len(lens), 32, 8, page, seed=len(lens) + page)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (12, 4), (5, 1), (64, 8), (40, 1), (16, 1)])
def test_head_groupings(spin_gpu, hq, hkv):
    both(spin_gpu, [130, 1, 77], [1, 1, 1], hq, hkv, 32, seed=hq)
    both(spin_gpu, [130, 3, 77], [2, 3, 1], hq, hkv, 32, seed=hq + 1)


@pytest.mark.parametrize("nq", [[2, 2], [5, 0], [0, 3], [8, 1], [33, 70], [130, 129]])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 2)])
def test_several_tokens(spin_gpu, nq, hq, hkv):
    both(spin_gpu, [131, 257], nq, hq, hkv, 64, seed=sum(nq))


def test_tokens_before_the_first_slot_see_nothing(spin_gpu):
    """More new tokens than slots: the first ones stand at positions below 0 and give 0."""
    lens, nq = [3, 0, 20], [7, 2, 21]
    q, cache, table, cu = make(lens, nq, 8, 2, 16, seed=4)
    got = run(spin_gpu, q, cache, table, lens, cu)
    ref.check_attention(got, ref.attention(q, cache, table, lens, cu))
    assert (got[:4] == 0).all() and (got[7:10] == 0).all() and (got[4] != 0).any()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (64, 0), (64, 70), (100, 3), (10 ** 9, 5),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (300, 0)])
@pytest.mark.parametrize("nq", [1, 4, 40])
def test_windows_and_sinks(spin_gpu, window, sinks, nq):
    both(spin_gpu, [333, 50, 1024], [nq, nq, 1], 8, 2, 16, seed=window % 97 + nq, window=window, sinks=sinks)


def prefill(spin, lens, nq, hq, hkv, page, seed, **kw):
    """Calls with enough rows for the kernel for chunks of prompts (37 blocks of 256 and more)."""
    assert hkv * sum(nq) * (hq // hkv) // 256 >= 74
    q, cache, table, cu = make(lens, nq, hq, hkv, page, seed)
    want = ref.attention(q, cache, table, lens, cu, **kw)
    got = run(spin, q, cache, table, lens, cu, out_dtype=torch.bfloat16, **kw)
    ref.check_attention(got, want, "prefill")
    assert spin.device_status() == 0
    return q, cache, table, cu, got


@pytest.mark.parametrize("lens,nq,page", [([700, 333, 5], [300, 333, 1], 64), ([640], [640], 16),
                                          ([129, 400, 90, 0, 257], [128, 300, 90, 0, 129], 32),
                                          ([1300, 64], [592, 16], 128)])
def test_chunks_of_prompts(spin_gpu, lens, nq, page):
    prefill(spin_gpu, lens, nq, 32, 8, page, seed=page)


@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 0), (100, 3), (128, 130), (300, 500), (2 ** 31 - 1, 4)])
def test_chunks_of_prompts_windows(spin_gpu, window, sinks):
    prefill(spin_gpu, [900, 400], [400, 300], 32, 8, 32, seed=window % 89, window=window, sinks=sinks)


@pytest.mark.parametrize("hq,hkv,n", [(64, 8, 310), (12, 4, 1600), (8, 8, 2400), (40, 1, 500)])
def test_chunks_of_prompts_head_groupings(spin_gpu, hq, hkv, n):
    prefill(spin_gpu, [n + 77], [n], hq, hkv, 64, seed=hq)


def test_chunks_of_prompts_longer_than_the_cache(spin_gpu):
    """Tokens before the first slot give 0, in a half, a block and a sequence of their own."""
    q, cache, table, cu, got = prefill(spin_gpu, [100, 20], [500, 120], 32, 8, 64, seed=3)
    assert (got[:400] == 0).all() and (got[500:600] == 0).all() and (got[400] != 0).any()


def test_chunks_of_prompts_masked_slots_may_hold_anything(spin_gpu):
    lens, nq = [500, 700], [300, 400]
    q, cache, table, cu = make(lens, nq, 32, 8, 32, seed=5)
    kw = dict(window=100, sinks=40)
    want = ref.attention(q, cache, table, lens, cu, **kw)
    for name, bad in zip(ref.STEPS, (math.nan, math.inf, -math.inf, math.nan)):
        cache[name][table[0, 15].item(), :, 20:] = bad  # behind slot 500
        cache[name][table[0, 1].item(), :, 8:] = bad    # between the sinks and the first window (101)
        cache[name][table[0, 3].item(), :, :5] = bad    # slots 96 .. 100
    table[0, 2] = -1
    table[1, 2:6] = 10 ** 6
    out = torch.full((700, 32, 128), -7.0, dtype=torch.bfloat16, device="cuda")
    got = run(spin_gpu, q, cache, table, lens, cu, out=out, **kw)
    ref.check_attention(got, want, "prefill")
    # a page gone from the middle of what is seen
    table[0, 10] = -1
    ref.check_attention(run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16, **kw),
                        ref.attention(q, cache, table, lens, cu, **kw), "prefill")


def test_chunks_of_prompts_beside_single_tokens(spin_gpu):
    """One call with chunks, drafted tokens and single tokens: both kernels, twice the same bits."""
    lens, nq = [800, 333, 64, 2000, 17, 1500], [400, 1, 64, 3, 17, 200]
    q, cache, table, cu, got = prefill(spin_gpu, lens, nq, 32, 8, 64, seed=6)
    again = run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16)
    assert torch.equal(got, again)


def test_long_sequences_are_cut_and_joined(spin_gpu):
    """Enough units that items are cut over many thread blocks, and several pieces per item."""
    both(spin_gpu, [40000, 9, 12345], [1, 1, 1], 8, 2, 128, seed=11)
    both(spin_gpu, [30001], [3], 32, 8, 64, seed=12)
    both(spin_gpu, [30001], [3], 32, 8, 64, seed=13, window=20000, sinks=100)


def test_many_sequences(spin_gpu):
    lens = [(37 * i) % 201 for i in range(700)]
    both(spin_gpu, lens, [1] * 700, 4, 1, 16, seed=14)


def test_masked_slots_may_hold_anything(spin_gpu):
    """Slots behind a sequence, and slots that left the window, with NaN and infinite scales and
    zeros and with pages that are gone from the table."""
    lens, nq = [70, 200], [2, 1]
    q, cache, table, cu = make(lens, nq, 8, 2, 16, seed=5)
    want = ref.attention(q, cache, table, lens, cu, window=40, sinks=2)
    for name, bad in zip(ref.STEPS, (math.nan, math.inf, -math.inf, math.nan)):
        flat = cache[name]
        flat[table[0, 4].item(), :, 6:] = bad        # behind slot 70
        flat[table[1, 12].item(), :, 8:] = bad       # behind slot 200
        flat[table[1, 9].item(), :, :15] = bad       # slots 144 .. 158, window begins at 160
        flat[table[1, 0].item(), :, 2:] = bad        # behind the sinks
    table[1, 3:9] = -1
    table[1, 5] = 2 ** 31 - 1
    for most in (2, 9, 64):
        got = run(spin_gpu, q, cache, table, lens, cu, window=40, sinks=2, max_q_len=most)
        ref.check_attention(got, want)


def test_page_ids_out_of_range_hide_their_slots(spin_gpu):
    lens, nq = [300, 40], [3, 1]
    q, cache, table, cu = make(lens, nq, 8, 2, 32, seed=6)
    table[0, 2], table[0, 5], table[1, :2] = -1, 10 ** 6, -7
    got = run(spin_gpu, q, cache, table, lens, cu)
    ref.check_attention(got, ref.attention(q, cache, table, lens, cu))
    assert (got[3] == 0).all()  # every page of the second sequence is gone


def test_lengths_and_offsets_are_clamped(spin_gpu):
    q, cache, table, cu = make([64, 64], [1, 1], 8, 2, 32, seed=7, cols=2)
    a = run(spin_gpu, q, cache, table, [64, 64], cu)
    assert torch.equal(a, run(spin_gpu, q, cache, table, [65, 2 ** 31 - 1], cu))
    z = run(spin_gpu, q, cache, table, [-3, 64], cu)
    assert (z[0] == 0).all() and torch.equal(z[1], a[1])
    out = torch.full((2, 8, 128), 5.0, device="cuda")
    run(spin_gpu, q, cache, table, [64, 64], [0, 1, 99], out=out, max_q_len=1)
    assert torch.equal(out, a)


def odd_zeros(q, cache, table, lens, cu, seed, **kw):
    """Any fp16 zeros of -4 .. 20 in the cache, and what check_attention needs for them.

    The narrow kernel splits a value (c - z) s into (c - y) s under the rounded weight, 0 <= c, y < 16, and
    (y - z) s under the fp32 one, |y - z| < 35: its terms are below 50 s. The kernel for chunks rounds
    c - z, |c - z| < 20, to fp16 (half a step, 2^-11, once more beside the weight's): 40 s. 80 s in the
    place of |vhat| bounds both. Its keys (c - z) s are rounded twice, the root of two times the
    deviation: 1.5 here."""
    g = torch.Generator().manual_seed(seed)
    for n in ("k_zero", "v_zero"):
        cache[n] = (24 * torch.rand(cache[n].shape, generator=g) - 4).half().cuda()
    out, _, s, _, s2 = ref.attention(q, cache, table, lens, cu, **kw)
    wide = dict(cache, v_cache=torch.zeros_like(cache["v_cache"]), v_zero=torch.full_like(cache["v_zero"], -80))
    _, size, _, floor, _ = ref.attention(q, wide, table, lens, cu, **kw)
    return out, size, s, floor, 1.5 * s2


@pytest.mark.parametrize("hq,hkv,nq,kw", [(32, 8, 1, {}), (32, 8, 5, dict(window=70, sinks=9)), (5, 5, 1, {})])
def test_zeros_between_the_codes(spin_gpu, hq, hkv, nq, kw):
    lens = [300, 77, 9]
    q, cache, table, cu = make(lens, [nq] * 3, hq, hkv, 32, seed=41)
    want = odd_zeros(q, cache, table, lens, cu, 42, **kw)
    ref.check_attention(run(spin_gpu, q, cache, table, lens, cu, **kw), want)
    ref.check_attention(run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16, **kw), want, "bf16")


def test_zeros_between_the_codes_in_chunks_of_prompts(spin_gpu):
    lens, nq = [600, 333], [400, 222]
    q, cache, table, cu = make(lens, nq, 32, 8, 64, seed=43)
    want = odd_zeros(q, cache, table, lens, cu, 44)
    ref.check_attention(run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16), want, "prefill")


def test_more_and_fewer_tokens_than_expected(spin_gpu):
    """max_q_len chooses a kernel; whatever it says, every token is computed."""
    lens, nq = [400, 90, 33], [300, 4, 1]
    q, cache, table, cu = make(lens, nq, 32, 8, 32, seed=45)
    want = ref.attention(q, cache, table, lens, cu)
    for most in (1, 2, 17, 2 ** 31 - 1):
        ref.check_attention(run(spin_gpu, q, cache, table, lens, cu, max_q_len=most), want)
        ref.check_attention(run(spin_gpu, q, cache, table, lens, cu, max_q_len=most, out_dtype=torch.bfloat16), want,
                            "prefill")
    lens, nq = [1 + i % 40 for i in range(600)], [1] * 600  # enough rows for chunks, and none there
    q, cache, table, cu = make(lens, nq, 32, 8, 16, seed=46)
    got = run(spin_gpu, q, cache, table, lens, cu, max_q_len=100, out_dtype=torch.bfloat16)
    ref.check_attention(got, ref.attention(q, cache, table, lens, cu), "bf16")


def test_tensors_inside_larger_ones(spin_gpu):
    """q and out that begin 16 bytes into their storage, and nothing written around out."""
    lens, nq = [500, 260], [300, 260]
    q, cache, table, cu = make(lens, nq, 32, 8, 32, seed=47)
    want = run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16)
    q2 = torch.full((q.numel() + 16,), 3.0, dtype=torch.bfloat16, device="cuda")
    q2[8:-8] = q.flatten()
    o2 = torch.full_like(q2, -7.0)
    got = run(spin_gpu, q2[8:-8].view(q.shape), cache, table, lens, cu, out=o2[8:-8].view(q.shape))
    assert torch.equal(got, want) and (o2[:8] == -7).all() and (o2[-8:] == -7).all()


def test_chunks_of_prompts_at_once_and_replayed(spin_gpu):
    """Two calls on two streams at once, and a captured one replayed after the lengths changed."""
    lens, nq = [900, 700], [400, 300]
    q, cache, table, cu, want = prefill(spin_gpu, lens, nq, 32, 8, 64, seed=48)
    one, many = make([3000], [1], 32, 8, 64, seed=49), [torch.cuda.Stream() for _ in range(2)]
    single = run(spin_gpu, *one[:3], [3000], one[3])
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for i, s in enumerate(many):
            with torch.cuda.stream(s):
                got.append(run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16) if i == 0 else
                           run(spin_gpu, *one[:3], [3000], one[3]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got[::2]) and all(torch.equal(x, single) for x in got[1::2])
    n, c = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, cu))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = spin_gpu.paged_attention_int4kv(q, cache, table, n, c, 400, out_dtype=torch.bfloat16)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    lens = [650, 5]
    n.copy_(torch.tensor(lens, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    ref.check_attention(out, ref.attention(q, cache, table, lens, cu), "prefill")
    assert spin_gpu.device_status() == 0


def test_rows_behind_the_last_sequence_stay(spin_gpu):
    lens, nq = [100, 33], [2, 3]
    q, cache, table, cu = make(lens, nq, 8, 2, 32, seed=8)
    q2 = torch.cat([q[:1], q, q[:3]]).contiguous()
    out = torch.full((q2.shape[0], 8, 128), -7.0, dtype=torch.bfloat16, device="cuda")
    run(spin_gpu, q2, cache, table, lens, [1, 3, 6], out=out)
    assert (out[0] == -7).all() and (out[6:] == -7).all()
    assert torch.equal(out[1:6], run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16))


def test_matches_the_contiguous_decode(spin_gpu):
    """A contiguous cache is one page per row: the paged call on it, and on the same slots dealt
    out to pages, agrees with decode_attention_int4kv."""
    B, L, hq, hkv = 3, 512, 32, 8
    cache = ref.random_pages(B, hkv, L, 21)
    lens = torch.tensor([512, 100, 1], dtype=torch.int32, device="cuda")
    q = torch.randn((B, hq, 128), device="cuda").bfloat16()
    want = spin_gpu.decode_attention_int4kv(q, cache, lens)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    got = spin_gpu.paged_attention_int4kv(q, cache, table, lens)
    assert torch.allclose(got, want, rtol=1e-4, atol=1e-4)
    pages = {n: t.reshape(B, hkv, L // 64, 64, *t.shape[3:]).transpose(1, 2).reshape(-1, hkv, 64, *t.shape[3:]).contiguous()
             for n, t in cache.items()}
    table = torch.arange(B * L // 64, dtype=torch.int32, device="cuda").view(B, -1)
    got = spin_gpu.paged_attention_int4kv(q, pages, table, lens)
    assert torch.allclose(got, want, rtol=1e-4, atol=1e-4)


def test_repeats_bit_for_bit_and_ignores_the_workspace(spin_gpu):
    q, cache, table, cu = make([5000, 700], [1, 1], 8, 2, 64, seed=9)
    ws = torch.full((spin_gpu.paged_attention_workspace_bytes(8, 2, 1),), 255, dtype=torch.uint8, device="cuda")
    a = run(spin_gpu, q, cache, table, [5000, 700], cu, workspace=ws)
    for _ in range(3):
        assert torch.equal(a, run(spin_gpu, q, cache, table, [5000, 700], cu))


def test_streams_and_graphs(spin_gpu):
    """Another stream; a captured call replayed after lens and table changed; two graphs with
    workspaces of their own on two streams at once."""
    spin = spin_gpu
    q, cache, table, cu = make([6000, 3000], [1, 1], 8, 2, 64, seed=10)
    want = run(spin, q, cache, table, [6000, 3000], cu)
    short = run(spin, q, cache, table, [70, 1000], cu)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    lens = [torch.tensor([6000, 3000], dtype=torch.int32, device="cuda") for _ in range(2)]
    got = spin.paged_attention_int4kv(q, cache, table, lens[0], stream=s1)
    s1.synchronize()
    assert torch.equal(got, want)
    graphs, outs = [], []
    for s, n in zip((s1, s2), lens):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(spin.paged_attention_int4kv(q, cache, table, n))
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    lens[1].copy_(torch.tensor([70, 1000], dtype=torch.int32))
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], short) and torch.equal(outs[0], want)


def test_offsets_past_32_bits(spin_gpu):
    """Pages whose code bytes lie behind 4 GiB."""
    pages, hkv, page = 135000, 8, 64  # 4.4 GB of codes each
    cache = spin_gpu.alloc_kv_cache(pages, hkv, page)
    small = ref.random_pages(5, hkv, page, 31)
    where = torch.tensor([134999, 5, 131073, 134000, 70000], device="cuda")
    for n in cache:
        cache[n][where] = small[n]
    q = torch.randn((1, 32, 128), device="cuda").bfloat16()
    lens = torch.tensor([5 * page - 3], dtype=torch.int32, device="cuda")
    got = spin_gpu.paged_attention_int4kv(q, cache, where.int()[None].contiguous(), lens)
    want = spin_gpu.paged_attention_int4kv(q, small, torch.arange(5, dtype=torch.int32, device="cuda")[None].contiguous(),
                                           lens)
    assert torch.equal(got, want)
    # copies by page and by slot read and write there too
    free = torch.tensor([134998, 6, 131074, 134001, 70001], dtype=torch.int32, device="cuda")
    spin_gpu.copy_kv_pages(cache, where.int(), free)
    for n in cache:
        assert torch.equal(cache[n][free.long()], small[n])
    keep = torch.arange(5 * page, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5 * page], dtype=torch.int32, device="cuda")
    to = torch.tensor([134997, 7, 131075, 134002, 70002], dtype=torch.int32, device="cuda")
    spin_gpu.copy_kv_slots(cache, free[None].contiguous(), keep, cu, cache, to[None].contiguous())
    for n in cache:
        assert torch.equal(cache[n][to.long()], small[n])
