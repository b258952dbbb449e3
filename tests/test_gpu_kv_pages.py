"""The paged INT4 KV cache's copies and the pool's reserve, fork and free against loops over
rows; and a serving run that uses them all together with R3 and the attention."""
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(a, b, where=None):
    for n in ref.CODES + ref.STEPS:
        x, y = (a[n], b[n]) if where is None else (a[n][where], b[n][where])
        assert torch.equal(x.view(torch.uint8) if x.dtype == torch.uint8 else x.view(torch.int16),
                           y.view(torch.uint8) if y.dtype == torch.uint8 else y.view(torch.int16)), n


@pytest.mark.parametrize("hkv,page,n", [(8, 16, 1), (8, 64, 37), (1, 16, 300), (3, 5, 11), (1, 1, 9), (2, 128, 64)])
def test_copy_pages(spin_gpu, hkv, page, n):
    cache = ref.random_pages(2 * n + 3, hkv, page, seed=n)
    want = {k: t.clone() for k, t in cache.items()}
    perm = torch.randperm(2 * n + 3, generator=torch.Generator().manual_seed(n)).cuda()
    src, dst = perm[:n].int().contiguous(), perm[n:2 * n].int().contiguous()
    for k in want:
        want[k][dst.long()] = want[k][src.long()]
    spin_gpu.copy_kv_pages(cache, src, dst)
    same(cache, want)


def test_copy_pages_between_caches_repeats_and_skips(spin_gpu):
    a, b = ref.random_pages(6, 2, 32, 1), ref.random_pages(4, 2, 32, 2)
    want = {k: t.clone() for k, t in b.items()}
    src, dst = [5, 5, 0, -1, 6, 3, 2], [0, 2, 3, 1, 1, 4, -9]
    for k in want:
        want[k][torch.tensor([0, 2, 3], device="cuda")] = a[k][torch.tensor([5, 5, 0], device="cuda")]
    spin_gpu.copy_kv_pages(a, ints(src), ints(dst), b)
    same(b, want)
    spin_gpu.copy_kv_pages(a, ints([]), ints([]), b)
    same(b, want)


@pytest.mark.parametrize("hkv,page,dst_page,rows,longest", [(8, 16, 64, 5, 40), (2, 64, 16, 3, 700), (1, 7, 5, 4, 60),
                                                           (8, 64, 64, 1, 5000), (3, 16, 32, 200, 9), (64, 16, 16, 2, 3)])
def test_copy_slots(spin_gpu, hkv, page, dst_page, rows, longest):
    g = torch.Generator().manual_seed(rows + longest)
    lens = torch.randint(0, longest + 1, (rows,), generator=g).tolist()
    kept = [sorted(torch.randperm(n, generator=g)[:n - n // 3].tolist()) for n in lens]
    start = torch.randint(0, 4, (rows,), generator=g).tolist()
    cols, dcols = -(-longest // page) + 1, -(-(longest + 4) // dst_page)
    src, dst = ref.random_pages(rows * cols, hkv, page, 3), ref.random_pages(rows * dcols, hkv, dst_page, 4)
    st = torch.randperm(rows * cols, generator=g).view(rows, cols)
    dt = torch.randperm(rows * dcols, generator=g).view(rows, dcols)
    want = {k: t.clone() for k, t in dst.items()}
    cu = [0]
    for k in kept:
        cu.append(cu[-1] + len(k))
    r = torch.tensor([b for b, k in enumerate(kept) for _ in k], dtype=torch.long)
    s = torch.tensor([x for k in kept for x in k], dtype=torch.long)
    d = torch.tensor([start[b] + i for b, k in enumerate(kept) for i in range(len(k))], dtype=torch.long)
    for k in want:
        want[k][dt[r, d // dst_page].cuda(), :, (d % dst_page).cuda()] = \
            src[k][st[r, s // page].cuda(), :, (s % page).cuda()]
    spin_gpu.copy_kv_slots(src, st.int().cuda(), s.int().cuda(), ints(cu), dst, dt.int().cuda(), ints(start))
    same(dst, want)


def test_copy_slots_skips_what_is_not_there(spin_gpu):
    """Negative and far slots, missing pages on either side, entries outside the rows, start
    offsets out of the table; everything else stays."""
    src, dst = ref.random_pages(4, 2, 16, 5), ref.random_pages(3, 2, 16, 6)
    want = {k: t.clone() for k, t in dst.items()}
    st, dt = ints([[0, 1], [2, -1]]), ints([[0, 9], [1, 2]])
    keep = ints([99, 3, -1, 32, 17, 5, 20, 6, 7, 0])
    cu = ints([1, 5, 9])  # entry 0 and entry 9 belong to no row
    # row 0: slots 3, -1, 32, 17 -> 14, 15, 16 (page 9: none), 17; row 1: 5, 20 (page -1), 6, 7 -> -2 .. 1
    for k in want:
        want[k][0, :, 14] = src[k][0, :, 3]
        want[k][1, :, 0], want[k][1, :, 1] = src[k][2, :, 6], src[k][2, :, 7]
    spin_gpu.copy_kv_slots(src, st, keep, cu, dst, dt, ints([14, -2]))
    same(dst, want)
    spin_gpu.copy_kv_slots(src, st, keep, ints([9, 9, 9]), dst, dt)
    spin_gpu.copy_kv_slots(src, st, ints([]), ints([0, 0, 0]), dst, dt)
    same(dst, want)


class Both:
    """A pool on the GPU and its model, kept side by side."""

    def __init__(self, spin, pages, hkv, page, rows, cols):
        self.spin = spin
        self.pool = spin.alloc_kv_pages(pages, hkv, page)
        data = ref.random_pages(pages, hkv, page, seed=pages)
        for n in data:
            self.pool[n].copy_(data[n])
        self.table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.model = ref.Pool(pages, page, self.table.tolist(), [0] * rows, [0] * pages,
                              list(range(pages - 1, -1, -1)))

    def check(self):
        m, n = self.model, len(self.model.stack)
        assert self.lens.tolist() == m.lens
        assert self.table.tolist() == m.table
        assert self.pool["refs"].tolist() == m.refs
        assert self.pool["free_count"].tolist() == [n]
        assert self.pool["free_pages"].tolist()[:n] == m.stack

    def reserve(self, add):
        st = self.spin.reserve_kv_pages(self.pool, self.table, self.lens, ints(add))
        assert st.tolist() == self.model.reserve(add)
        self.check()

    def fork(self, parents, children):
        before = {n: self.pool[n].clone() for n in ref.CODES + ref.STEPS}
        st = self.spin.fork_kv_pages(self.pool, self.table, self.lens, ints(parents), ints(children))
        want, copies = self.model.fork(parents, children)
        assert st.tolist() == want
        self.check()
        for s, d, tail in copies:
            for n in before:
                before[n][d, :, :tail] = before[n][s, :, :tail]
        same(self.pool, before)

    def free(self, rows):
        self.spin.free_kv_pages(self.pool, self.table, self.lens, ints(rows))
        self.model.free(rows)
        self.check()


def test_pool_life(spin_gpu):
    b = Both(spin_gpu, pages=40, hkv=2, page=16, rows=8, cols=6)
    b.reserve([0, 1, 16, 17, 40, 0, 0, 0])
    b.fork([4, 4, 2, 3], [5, 6, 7, 0])  # shared full pages, a whole last page, a tail
    b.reserve([1] * 8)
    b.free([4, 4, 1])                   # listed twice; row 4's pages live on in its children
    b.fork([5], [4])
    b.free([5, 6, 4, 7])
    b.free([0, 2, 3, 1, -1, 99])        # an empty row and rows that are none
    assert sorted(b.model.stack) == list(range(40))


def test_pool_refusals(spin_gpu):
    b = Both(spin_gpu, pages=6, hkv=1, page=16, rows=6, cols=4)
    b.reserve([16, 65, -1, 2 ** 31 - 1, 64, 5])  # too long for the table, negative, overflow, fits
    b.reserve([17, 0, 0, 0, 0, 1])               # one page left, two wanted: the last row wants none
    b.reserve([0, 16, 16, 16, 0, 0])             # none left
    b.fork([0, 9, 5, 5, 5, 4], [1, 2, -1, 0, 5, 1])  # bad rows, full child, itself, a taken child
    b.fork([5, 5], [2, 3])                       # no page for the tail
    b.lens[3] = -5
    b.model.lens[3] = -5
    b.reserve([0] * 6)
    b.fork([3, 5], [2, 3])
    b.free([3])


def test_fork_reads_parents_as_they_were(spin_gpu):
    """A child of one fork that is the parent of the next; two forks into one row."""
    b = Both(spin_gpu, pages=30, hkv=2, page=16, rows=6, cols=4)
    b.reserve([20, 0, 0, 0, 0, 33])
    b.fork([0, 1, 5, 0], [1, 2, 3, 3])
    b.fork([2], [4])  # an empty parent
    b.free([1, 3])


@pytest.mark.parametrize("rows,page", [(1500, 16), (3000, 64)])
def test_pool_many_rows(spin_gpu, rows, page):
    """More rows and forks than threads of the planning block, and a pool of several turns."""
    b = Both(spin_gpu, pages=21000, hkv=1, page=page, rows=2 * rows, cols=12)
    g = torch.Generator().manual_seed(rows)
    add = torch.randint(0, 12 * page + 3, (2 * rows,), generator=g)
    add[rows:] = 0
    b.reserve(add.tolist())
    parents = torch.randint(0, rows, (rows,), generator=g).tolist()
    children = (rows + torch.randperm(rows, generator=g)).tolist()
    b.fork(parents, children)
    b.free(torch.randint(0, 2 * rows, (rows,), generator=g).tolist())
    b.reserve(torch.randint(0, 4, (2 * rows,), generator=g).tolist())
    b.free(list(range(2 * rows)))
    assert sorted(b.model.stack) == list(range(21000))


def test_one_row_takes_many_pages(spin_gpu):
    b = Both(spin_gpu, pages=5000, hkv=1, page=16, rows=2, cols=4096)
    b.reserve([4000 * 16 + 1, 5])
    b.fork([0], [1])   # refused: the row is not empty
    b.free([1])
    b.fork([0], [1])
    b.free([0, 1])


def test_serving_run(spin_gpu):
    """Prompts through R3 into a small contiguous cache, moved to pages; steps of one token;
    a fork that goes its own way; drafted tokens of which some are kept; rows let go. The paged
    attention is compared at each point with the same slots read by its binary64 form."""
    spin = spin_gpu
    hq, hkv, page, rows, cols = 8, 2, 16, 4, 8
    pool = spin.alloc_kv_pages(40, hkv, page)
    table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)

    def step(counts):
        """New tokens for every row: queries in token order, their keys and values in pages."""
        most = max(counts)
        x = lambda h: torch.randn((rows, most, h, 128), generator=g, device="cuda").bfloat16()  # noqa: E731
        q, k, v = x(hq), x(hkv), x(hkv)
        start = lens.clone()
        assert spin.reserve_kv_pages(pool, table, lens, ints(counts)).tolist() == [0] * rows
        pos = (start[:, None] + torch.arange(most, device="cuda")).int().contiguous()
        fresh = spin.alloc_kv_cache(rows, hkv, most)
        rotated = spin.rope_hadamard_kvquant(q, k, v, pos, fresh, clip=0.95)
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        keep = ints([j for n in counts for j in range(n)])
        spin.copy_kv_slots(fresh, torch.arange(rows, dtype=torch.int32, device="cuda")[:, None].contiguous(), keep,
                           ints(cu), pool, table, start)
        q = torch.cat([rotated[b, :n] for b, n in enumerate(counts)]).contiguous()
        out = spin.paged_attention_int4kv(q, pool, table, lens, ints(cu), most)
        ref.check_attention(out, ref.attention(q, pool, table, lens.tolist(), cu))
        return out

    step([33, 16, 0, 7])                 # prompts
    for _ in range(3):
        step([1, 1, 0, 1])               # decode
    assert spin.fork_kv_pages(pool, table, lens, ints([0]), ints([2])).tolist() == [0]
    shared = table[0, :2].tolist()
    assert table[2, :2].tolist() == shared and pool["refs"][torch.tensor(shared)].tolist() == [2, 2]
    step([1, 1, 1, 1])                   # both branches write on
    assert (table[0, 2] != table[2, 2]).item()
    step([4, 4, 4, 4])                   # drafted tokens; of row 1 the first and third are kept
    fresh_rows = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
    fresh_lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    n = int(lens[1])
    kept = list(range(n - 4)) + [n - 4, n - 2]
    spin.reserve_kv_pages(pool, fresh_rows, fresh_lens, ints([0, len(kept), 0, 0]))
    before = ref.attention(torch.ones((1, hq, 128), device="cuda"), pool, table[1:2], [n - 3], [0, 1])[0]
    spin.copy_kv_slots(pool, table, ints(kept), ints([0, 0, len(kept), len(kept), len(kept)]), pool, fresh_rows)
    after = ref.attention(torch.ones((1, hq, 128), device="cuda"), pool, fresh_rows[1:2], [n - 3], [0, 1])[0]
    assert torch.equal(before, after)
    spin.free_kv_pages(pool, table, lens, ints([1]))
    table[1], lens[1] = fresh_rows[1], fresh_lens[1]
    step([1, 1, 1, 1])
    spin.free_kv_pages(pool, table, lens, ints([0, 1, 2, 3]))
    assert pool["free_count"].item() == 40 and (pool["refs"] == 0).all()
    assert sorted(pool["free_pages"].tolist()) == list(range(40))


def test_pool_calls_captured_and_replayed(spin_gpu):
    """A captured step (reserve, fork, free) replayed: the pool comes back to where it was."""
    spin = spin_gpu
    pool = spin.alloc_kv_pages(16, 1, 16)
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    add, rows, parent, child = ints([20, 0, 40]), ints([0, 1, 2]), ints([2]), ints([1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st = spin.reserve_kv_pages(pool, table, lens, add)
        spin.fork_kv_pages(pool, table, lens, parent, child)
        spin.free_kv_pages(pool, table, lens, rows)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert st.tolist() == [0, 0, 0] and lens.tolist() == [0, 0, 0]
        assert pool["free_count"].item() == 16 and sorted(pool["free_pages"].tolist()) == list(range(16))


def test_copies_and_pool_calls_on_another_stream(spin_gpu):
    """A stream argument, and the current stream where there is none: each call sees what was enqueued before it."""
    spin = spin_gpu
    for given in (True, False):
        s = torch.cuda.Stream()
        kw = dict(stream=s) if given else {}
        cache, big = ref.random_pages(12, 2, 16, 5), torch.zeros(1 << 26, device="cuda")
        pool = spin.alloc_kv_pages(8, 2, 16)
        table, lens, add = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), ints([0, 0]), ints([0, 0])
        src, dst = ints([0, 0]), ints([5, 7])
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(20):
                big.add_(1)  # what is read below is written well after the calls were made
            src.copy_(ints([3, 1]))
            add.copy_(ints([20, 33]))
        if given:
            st = spin.reserve_kv_pages(pool, table, lens, add, **kw)
            spin.copy_kv_pages(cache, src, dst, **kw)
        else:
            with torch.cuda.stream(s):
                st = spin.reserve_kv_pages(pool, table, lens, add)
                spin.copy_kv_pages(cache, src, dst)
        s.synchronize()
        assert st.tolist() == [0, 0] and lens.tolist() == [20, 33] and pool["free_count"].item() == 3
        for name, t in cache.items():
            assert torch.equal(t[5], t[3]) and torch.equal(t[7], t[1]), name
