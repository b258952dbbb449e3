"""Rows of the page pool that were cut (their length lowered, as after rejected drafts): the pages
behind the new length stay the row's, are written on by the next growth and come back when the row
is let go. Against loops over rows."""
import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_kv_pages import Both, ints

pytestmark = pytest.mark.gpu


class Pool(ref.Pool):
    """The pool's rules with rows that may have been cut: the columns behind a row's length hold pages
    of its own up to the first that names none."""

    def holders(self, page):
        return self.refs[page] if 0 <= page < self.pages else 0

    def reserve(self, add):
        status, free, asked = [], len(self.stack), 0
        cols = len(self.table[0])
        for b, n in enumerate(add):
            length, row = self.lens[b], self.table[b]
            if n < 0 or length < 0 or length > cols * self.page or -(-(length + n) // self.page) > cols:
                status.append(2)
                continue
            have, total = -(-length // self.page), -(-(length + n) // self.page)
            shared = n > 0 and length % self.page and self.holders(row[have - 1]) > 1
            while length > 0 and have < total and self.holders(row[have]) == 1:
                have += 1
            if shared or (length > 0 and have < total and self.holders(row[have]) > 1):
                status.append(2)
                continue
            asked += total - have
            if total > have and asked > free:
                status.append(1)
                continue
            if total > have and total < cols:
                row[total] = -1
            for j in range(have, total):
                row[j] = self.stack.pop()
                self.refs[row[j]] = 1
            self.lens[b] = length + n
            status.append(0)
        return status

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.table) and self.lens[r] > 0:  # its kept pages count as held
                j = -(-self.lens[r] // self.page)
                while j < len(self.table[r]) and 0 <= self.table[r][j] < self.pages:
                    j += 1
                self.lens[r] = j * self.page
        super().free(rows)


class Cut(Both):
    def __init__(self, spin, pages, hkv, page, rows, cols, fill=-1):
        super().__init__(spin, pages, hkv, page, rows, cols)
        self.table.fill_(fill)
        m = self.model
        self.model = Pool(m.pages, m.page, self.table.tolist(), m.lens, m.refs, m.stack)

    def cut(self, lens):
        for b, n in lens.items():
            self.lens[b] = n
            self.model.lens[b] = n

    def everything_back(self):
        assert self.pool["free_count"].item() == self.model.pages and (self.pool["refs"] == 0).all()
        assert sorted(self.model.stack) == list(range(self.model.pages))


def test_rejected_drafts_lose_no_page(spin_gpu):
    b = Cut(spin_gpu, pages=6, hkv=1, page=16, rows=1, cols=6)
    b.reserve([30])
    for _ in range(3):
        b.reserve([4])
        b.cut({0: 31})
    b.reserve([4])
    assert b.pool["free_count"].item() == 3
    b.free([0])
    b.everything_back()


def test_cut_rows_grow_over_what_they_kept(spin_gpu):
    """Part of the kept columns, exactly them, more than them; a row that wants new pages after one
    that does not; a row let go while it is cut."""
    b = Cut(spin_gpu, pages=64, hkv=2, page=16, rows=6, cols=40)
    b.reserve([200, 200, 200, 200, 33, 16])
    b.cut({0: 100, 1: 97, 2: 17, 3: 16, 4: 1})
    b.reserve([30, 103, 300, 0, 0, 1])
    b.cut({2: 16, 1: 32})
    b.reserve([1, 17, 16 * 39, 1, 1, 600])  # the last finds too few pages and is left as it was
    b.cut({0: 5, 1: 5})
    b.free([0, 5])
    b.reserve([700, 64, 0, 40, 40, 1])
    b.free(list(range(6)))
    b.everything_back()


def test_forked_rows_that_were_cut(spin_gpu):
    """A child's own tail page, and a parent's kept pages, which the child does not get."""
    b = Cut(spin_gpu, pages=30, hkv=1, page=16, rows=4, cols=12)
    b.reserve([100, 0, 0, 0])
    b.cut({0: 40})
    b.fork([0, 0], [1, 2])
    b.reserve([30, 30, 5, 0])
    b.cut({1: 41})
    b.reserve([0, 9, 90, 0])
    b.free([0])
    b.free([1, 2])
    b.everything_back()


@pytest.mark.parametrize("fill", [0, 3, 10 ** 6])
def test_a_new_table_may_hold_anything(spin_gpu, fill):
    """Rows that grew from empty take nothing from what the table held before."""
    b = Cut(spin_gpu, pages=50, hkv=1, page=16, rows=5, cols=12, fill=fill)
    b.reserve([1, 70, 0, 192, 16])
    b.reserve([40, 1, 3, 0, 16])
    b.cut({1: 20})
    b.reserve([16, 52, 16, 0, 100])
    b.free([0, 1, 2, 3, 4])
    b.everything_back()


def test_many_cut_rows(spin_gpu):
    """More rows than threads of the planning block, long ones among them."""
    rows, page = 1500, 16
    b = Cut(spin_gpu, pages=21000, hkv=1, page=page, rows=rows, cols=40)
    g = torch.Generator().manual_seed(2)
    draw = lambda lo, hi: torch.randint(lo, hi, (rows,), generator=g).tolist()  # noqa: E731
    b.reserve(draw(0, 13 * page))
    for most in (6, 300):
        b.cut({i: max(1, n - k) if n else 0 for i, (n, k) in enumerate(zip(b.model.lens, draw(0, 150)))})
        b.reserve(draw(0, most))
    b.free(torch.randperm(rows, generator=g).tolist())
    b.everything_back()


def test_captured_draft_steps(spin_gpu):
    """Grow by four drafted tokens, keep one: captured, replayed over many pages."""
    spin = spin_gpu
    pool = spin.alloc_kv_pages(12, 1, 16)
    table = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
    lens = ints([0, 0])
    spin.reserve_kv_pages(pool, table, lens, ints([5, 30]))
    add = ints([4, 4])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st = spin.reserve_kv_pages(pool, table, lens, add)
        lens -= 3
    for i in range(50):
        g.replay()
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0] and lens.tolist() == [55, 80]
    held = [set(x for x in row if x >= 0) for row in table.tolist()]
    assert len(held[0]) == 4 and len(held[1]) == 6 and not held[0] & held[1]
    assert pool["free_count"].item() == 2
    spin.free_kv_pages(pool, table, lens, ints([0, 1]))
    assert pool["free_count"].item() == 12 and (pool["refs"] == 0).all()


@pytest.mark.parametrize("far", [0, 200])
def test_no_row_grows_onto_a_shared_page(spin_gpu, far):
    """Forked rows cut into the pages they share: refused while others hold these, at a page's end and
    inside it, for a few slots and for many (`far`); served once the row alone holds them."""
    b = Cut(spin_gpu, pages=60, hkv=1, page=16, rows=4, cols=20)
    b.reserve([100, 0, 0, 40])
    b.fork([0, 0], [1, 2])
    b.cut({0: 32, 1: 33, 2: 95})
    b.reserve([far + 1, 0, 0, 0])            # the next column names a shared page
    b.reserve([0, far + 15, far + 1, 4])     # the last page is shared
    b.reserve([0, 0, 0, 0])                  # nothing wanted, nothing refused
    assert b.lens.tolist() == [32, 33, 95, 44]
    b.free([0])
    b.reserve([5, far + 1, 0, 0])            # still shared by the two children
    b.free([1])
    b.reserve([0, 7, far + 2, 0])
    assert b.lens.tolist() == [5, 7, 97 + far, 44]
    b.cut({2: 20})
    b.reserve([0, 0, far + 60, 0])
    b.free([0, 1, 2, 3])
    b.everything_back()
