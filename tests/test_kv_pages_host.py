"""Argument rules of the paged INT4 KV cache's entry points that need no GPU: every rejected
call and every empty one returns before any device access, and the binding refuses host
tensors, wrong types and shapes."""
import pytest
import torch

import online_hadamard_rotation_b200 as spin

FAKE = 0x10000  # 16-byte aligned, never dereferenced
OK, BAD, SIZE, MIS = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from online_hadamard_rotation_b200 import build
    build.build()
    return spin.lib()


def pages(**kw):
    a = dict(k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, k_zero=FAKE, v_scale=FAKE, v_zero=FAKE, pages=10, n_kv_heads=8,
             page_size=16, head_dim=128)
    a.update(kw)
    return spin._pack_pages(*(a[n] or 0 for n, _ in spin._KV_ARRAYS), a["pages"], a["n_kv_heads"], a["page_size"],
                            a["head_dim"])


def pool(**kw):
    a = dict(refs=FAKE, free_pages=FAKE, free_count=FAKE)
    a.update(kw)
    return spin._pack_pool(*(a[n] or 0 for n in ("refs", "free_pages", "free_count")))


def attn(L, cache=None, **kw):
    a = dict(q=FAKE, tokens=4, table=FAKE, seqs=2, cols=800, lens=FAKE, cu=FAKE, most=2, hq=32, scale=0.088, window=0,
             sinks=0, out=FAKE, dtype=1, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return L.spin_paged_attention_int4kv(a["q"], a["tokens"], cache or pages(), a["table"], a["seqs"], a["cols"],
                                         a["lens"], a["cu"], a["most"], a["hq"], a["scale"], a["window"], a["sinks"],
                                         a["out"], a["dtype"], a["ws"], a["bytes"], None)


def test_attention_rules(L):
    none = dict(q=None, table=None, lens=None, cu=None, out=None, ws=None, bytes=0)
    assert attn(L, **dict(none, tokens=0, seqs=0)) == OK
    assert attn(L, tokens=0) == OK and attn(L, seqs=0) == OK
    assert attn(L, seqs=0, cu=None, tokens=4) == BAD  # without offsets every sequence has one token
    for kw in (dict(tokens=-1), dict(seqs=-1), dict(cols=0), dict(most=0), dict(hq=0), dict(hq=30), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(sinks=-1), dict(dtype=2),
               dict(cu=None), dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(ws=None),
               dict(bytes=1000)):
        assert attn(L, **kw) == BAD, kw
    for kw in (dict(page_size=8), dict(page_size=48), dict(page_size=1 << 17), dict(head_dim=64),
               dict(n_kv_heads=1 << 21)):
        assert attn(L, pages(**kw), hq=1 << 21 if "n_kv_heads" in kw else 32) == SIZE, kw
    assert attn(L, tokens=1 << 27) == SIZE  # tokens x heads
    assert attn(L, pages(n_kv_heads=0)) == BAD and attn(L, pages(pages=-1)) == BAD
    assert attn(L, pages(k_cache=None)) == BAD and attn(L, pages(v_zero=None)) == BAD
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 4), dict(ws=FAKE + 8), dict(table=FAKE + 2), dict(lens=FAKE + 1),
               dict(cu=FAKE + 2)):
        assert attn(L, **kw) == MIS, kw
    assert attn(L, pages(k_scale=FAKE + 2)) == MIS and attn(L, pages(v_cache=FAKE + 8)) == MIS


def test_limits_of_counts(L):
    """What a kernel's grid and int counters cannot hold is refused before the device is asked."""
    big, most = 1 << 30, (1 << 31) - 1
    small = pages(n_kv_heads=8, page_size=64)  # 2^31 - 1 pairs: 2^40 slot rows of 8.5 pieces, 2048 pieces a block
    assert L.spin_kv_pages_copy(small, FAKE, small, FAKE, most, None) == SIZE
    assert L.spin_kv_pages_copy(small, FAKE, small, FAKE, (1 << 29) + 1, None) == SIZE
    assert attn(L, seqs=big + 1) == SIZE and attn(L, seqs=most) == SIZE
    assert L.spin_kv_slots_copy(pages(), FAKE, 4, FAKE, FAKE, 9, big + 1, pages(), FAKE, 4, None, None) == SIZE
    for rows, n in ((big + 1, 3), (4, big + 1), (most, most)):
        assert L.spin_kv_pages_fork(pages(), pool(), FAKE, rows, 8, FAKE, FAKE, FAKE, n, FAKE, None) == SIZE
        assert L.spin_kv_pages_free(pages(), pool(), FAKE, rows, 8, FAKE, FAKE, n, None) == SIZE
    assert L.spin_kv_pages_reserve(pages(), pool(), FAKE, big + 1, 8, FAKE, FAKE, FAKE, None) == SIZE


def test_workspace_bytes(L):
    f = L.spin_paged_attention_workspace_bytes
    n = 1 << 40
    assert f(32, 8, 1, n) > 0 and f(32, 8, 1, n) % 16 == 0 and f(32, 8, 1, 4096) == f(32, 8, 1, n)
    assert f(32, 8, 1, n) <= f(32, 8, 4, n) <= f(32, 8, 100, n) == f(32, 8, 1 << 30, n)
    assert f(0, 8, 1, n) == f(32, 0, 1, n) == f(32, 8, 0, n) == f(30, 8, 1, n) == f(-32, -8, 1, n) == f(32, 8, 1, 0) == 0
    assert f(32, 8, 1, 64) == 0  # a short row is never cut


def test_copy_rules(L):
    f = L.spin_kv_pages_copy
    assert f(pages(), FAKE, pages(), FAKE, 0, None) == OK
    assert f(pages(k_cache=None), None, pages(), None, 0, None) == OK  # nothing to copy
    assert f(pages(), FAKE, pages(), FAKE, -1, None) == BAD
    assert f(pages(), None, pages(), FAKE, 3, None) == BAD and f(None, FAKE, pages(), FAKE, 3, None) == BAD
    assert f(pages(), FAKE, pages(page_size=32), FAKE, 3, None) == SIZE
    assert f(pages(), FAKE, pages(n_kv_heads=4), FAKE, 3, None) == SIZE
    assert f(pages(head_dim=256), FAKE, pages(head_dim=256), FAKE, 3, None) == SIZE
    assert f(pages(), FAKE + 2, pages(), FAKE, 3, None) == MIS
    assert f(pages(n_kv_heads=1024, page_size=16384), FAKE, pages(n_kv_heads=1024, page_size=16384), FAKE, 1 << 20,
             None) == SIZE
    g = L.spin_kv_slots_copy
    ok = [pages(), FAKE, 4, FAKE, FAKE, 9, 2, pages(page_size=5), FAKE, 4, None, None]
    put = lambda i, v: ok[:i] + [v] + ok[i + 1:]  # noqa: E731
    assert g(*put(5, 0)) == OK and g(*put(6, 0)) == OK
    for i, v in ((5, -1), (6, -1), (2, 0), (9, 0), (1, None), (3, None), (4, None), (8, None), (0, None)):
        assert g(*put(i, v)) == BAD, (i, v)
    assert g(*put(7, pages(n_kv_heads=2))) == SIZE
    for i in (1, 3, 4, 8, 10):
        assert g(*put(i, FAKE + 2)) == MIS, i


def test_pool_rules(L):
    for f, ok, n in ((L.spin_kv_pages_reserve, [pages(), pool(), FAKE, 4, 8, FAKE, FAKE, FAKE, None], 3),
                     (L.spin_kv_pages_fork, [pages(), pool(), FAKE, 4, 8, FAKE, FAKE, FAKE, 3, FAKE, None], 8),
                     (L.spin_kv_pages_free, [pages(), pool(), FAKE, 4, 8, FAKE, FAKE, 3, None], 7)):
        put = lambda i, v: ok[:i] + [v] + ok[i + 1:]  # noqa: B023,E731
        assert f(*put(n, 0)) == OK and f(*put(n, -1)) == BAD
        assert f(*put(4, 0)) == BAD and f(*put(3, -1)) == BAD
        for i in (0, 1, 2, 5, 6):
            assert f(*put(i, None)) == BAD, (f, i)
        for i in (2, 5, 6):
            assert f(*put(i, FAKE + 2)) == MIS, (f, i)
        assert f(*put(1, pool(refs=None))) == BAD and f(*put(1, pool(free_count=FAKE + 1))) == MIS
        assert f(*put(0, pages(head_dim=64))) == SIZE


def test_binding_refuses(L):
    cache = dict(k_cache=torch.zeros((2, 1, 16, 64), dtype=torch.uint8), v_cache=torch.zeros((2, 1, 16, 64), dtype=torch.uint8),
                 **{n: torch.zeros((2, 1, 16), dtype=torch.float16) for n in ("k_scale", "k_zero", "v_scale", "v_zero")})
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        spin.paged_attention_int4kv(torch.zeros((1, 4, 128), dtype=torch.bfloat16), cache, i[None], i)
    with pytest.raises(ValueError, match="CUDA"):
        spin.copy_kv_pages(cache, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        spin.free_kv_pages(cache, i[None], i, i)
    with pytest.raises(ValueError, match="k_cache"):
        spin.copy_kv_pages(dict(cache, k_cache=cache["k_cache"][0]), i, i)


def test_declared_and_exported(L):
    for name in ("spin_paged_attention_int4kv", "spin_paged_attention_workspace_bytes", "spin_kv_pages_copy",
                 "spin_kv_slots_copy", "spin_kv_pages_reserve", "spin_kv_pages_fork", "spin_kv_pages_free"):
        assert name in spin.exported_symbols() and getattr(L, name) is not None
    assert len(pages()) == 64 and len(pool()) == 24  # the C structs' sizes
