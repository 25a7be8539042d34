"""The paged-cache entry points on the host: workspace sizes, argument checks before any CUDA
call, and the oracle's own hand cases.  No compute call is made here (CPU only)."""

import numpy as np
import pytest

import oracle.paged_oracle as po


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from long_context_block_b200 import _binding
    return _binding


def test_workspace_sizes(lib):
    c = lib.library()
    a256 = lambda x: (x + 255) // 256 * 256
    # nseq, T, Hq, Hkv, d, page_size, max_pages, topk.  Partials: two row blocks per CTA (296 at
    # most), of 16 rows, or 32 when more share a head
    att = lambda rb, d, ctas=296: (a256(2 * ctas * rb * d * 4) + a256(2 * ctas * rb * 8)
                                   + a256(ctas * 8))
    f = c.misa_paged_attention_workspace_size
    assert f(32, 1, 32, 8, 128, 64, 512, 0) == att(16, 128)
    assert f(32, 1, 32, 8, 64, 64, 512, 0) == att(16, 64)
    assert f(8, 4, 32, 8, 128, 64, 512, 0) == att(16, 128)
    assert f(8, 6, 32, 8, 128, 64, 512, 0) == att(32, 128)
    # more than 32 rows: the tensor-core form, 148 CTAs of 128 rows
    assert f(8, 16, 32, 8, 128, 64, 512, 0) == att(128, 128, 148)
    assert f(8, 16, 32, 8, 128, 64, 512, 2048) == att(16, 128)   # each query its own tokens
    assert f(1, 1, 16, 2, 128, 16, 50, 0) == 0                   # a cluster per item: no partials
    for bad in ((0, 1, 32, 8, 128, 64, 512, 0), (1, 0, 32, 8, 128, 64, 512, 0),
                (1, 1, 30, 8, 128, 64, 512, 0), (1, 1, 32, 0, 128, 64, 512, 0),
                (1, 1, 32, 8, 96, 64, 512, 0), (1, 1, 32, 8, 128, 64, 512, -1),
                (1, 1, 32, 8, 128, 0, 512, 0), (1, 1, 32, 8, 128, 64, 0, 0),
                (1 << 20, 1 << 12, 32, 8, 128, 64, 512, 0)):
        assert f(*bad) == 0, bad
    g = c.misa_pages_workspace_size
    for op in (7, 9):                        # resize, compact
        assert g(op, 4, 8, 1000) == a256(32) + 3 * a256(4000) + 3 * a256(16)
    assert g(8, 100, 300, 10) == 0           # fork: a table that one cluster holds
    assert g(8, 100, 1000, 10) == a256(100 * 1000 * 4)
    for op in (7, 8, 9):
        for bad in ((0, 8, 10), (4, 0, 10), (4, 8, 0), (4, 8, (1 << 30) + 1), (1 << 16, 1 << 15, 9)):
            assert g(op, *bad) == 0, bad
    assert g(6, 4, 8, 1000) == 0


def _attention(c, dtype=0, nseq=2, T=1, Hq=8, Hkv=2, d=128, num_pages=16, page_size=16,
               max_pages=4, topk=0, scale=0.1):
    return c.misa_paged_attention(None, None, None, None, None, None, dtype, nseq, T, Hq, Hkv, d,
                                  num_pages, page_size, max_pages, topk, scale, None, None, None,
                                  None, 0, None)


@pytest.mark.parametrize("kw, status", [
    ({}, 1),                                   # null pointers
    (dict(d=96), 2), (dict(d=0), 1), (dict(dtype=2), 1), (dict(dtype=-1), 1),
    (dict(Hq=7), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(T=0), 1), (dict(nseq=0), 1),
    (dict(topk=-1), 1), (dict(topk=16), 1),    # a count without a list
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(page_size=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1),
    (dict(max_pages=1 << 20, page_size=2048), 2), (dict(num_pages=1 << 20, page_size=2048), 2),
    (dict(nseq=1 << 20, T=1 << 12), 2), (dict(nseq=1 << 16, T=1 << 12, Hq=64), 2),
])
def test_attention_refusals(lib, kw, status):
    assert _attention(lib.library(), **kw) == status


@pytest.mark.parametrize("kw, status", [
    ({}, 1), (dict(d=32), 2), (dict(dtype=5), 1), (dict(Hkv=0), 1), (dict(T=0), 1),
    (dict(page_size=0), 1), (dict(max_pages=1 << 20, page_size=2048), 2),
])
def test_append_refusals(lib, kw, status):
    a = dict(dtype=0, nseq=2, T=3, Hkv=2, d=64, num_pages=8, page_size=16, max_pages=4)
    a.update(kw)
    assert lib.library().misa_paged_append(None, None, None, None, *a.values(), None, None, None,
                                           None) == status


def test_wait_probe_refusals(lib):
    f = lib.library().misa_testing_paged_attention_wait_expiry
    for wait, skip in ((10, -1), (5_000_000_000, -1), (100000, -2), (100000, 0)):
        assert f(None, None, None, None, None, None, 0, 2, 1, 8, 2, 128, 16, 16, 4, 0, 0.1, None,
                 None, None, None, 0, wait, skip, None) == 1


def test_upkeep_refusals(lib):
    c = lib.library()
    big = (1 << 30) + 1
    # null pointers, sizes below 1, too many pages, a too long table row
    assert c.misa_pages_resize(None, None, None, None, 2, 4, 8, 16, None, None, 0, None, None,
                               None, None, 0, None) == 1
    assert c.misa_pages_resize(None, None, None, None, 2, 4, 8, 0, None, None, 0, None, None,
                               None, None, 0, None) == 1
    assert c.misa_pages_resize(None, None, None, None, 2, 1 << 20, 8, 2048, None, None, 0, None,
                               None, None, None, 0, None) == 2
    assert c.misa_pages_fork(None, None, None, 2, 4, 8, None, None, None, None, 0, None) == 1
    assert c.misa_pages_fork(None, None, None, 0, 4, 8, None, None, None, None, 0, None) == 1
    assert c.misa_pages_fork(None, None, None, 2, 4, big, None, None, None, None, 0, None) == 2
    assert c.misa_pages_compact(None, None, 2, 4, 8, None, None, 0, None, None, None, None, None,
                                0, None) == 1
    assert c.misa_pages_compact(None, None, 2, 4, big, None, None, 0, None, None, None, None,
                                None, 0, None) == 2
    assert c.misa_status_string(8) == b"not enough free pages"


def test_cpu_tensors_are_refused(lib):
    import torch
    z = torch.zeros
    cache = z(4, 16, 2, 64, dtype=torch.float16)
    table, pos = z(1, 2, dtype=torch.int32), z(1, 1, dtype=torch.int32)
    q = z(1, 1, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        lib.misa_paged_attention(q, cache, cache, table, pos)
    with pytest.raises(TypeError):
        lib.misa_paged_attention(q.float(), cache.float(), cache.float(), table, pos)
    with pytest.raises(ValueError):
        lib.misa_paged_append(q, q, pos, table, cache, cache)
    with pytest.raises(ValueError):
        lib.misa_pages_fork(table, pos[0], pos[0])


# ----------------------------------------------------------------- the oracle on hand cases

def test_oracle_attention_by_hand():
    # two tokens with equal scores: the mean of their values; one token: its value
    k = np.zeros((2, 2, 1, 2))
    v = np.arange(8, dtype=float).reshape(2, 2, 1, 2)
    q = np.ones((1, 2))
    out, lse, _, _ = po.attention_row(q, k, v, [1, 0], 2, [0, 3], 1.0)
    assert out.tolist() == [[(4 + 2) / 2, (5 + 3) / 2]] and np.isclose(lse[0], np.log(2))
    out, lse, _, _ = po.attention_row(q, k, v, [1, 0], 2, [1], 1.0)
    assert out.tolist() == [[6, 7]] and lse[0] == 0
    out, lse, _, _ = po.attention_row(q, k, v, [1, 0], 2, [], 1.0)
    assert out.tolist() == [[0, 0]] and lse[0] == -np.inf
    k[1, 0, 0] = [np.log(3), 0]   # weight 3 against 1
    out, lse, _, _ = po.attention_row(q, k, v, [1, 0], 2, [0, 3], 1.0)
    assert np.allclose(out, [[(3 * 4 + 2) / 4, (3 * 5 + 3) / 4]]) and np.isclose(lse[0], np.log(4))


def test_oracle_resize_by_hand():
    # rows 0 and 1 share a full page (0) and a half-filled one (2); both grow by one token: the
    # first takes a copy on the lowest free page, the last holder keeps the page
    table, refs = [[0, 2, -1], [0, 2, -1]], [2, 0, 2, 0]
    t, r, c = po.resize(table, refs, [6, 6], [7, 7], 4)
    assert t == [[0, 1, -1], [0, 2, -1]] and r == [2, 1, 1, 0] and c == [(2, 1)]
    # only row 1 grows, past the page: a copy and a fresh page
    t, r, c = po.resize(table, refs, [6, 6], [6, 9], 4)
    assert t == [[0, 2, -1], [0, 1, 3]] and r == [2, 1, 1, 1] and c == [(2, 1)]
    # a full last page needs no copy; shrinking lets go
    t, r, c = po.resize([[0, 2, -1]], [1, 0, 1, 0], [8], [9], 4)
    assert t == [[0, 2, 1]] and c == []
    t, r, c = po.resize(table, refs, [6, 6], [4, 0], 4)
    assert t == [[0, -1, -1], [-1, -1, -1]] and r == [1, 0, 0, 0]
    with pytest.raises(po.OutOfPages):
        po.resize(table, refs, [6, 6], [12, 12], 4)


def test_oracle_fork_and_compact_by_hand():
    t, r = po.fork([[0, 1], [2, -1], [3, -1]], [1, 1, 1, 1], [0, 0, -1])
    assert t == [[0, 1], [0, 1], [-1, -1]] and r == [2, 2, 0, 0]
    t, r, n, c = po.compact([[5, 1], [3, -1]], [0, 1, 0, 1, 0, 1])
    assert n == 3 and c == [(3, 0), (5, 2)]
    assert t == [[2, 1], [0, -1]] and r == [1, 1, 1, 0, 0, 0]
