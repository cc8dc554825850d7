"""The operators on a cache's pages without a GPU: refusals of the entry points
and of the binding, and pins of the tests' restatement (tests/_kv_pages.py)."""
import ctypes as C

import numpy as np
import pytest

import _kv4
import _kv_pages
from activation_sparse_moe_gb300 import build as hsbuild
from activation_sparse_moe_gb300 import hs

A = 0x100000  # a fake, aligned device address: validation fails before it is touched
STEP = 4096   # each buffer this far from the next one


@pytest.fixture(scope="module")
def lib():
    hsbuild.build()
    return hs.lib()


# Of 4 rows of 8 entries over 100 pages, 3 forks, 50 copies: every buffer's bytes.
ROWS = dict(n=4, page=64, pages=100, width=8, stream=None)
WS = 256 + 256 + 256 + 2 * 512
CALLS = {
    "hs_kv_fork": dict(
        names="parent child length forks cached n page pages table_in width shared ring counters_in table_out len_out copy_src copy_dst "
              "counters_out short stream",
        size=dict(parent=12, child=12, length=12, cached=16, table_in=128, shared=400, ring=400, counters_in=16, table_out=128, len_out=16,
                  copy_src=12, copy_dst=12, counters_out=16, short=4),
        written="shared table_out len_out copy_src copy_dst counters_out short", same=[{"table_in", "table_out"}], forks=3),
    "hs_kv_release": dict(
        names="cached keep n page pages table_in width shared ring counters_in table_out len_out counters_out ws nb stream",
        size=dict(cached=16, keep=16, table_in=128, shared=400, ring=400, counters_in=16, table_out=128, len_out=16, counters_out=16, ws=WS),
        written="shared ring table_out len_out counters_out ws", same=[{"table_in", "table_out"}], nb=WS),
    "hs_kv_compact": dict(
        names="cached n page pages table_in width shared_in ring counters_in copies table_out shared_out copy_src copy_dst counters_out short "
              "ws nb stream",
        size=dict(cached=16, table_in=128, shared_in=400, ring=400, counters_in=16, table_out=128, shared_out=400, copy_src=200, copy_dst=200,
                  counters_out=16, short=4, ws=WS),
        written="ring table_out shared_out copy_src copy_dst counters_out short ws",
        same=[{"table_in", "table_out"}, {"shared_in", "shared_out"}], copies=50, nb=WS),
}


def _caller(lib, fn):
    c = CALLS[fn]
    ok = {x: A + STEP * i for i, x in enumerate(c["size"])}

    def call(**kw):
        a = {**ROWS, **{x: c[x] for x in ("forks", "copies", "nb") if x in c}, **ok, **kw}
        return getattr(lib, fn)(*(a[x] for x in c["names"].split()))
    return c, ok, call


def test_workspace_size(lib):
    assert hs.hs_kv_pages_workspace_size(100) == WS
    assert hs.hs_kv_pages_workspace_size(1 << 20) == 256 + (1 << 20) + (1 << 17) + 2 * (1 << 22)
    assert hs.hs_kv_pages_workspace_size(0) == hs.hs_kv_pages_workspace_size(-1) == hs.hs_kv_pages_workspace_size(1 << 30) == 0


@pytest.mark.parametrize("fn", CALLS)
def test_refusals(lib, fn):
    c, ok, call = _caller(lib, fn)
    for x in ok:
        assert call(**{x: None}) == (hs.HS_ERR_WORKSPACE if x == "ws" else hs.HS_ERR_INVALID_ARG), x
    for kw in (dict(n=0), dict(n=-1), dict(pages=0), dict(width=0), *([dict(forks=0)] if "forks" in c else []),
               *([dict(copies=0), dict(copies=-5)] if "copies" in c else [])):
        assert call(**kw) == hs.HS_ERR_INVALID_ARG, kw
    for kw in (dict(page=0), dict(page=48), dict(page=128), dict(n=4097), dict(n=4096, width=1 << 18), dict(n=1, width=1 << 25),
               dict(pages=1 << 30), *([dict(forks=4097)] if "forks" in c else []), *([dict(copies=1 << 30)] if "copies" in c else [])):
        assert call(**kw) == hs.HS_ERR_UNSUPPORTED_SHAPE, kw
    for x in ok:
        assert call(**{x: ok[x] + 2}) == hs.HS_ERR_MISALIGNED, x
    for x in ("counters_in", "counters_out", *(["ws"] if "nb" in c else [])):
        assert call(**{x: ok[x] + 4}) == hs.HS_ERR_MISALIGNED, x
    if "nb" in c:
        assert call(nb=WS - 1) == hs.HS_ERR_WORKSPACE


@pytest.mark.parametrize("fn", CALLS)
def test_outputs_that_overlap_are_refused(lib, fn):
    c, ok, call = _caller(lib, fn)
    size = c["size"]
    for x in c["written"].split():
        for y in size:
            if y == x:
                continue
            wide = 16  # both ends: y's first bytes on x's last ones, and the other way round
            ends = [ok[x] + (size[x] - 1) // wide * wide, ok[x] - (size[y] - 1) // wide * wide]
            if {x, y} not in c["same"]:
                ends.append(ok[x])
            for at in ends:
                if at == ok[x] and {x, y} in c["same"]:
                    continue
                assert call(**{y: at}) == hs.HS_ERR_INVALID_ARG, (x, y, at - ok[x])


def test_copy_refusals(lib):
    def call(pools=(A, A + (1 << 20)), n=None, nb=4096, pages=8, src=A, dst=A, copies=4):
        p = None if pools is None else (C.c_void_p * max(1, len(pools)))(*pools)
        return lib.hs_kv_copy_pages(p, len(pools or ()) if n is None else n, nb, pages, src, dst, copies, None)
    for kw in (dict(pools=None, n=1), dict(pools=()), dict(pools=(A, None)), dict(nb=0), dict(nb=-16), dict(pages=0), dict(src=None),
               dict(dst=None), dict(copies=-1)):
        assert call(**kw) == hs.HS_ERR_INVALID_ARG, kw
    for kw in (dict(pools=(A,) * 65), dict(nb=(1 << 30) + 16), dict(copies=1 << 30)):
        assert call(**kw) == hs.HS_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(pools=(A, A + 8)), dict(nb=4100), dict(src=A + 2), dict(dst=A + 1)):
        assert call(**kw) == hs.HS_ERR_MISALIGNED, kw
    assert call(copies=0) == hs.HS_OK


def test_binding_refuses_tensors_that_do_not_fit(lib):
    import torch
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64)  # noqa: E731
    ws = torch.zeros(4096, dtype=torch.uint8)

    def refused(f, base, names32, names64):
        for name in names32 + names64:
            t = base[name]
            wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]
            for bad in (t.flatten()[:-1], t.to(torch.int64 if name in names32 else torch.int32), wide):
                if bad.numel() == 1 and bad.dtype == t.dtype:
                    continue  # (one element of two is contiguous)
                with pytest.raises(hs.HsError) as e:
                    f(**{**base, name: bad})
                assert e.value.status == hs.HS_ERR_INVALID_ARG, name
    rows = dict(cached_len=i32(4), n_seqs=4, page_tokens=64, n_pages=100, table_in=i32(4, 8), table_width=8, ring=i32(100),
                counters_in=i64(2), table_out=i32(4, 8), counters_out=i64(2), stream=0)
    refused(hs.hs_kv_fork, dict(rows, parent=i32(3), child=i32(3), length=i32(3), n_forks=3, shared=i32(100), len_out=i32(4),
                                copy_src=i32(3), copy_dst=i32(3), short=i32(1)),
            ["parent", "child", "length", "cached_len", "table_in", "shared", "ring", "table_out", "len_out", "copy_src", "copy_dst",
             "short"], ["counters_in", "counters_out"])
    refused(hs.hs_kv_release, dict(rows, keep_len=i32(4), shared=i32(100), len_out=i32(4), workspace=ws),
            ["cached_len", "keep_len", "table_in", "shared", "ring", "table_out", "len_out"], ["counters_in", "counters_out"])
    refused(hs.hs_kv_compact, dict(rows, shared_in=i32(100), shared_out=i32(100), max_copies=50, copy_src=i32(50), copy_dst=i32(50),
                                   short=i32(1), workspace=ws),
            ["cached_len", "table_in", "shared_in", "ring", "table_out", "shared_out", "copy_src", "copy_dst", "short"],
            ["counters_in", "counters_out"])
    pool = torch.zeros(8, 64, dtype=torch.uint8)
    copy = dict(pools=[pool, pool.clone()], page_bytes=64, n_pages=8, src=i32(4), dst=i32(4), n_copies=4, stream=0)
    refused(hs.hs_kv_copy_pages, copy, ["src", "dst"], [])
    for kw in (dict(pools=[]), dict(pools=[pool, torch.zeros(7, 64, dtype=torch.uint8)]), dict(pools=[pool[:, ::2]]), dict(n_pages=9),
               dict(page_bytes=80), dict(n_copies=5)):
        with pytest.raises(hs.HsError) as e:
            hs.hs_kv_copy_pages(**{**copy, **kw})
        assert e.value.status == hs.HS_ERR_INVALID_ARG, kw
    with pytest.raises(hs.HsError) as e:
        hs.hs_kv_release(**dict(rows, keep_len=i32(4), shared=i32(100), len_out=i32(4)))
    assert e.value.status == hs.HS_ERR_WORKSPACE


# ------------------------------------------------ pins of the restatement
def test_fork_by_hand():
    table = np.array([[5, 2, 7], [-1] * 3, [-1] * 3, [9, -1, -1]], np.int32)
    ring = np.array([0, 1, 3, 4, 6, 8, -1, -1, -1, -1], np.int32)
    zero = np.zeros(10, np.int32)
    r = _kv_pages.fork([0, 0], [1, 2], [40, 32], [44, 0, 0, 16], 16, 10, table, zero, ring, [20, 26])
    assert r["short"] == 0 and r["counters"] == [21, 26] and r["len"] == [44, 40, 32, 16]
    assert r["table"].tolist() == [[5, 2, 7], [5, 2, 0], [5, 2, -1], [9, -1, -1]]
    assert r["copy_src"] == [7, -1] and r["copy_dst"] == [0, -1]
    assert r["shared"].tolist() == [0, 0, 2, 0, 0, 2, 0, 0, 0, 0]
    for bad in (([0, 0], [1, 1], [8, 8]), ([0, 0], [1, 3], [8, 8]), ([0, 4], [1, 2], [8, 8]), ([0, 0], [1, 2], [8, 45]),
                ([0, 0], [1, 2], [8, -1]), ([0, 1], [2, 1], [8, 0])):
        r = _kv_pages.fork(*bad, [44, 0, 0, 16], 16, 10, table, zero, ring, [20, 26])
        assert r["short"] == (2 if bad[1] == [1, 1] else 1) and np.array_equal(r["table"], table) and not r["shared"].any()
    assert _kv_pages.fork([0, 0], [1, 2], [8, 8], [44, 0, 0, 16], 16, 10, table, zero, ring, [20, 21])["short"] == 1


def test_release_by_hand():
    table = np.array([[5, 2, 7], [5, 2, 0], [5, 2, -1]], np.int32)
    shared = np.zeros(10, np.int32)
    shared[[5, 2]] = 2
    ring = np.arange(10, dtype=np.int32) * 0 - 1
    r = _kv_pages.release([44, 40, 32], [33, 0, 16], 16, 10, table, shared, ring, [21, 26])
    assert r["len"] == [33, 0, 16] and r["table"].tolist() == [[5, 2, 7], [-1] * 3, [5, -1, -1]]
    assert r["shared"][5] == 1 and r["shared"][2] == 0 and r["ring"][6] == 0 and r["counters"] == [21, 27]
    r = _kv_pages.release([44, 40, 32], [0, 0, 0], 16, 10, table, shared, ring, [21, 26])
    assert not r["shared"].any() and [r["ring"][i % 10] for i in range(26, 30)] == [0, 2, 5, 7] and r["counters"] == [21, 30]


def test_compact_by_hand():
    table = np.array([[5, 2, -1], [5, 9, 0]], np.int32)
    shared = np.array([0, 3, 0, 0, 0, 1, 0, 0, 0, 0], np.int32)
    ring = np.full(10, -1, np.int32)
    r = _kv_pages.compact([20, 40], 16, 10, table, shared, ring, [7, 9], 3)
    assert r["short"] == 0 and r["copy_src"] == [5, 9, -1] and r["copy_dst"] == [1, 3, -1]  # 0 2 5 9 are used
    assert r["table"].tolist() == [[1, 2, -1], [1, 3, 0]] and r["shared"].tolist() == [0, 1] + [0] * 8
    assert r["ring"].tolist()[:6] == [4, 5, 6, 7, 8, 9] and r["counters"] == [0, 6]
    r = _kv_pages.compact([20, 40], 16, 10, table, shared, ring, [7, 9], 1)
    assert r["short"] == 1 and np.array_equal(r["table"], table) and r["counters"] == [7, 9] and r["copy_src"] == [-1]


def test_rows_keep_their_books():
    """Of the tests' rows every page has one place: with as many rows as its count
    says, in the ring, or lost."""
    for seed in range(20):
        r = _kv_pages.Rows(seed, 30, 16, 6, 5, lost=3)
        times = np.bincount(r.table[r.table >= 0], minlength=r.n_pages)
        ring = r.ring[r.ring >= 0]
        assert np.array_equal(np.maximum(times - 1, 0), r.shared) and len(set(ring)) == len(ring) == r.counters[1] - r.counters[0]
        assert not times[ring].any()
        p, c, m = r.forks(5)
        f = _kv_pages.fork(p, c, m, r.cached, 16, r.n_pages, r.table, r.shared, r.ring, r.counters)
        if f["short"] == 0:
            keep = np.where(np.isin(np.arange(30), c), 0, f["len"])
            b = _kv_pages.release(f["len"], keep, 16, r.n_pages, f["table"], f["shared"], r.ring, f["counters"])
            assert np.array_equal(b["shared"], r.shared) and np.array_equal(b["table"], r.table)
            assert b["counters"][1] - b["counters"][0] == r.counters[1] - r.counters[0]
    assert _kv4.record_bytes(16, 64) % 16 == 0
