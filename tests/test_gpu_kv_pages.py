"""The operators on a cache's pages on the GPU, entry by entry against their
plain restatement (tests/_kv_pages.py): whole numbers, so all of it is exact."""
import numpy as np
import pytest
import torch

import _kv4
import _kv_pages
from activation_sparse_moe_gb300 import hs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from activation_sparse_moe_gb300 import build
    build.build()
    hs.lib()


def _d(a, t=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to("cuda", t)


def _i(*s, t=torch.int32):
    return torch.full(s, -7, dtype=t, device="cuda")


def _np(**kw):
    return {k: v.cpu().numpy() for k, v in kw.items()}


def _same(got, want):
    for name in want:
        assert np.array_equal(np.atleast_1d(got[name]), np.atleast_1d(np.asarray(want[name]))), name


def _workspace(n_pages):
    return torch.zeros(hs.hs_kv_pages_workspace_size(n_pages), dtype=torch.uint8, device="cuda")


def _fork(p, c, m, r, in_place=False, counters=None):
    n, w = r.table.shape
    table = _d(r.table)
    out = table if in_place else torch.full_like(table, -7)
    shared, length, src, dst, short, cout = _d(r.shared), _i(n), _i(len(p)), _i(len(p)), _i(1), _i(2, t=torch.int64)
    hs.hs_kv_fork(_d(p), _d(c), _d(m), len(p), _d(r.cached), n, r.page, r.n_pages, table, w, shared, _d(r.ring),
                  _d(counters or r.counters, torch.int64), out, length, src, dst, cout, short)
    return _np(table=out, shared=shared, len=length, copy_src=src, copy_dst=dst, counters=cout, short=short)


def _release(cached, keep, r, table, shared, ring, counters, in_place=False, ws=None):
    n, w = table.shape
    tin, shared, ring = _d(table), _d(shared), _d(ring)
    out = tin if in_place else torch.full_like(tin, -7)
    length, cout = _i(n), _i(2, t=torch.int64)
    ws = _workspace(r.n_pages) if ws is None else ws
    hs.hs_kv_release(_d(cached), _d(keep), n, r.page, r.n_pages, tin, w, shared, ring, _d(counters, torch.int64), out, length, cout, ws)
    return _np(table=out, shared=shared, ring=ring, len=length, counters=cout)


def _compact(r, copies, in_place=False, ws=None, cached=None):
    n, w = r.table.shape
    tin, sin, ring = _d(r.table), _d(r.shared), _d(r.ring)
    out, sout = (tin, sin) if in_place else (torch.full_like(tin, -7), torch.full_like(sin, -7))
    src, dst, short, cout = _i(copies), _i(copies), _i(1), _i(2, t=torch.int64)
    ws = _workspace(r.n_pages) if ws is None else ws
    hs.hs_kv_compact(_d(r.cached if cached is None else cached), n, r.page, r.n_pages, tin, w, sin, ring, _d(r.counters, torch.int64),
                     copies, out, sout, src, dst, cout, short, ws)
    return _np(table=out, shared=sout, ring=ring, copy_src=src, copy_dst=dst, counters=cout, short=short)


SIZES = [(2, 16, 1, 1), (3, 64, 5, 2), (9, 32, 33, 7), (40, 16, 64, 50), (300, 64, 7, 31), (1000, 16, 129, 5), (4096, 16, 3, 999),
         (257, 32, 300, 1)]


@pytest.mark.parametrize("n,page,width,spare", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(n, page, width, spare, in_place):
    r = _kv_pages.Rows(n + page, n, page, width, spare + n)
    p, c, m = r.forks(n)
    want = _kv_pages.fork(p, c, m, r.cached, page, r.n_pages, r.table, r.shared, r.ring, r.counters)
    assert want["short"] == 0 or len(p) < 1
    if len(p):
        _same(_fork(p, c, m, r, in_place), want)


def test_fork_of_one_parent_many_times():
    """4000 children of one row: one page has 4000 owners more."""
    r = _kv_pages.Rows(1, 4001, 16, 5, 5000, share=0, empty=1)
    r.cached[17] = 5 * 16 - 3
    r.table[17] = r.ring[r.ring >= 0][-5:]
    r.counters[1] -= 5
    kids = np.setdiff1d(np.arange(4001), [17]).astype(np.int32)[:4000]
    p, m = np.full(4000, 17, np.int32), np.full(4000, 77, np.int32)
    m[::7] = 64
    m[1::7] = 0
    want = _kv_pages.fork(p, kids, m, r.cached, 16, r.n_pages, r.table, r.shared, r.ring, r.counters)
    assert want["short"] == 0 and want["shared"].max() > 3000
    _same(_fork(p, kids, m, r), want)


@pytest.mark.parametrize("why", ["ring", "rows", "itself", "longer", "negative", "width", "holds", "twice", "all"])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_is_refused_as_a_whole(why, in_place):
    r = _kv_pages.Rows(7, 60, 16, 12, 60, empty=0.5)
    p, c, m = r.forks(12)
    m[0] = max(int(r.cached[p[0]]) // 16 * 16 - 5, 1)
    counters = list(r.counters)
    full = int(np.flatnonzero(r.cached > 0)[0])
    if why in ("ring", "all"):
        counters[1] = counters[0]
    if why in ("rows", "all"):
        p[3], c[4] = 60, -1
    if why in ("itself", "all"):
        p[5] = c[5]
    if why in ("longer", "all"):
        m[6] = r.cached[p[6]] + 1
    if why in ("negative", "all"):
        m[7] = -3
    if why == "width":
        r.cached[p[8]] = 12 * 16 + 5
        m[8] = 12 * 16 + 1
    if why in ("holds", "all"):
        c[9] = full
    if why in ("twice", "all"):
        c[10] = c[11]
    want = _kv_pages.fork(p, c, m, r.cached, 16, r.n_pages, r.table, r.shared, r.ring, counters)
    assert want["short"] > 0 and np.array_equal(want["table"], r.table)
    _same(_fork(p, c, m, r, in_place, counters), want)


@pytest.mark.parametrize("n,page,width,spare", SIZES + [(1, 16, 1, 0), (64, 16, 4000, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release(n, page, width, spare, in_place):
    r = _kv_pages.Rows(3 * n + page, n, page, width, spare, share=0.5)
    keep = np.where(r.rng.random(n) < 0.5, 0, r.rng.integers(-2, width * page + 9, n)).astype(np.int32)
    want = _kv_pages.release(r.cached, keep, page, r.n_pages, r.table, r.shared, r.ring, r.counters)
    _same(_release(r.cached, keep, r, r.table, r.shared, r.ring, r.counters, in_place), want)


def test_release_of_everything_and_of_nothing():
    """All owners of every page at once (the last one frees it, whoever that is), the
    ring's order that of the pages; then nothing is left to give.  One workspace."""
    r = _kv_pages.Rows(5, 800, 16, 40, 0, share=0.8)
    ws = _workspace(r.n_pages)
    keep = np.full(800, -1, np.int32)
    want = _kv_pages.release(r.cached, keep, 16, r.n_pages, r.table, r.shared, r.ring, r.counters)
    assert want["counters"][1] - want["counters"][0] == r.n_pages and not want["shared"].any()
    for _ in range(3):
        _same(_release(r.cached, keep, r, r.table, r.shared, r.ring, r.counters, ws=ws), want)
    again = _kv_pages.release(np.zeros(800, np.int32), keep, 16, r.n_pages, want["table"], want["shared"], want["ring"], want["counters"])
    assert again["counters"] == want["counters"]
    _same(_release(np.zeros(800, np.int32), keep, r, want["table"], want["shared"], want["ring"], want["counters"], ws=ws), again)
    assert not ws[256:256 + r.n_pages].any() and not ws[:4].any()


def test_release_passes_over_pages_outside_the_pool():
    r = _kv_pages.Rows(6, 50, 32, 20, 4, hole=0.2)
    r.table[3, 2], r.table[5, 1] = r.n_pages, 1 << 29
    r.cached[[3, 5]] = 20 * 32
    keep = (r.cached // 3).astype(np.int32)
    want = _kv_pages.release(r.cached, keep, 32, r.n_pages, r.table, r.shared, r.ring, r.counters)
    _same(_release(r.cached, keep, r, r.table, r.shared, r.ring, r.counters), want)


@pytest.mark.parametrize("n,page,width,spare", SIZES + [(1, 16, 1, 0), (5, 16, 2, 40), (64, 16, 4000, 70000), (3, 16, 2, 262144)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(n, page, width, spare, in_place):
    r = _kv_pages.Rows(5 * n + page, n, page, width, spare, share=0.4, lost=2)
    copies = r.n_pages // 2 + 1
    want = _kv_pages.compact(r.cached, page, r.n_pages, r.table, r.shared, r.ring, r.counters, copies)
    assert want["short"] == 0
    _same(_compact(r, copies, in_place), want)


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_of_more_moves_than_asked_for_does_nothing(in_place):
    r = _kv_pages.Rows(8, 100, 16, 30, 700)
    moves = sum(x >= 0 for x in _kv_pages.compact(r.cached, 16, r.n_pages, r.table, r.shared, r.ring, r.counters, r.n_pages)["copy_src"])
    ws = _workspace(r.n_pages)
    for copies in (1, moves - 1, moves, moves + 1):
        want = _kv_pages.compact(r.cached, 16, r.n_pages, r.table, r.shared, r.ring, r.counters, copies)
        assert (want["short"] > 0) == (copies < moves)
        _same(_compact(r, copies, in_place, ws), want)


def test_compact_of_no_page_and_of_all():
    r = _kv_pages.Rows(9, 10, 16, 4, 33)
    none = np.full(10, -4, np.int32)
    want = _kv_pages.compact(none, 16, r.n_pages, r.table, r.shared, r.ring, r.counters, 3)
    assert want["counters"] == [0, r.n_pages]
    _same(_compact(r, 3, cached=none), want)
    r = _kv_pages.Rows(10, 10, 16, 8, 0, share=0, empty=0)
    want = _kv_pages.compact(r.cached, 16, r.n_pages, r.table, r.shared, r.ring, r.counters, 3)
    assert want["counters"] == [0, 0] and np.array_equal(want["table"], r.table)
    _same(_compact(r, 3), want)


def test_compact_leaves_entries_outside_the_pool():
    r = _kv_pages.Rows(11, 30, 16, 20, 100, hole=0.3)
    r.table[4, 1], r.cached[4] = r.n_pages + 5, 100
    want = _kv_pages.compact(r.cached, 16, r.n_pages, r.table, r.shared, r.ring, r.counters, r.n_pages)
    _same(_compact(r, r.n_pages), want)


@pytest.mark.parametrize("page_bytes,n_pages,pools,copies", [(16, 9, 1, 4), (8192, 40, 3, 1), (8208, 300, 2, 150), (16 * 257, 999, 5, 400),
                                                             (32896, 77, 64, 30), (1 << 20, 20, 2, 9), (48, 9000, 1, 4096)])
def test_copy_pages(page_bytes, n_pages, pools, copies):
    rng = np.random.default_rng(page_bytes)
    data = [torch.from_numpy(rng.integers(0, 256, (n_pages, page_bytes), dtype=np.uint8)) for _ in range(pools)]
    perm = rng.permutation(n_pages)
    used = min(copies, n_pages // 2)
    src, dst = np.full(copies, -1), np.full(copies, -1)
    where = np.sort(rng.permutation(copies)[:used])
    src[where], dst[where] = perm[:used], perm[used:2 * used]
    if copies > 8:                                  # several from one page, pairs that are none
        src[where[1]] = src[where[0]]
        src[where[2]], dst[where[3]], src[where[4]], dst[where[5]] = -1, n_pages, n_pages + 100, -(1 << 31)
    want = [x.clone() for x in data]
    for x, y in zip(want, data):
        for a, b in zip(src, dst):
            if 0 <= a < n_pages and 0 <= b < n_pages:
                x[b] = y[a]
    dev = [x.cuda() for x in data]
    hs.hs_kv_copy_pages(dev, page_bytes, n_pages, _d(src), _d(dst), copies)
    for x, y in zip(dev, want):
        assert torch.equal(x.cpu(), y)


def test_copy_of_pages_past_4_gb():
    """Offsets that do not fit 32 bits, and no byte beside the target changes."""
    page_bytes, n_pages = 1 << 20, 4200
    pool = torch.zeros(n_pages, page_bytes, dtype=torch.uint8, device="cuda")
    pool[4199] = torch.arange(page_bytes, device="cuda") % 251
    pool[1] = 7
    hs.hs_kv_copy_pages([pool], page_bytes, n_pages, _d([4199, 1]), _d([4, 4198]), 2)
    assert torch.equal(pool[4], pool[4199]) and bool((pool[4198] == 7).all())
    assert not pool[3].any() and not pool[5].any() and not pool[4197].any()


def test_fork_copy_decode_end_and_compact_as_a_server_does():
    """A prompt's samples decode on pages of their own behind shared ones, end, and the
    pool is compacted: plan, append and read between the calls see each request's own
    tokens all along."""
    page, hkv, dim, n_pages, width, rows = 16, 2, 64, 64, 12, 6
    rng = np.random.default_rng(12)
    pools = [torch.full((n_pages, hkv, _kv4.record_bytes(page, dim)), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    caches = [hs.make_kv4_cache(p, n_pages, page, hkv, dim) for p in pools]
    size = hkv * _kv4.record_bytes(page, dim)
    table, ring = torch.full((rows, width), -1, dtype=torch.int32, device="cuda"), _d(rng.permutation(n_pages))
    length, counters, shared, ws = _d(np.zeros(rows)), _d([0, n_pages], torch.int64), _d(np.zeros(n_pages)), _workspace(n_pages)
    short, src, dst = _i(1), _i(n_pages), _i(n_pages)
    held = [[np.zeros((0, hkv, dim), np.float32) for _ in range(rows)] for _ in range(2)]  # keys, by layer and row

    def step(new):
        nonlocal length, counters
        seq, qs, slot, cout = _i(rows), _i(rows + 1), _i(128, t=torch.int64), _i(2, t=torch.int64)
        hs.hs_kv4_plan(length, _d(new), rows, page, n_pages, table, width, ring, counters, 128, table, seq, qs, slot, None, cout, short)
        assert int(short) == 0
        for layer, c in enumerate(caches):
            t = int(sum(new))
            k = _kv4.bf16(rng, (t, hkv, dim))
            hs.hs_kv4_append(c, k.cuda(), (-k).cuda(), slot, t)
            at = 0
            for i, m in enumerate(new):
                held[layer][i] = np.concatenate((held[layer][i], _kv4.values(k[at:at + m].float().numpy())))
                at += m
        length, counters = seq, cout

    def check():
        for layer, c in enumerate(caches):
            for i in range(rows):
                m = len(held[layer][i])
                assert m == int(length[i])
                if m:
                    j = torch.arange(m, device="cuda")
                    slots = table[i, j // page].long() * page + j % page
                    k, v = (torch.empty(m, hkv, dim, device="cuda") for _ in range(2))
                    hs.hs_kv4_read(c, slots, m, k_f32=k, v_f32=v)
                    assert np.array_equal(k.cpu().numpy(), held[layer][i].astype(np.float32)) and v.shape == k.shape

    def fork(p, c, m):
        nonlocal length, counters
        out, cout = _i(rows), _i(2, t=torch.int64)
        hs.hs_kv_fork(_d(p), _d(c), _d(m), len(p), length, rows, page, n_pages, table, width, shared, ring, counters, table, out, src, dst,
                      cout, short)
        assert int(short) == 0
        hs.hs_kv_copy_pages(pools, size, n_pages, src, dst, len(p))
        for x, y, z in zip(p, c, m):
            for layer in range(2):
                held[layer][y] = held[layer][x][:z]
        length, counters = out, cout

    def release(keep):
        nonlocal length, counters
        out, cout = _i(rows), _i(2, t=torch.int64)
        hs.hs_kv_release(length, _d(keep), rows, page, n_pages, table, width, shared, ring, counters, table, out, cout, ws)
        for layer in range(2):
            held[layer][:] = [x[:max(z, 0)] for x, z in zip(held[layer], keep)]
        length, counters = out, cout

    step([53, 0, 0, 20, 0, 0])
    fork([0, 0, 0], [1, 2, 4], [53, 48, 37])
    check()
    for _ in range(3):
        step([1, 1, 1, 1, 1, 0])
    step([0, 20, 0, 0, 0, 0])
    check()
    fork([1], [5], [70])                      # a sample of a sample
    step([1, 1, 1, 1, 1, 30])
    release([0, 1 << 20, 0, 1 << 20, 25, 1 << 20])   # the prompt itself ends, its pages live on in its samples
    check()
    used = len({int(p) for i in range(rows) for p in table[i, :_kv_pages.up(int(length[i]), page)]})
    assert int(counters[1] - counters[0]) == n_pages - used
    cout = _i(2, t=torch.int64)
    hs.hs_kv_compact(length, rows, page, n_pages, table, width, shared, ring, counters, n_pages, table, shared, src, dst, cout, short, ws)
    hs.hs_kv_copy_pages(pools, size, n_pages, src, dst, n_pages)
    counters = cout
    assert int(short) == 0 and int(table.max()) == used - 1 and counters.tolist() == [0, n_pages - used]
    check()
    step([7, 1, 9, 1, 0, 1])
    check()
    release([0] * rows)
    assert not shared.any() and int(counters[1] - counters[0]) == n_pages and not bool((table >= 0).any())
    assert hs.hs_device_status() == hs.HS_OK


def test_calls_in_a_graph_and_two_graphs_that_share_a_workspace():
    """Captured once, replayed in turn: each leaves the workspace as the next needs it."""
    r = _kv_pages.Rows(13, 200, 16, 20, 300, share=0.5)
    keep = np.where(r.rng.random(200) < 0.5, 0, r.cached // 2).astype(np.int32)
    ws, copies, w = _workspace(r.n_pages), r.n_pages, r.width
    cached, keep_d, table, counters = _d(r.cached), _d(keep), _d(r.table), _d(r.counters, torch.int64)
    a = dict(table=_i(200, w), shared=_d(r.shared), ring=_d(r.ring), len=_i(200), counters=_i(2, t=torch.int64))
    b = dict(table=_i(200, w), shared=_i(r.n_pages), ring=_d(r.ring), copy_src=_i(copies), copy_dst=_i(copies),
             counters=_i(2, t=torch.int64), short=_i(1))
    shared = _d(r.shared)

    def release():
        a["shared"].copy_(shared)
        hs.hs_kv_release(cached, keep_d, 200, 16, r.n_pages, table, w, a["shared"], a["ring"], counters, a["table"], a["len"], a["counters"], ws)

    def compact():
        hs.hs_kv_compact(cached, 200, 16, r.n_pages, table, w, shared, b["ring"], counters, copies, b["table"], b["shared"], b["copy_src"],
                         b["copy_dst"], b["counters"], b["short"], ws)
    stream, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(stream):
        for f in (release, compact):
            f()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                f()
            graphs.append(g)
        for g in (graphs[0], graphs[1], graphs[1], graphs[0], graphs[1]):
            a["ring"].copy_(_d(r.ring))
            for x in (a["table"], a["len"], b["table"], b["copy_src"], b["short"]):
                x.fill_(-9)
            g.replay()
    torch.cuda.synchronize()
    want = _kv_pages.compact(r.cached, 16, r.n_pages, r.table, r.shared, r.ring, r.counters, copies)
    _same(_np(**b), want)
    with torch.cuda.stream(stream):
        graphs[0].replay()
    torch.cuda.synchronize()
    _same(_np(**a), _kv_pages.release(r.cached, keep, 16, r.n_pages, r.table, r.shared, r.ring, r.counters))


def test_calls_on_other_streams_than_the_current_one():
    """The stream given, as an object or as its handle; two at once with a workspace each."""
    r = _kv_pages.Rows(14, 300, 16, 30, 400, share=0.5)
    keep = (r.cached // 2).astype(np.int32)
    rel = _kv_pages.release(r.cached, keep, 16, r.n_pages, r.table, r.shared, r.ring, r.counters)
    com = _kv_pages.compact(r.cached, 16, r.n_pages, r.table, r.shared, r.ring, r.counters, r.n_pages)
    p, c, m = r.forks(50)
    frk = _kv_pages.fork(p, c, m, r.cached, 16, r.n_pages, r.table, r.shared, r.ring, r.counters)
    assert frk["short"] == 0
    cached, keep_d, table, counters, shared = _d(r.cached), _d(keep), _d(r.table), _d(r.counters, torch.int64), _d(r.shared)
    i64 = lambda: _i(2, t=torch.int64)  # noqa: E731
    a = dict(table=_i(300, 30), shared=_d(r.shared), ring=_d(r.ring), len=_i(300), counters=i64())
    b = dict(table=_i(300, 30), shared=_i(r.n_pages), ring=_d(r.ring), copy_src=_i(r.n_pages), copy_dst=_i(r.n_pages), counters=i64(), short=_i(1))
    f = dict(table=_i(300, 30), shared=_d(r.shared), len=_i(300), copy_src=_i(50), copy_dst=_i(50), counters=i64(), short=_i(1))
    ring, fp, fc, fm = _d(r.ring), _d(p), _d(c), _d(m)
    pool = torch.arange(r.n_pages, dtype=torch.int32, device="cuda").repeat_interleave(64).view(r.n_pages, 64)
    ws, streams = [_workspace(r.n_pages) for _ in range(2)], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    hs.hs_kv_release(cached, keep_d, 300, 16, r.n_pages, table, 30, a["shared"], a["ring"], counters, a["table"], a["len"], a["counters"], ws[0],
                     stream=streams[0])
    hs.hs_kv_compact(cached, 300, 16, r.n_pages, table, 30, shared, b["ring"], counters, r.n_pages, b["table"], b["shared"], b["copy_src"],
                     b["copy_dst"], b["counters"], b["short"], ws[1], stream=streams[1].cuda_stream)
    hs.hs_kv_copy_pages([pool], 256, r.n_pages, b["copy_src"], b["copy_dst"], r.n_pages, stream=streams[1])
    hs.hs_kv_fork(fp, fc, fm, 50, cached, 300, 16, r.n_pages, table, 30, f["shared"], ring, counters, f["table"], f["len"], f["copy_src"],
                  f["copy_dst"], f["counters"], f["short"], stream=streams[2].cuda_stream)
    torch.cuda.synchronize()
    _same(_np(**a), rel)
    _same(_np(**b), com)
    _same(_np(**f), frk)
    for x, y in zip(com["copy_src"], com["copy_dst"]):
        if x >= 0:
            assert int(pool[y, 63]) == x
