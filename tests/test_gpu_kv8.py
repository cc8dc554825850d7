"""The 8-bit key/value cache on the GPU: append, read and attention against their
64-bit restatements (tests/_kv8.py)."""
import numpy as np
import pytest
import torch

import _kv4
import _kv8
from activation_sparse_moe_gb300 import hs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from activation_sparse_moe_gb300 import build
    build.build()
    hs.lib()


# --------------------------------------------------------- append and read
def _cache(n_pages, page, hkv, dim, fill=0xFF):
    pool = torch.full((n_pages, hkv, _kv8.record_bytes(page, dim)), fill, dtype=torch.uint8, device="cuda")
    c = hs.make_kv8_cache(pool, n_pages, page, hkv, dim)
    assert hs.hs_kv8_pool_bytes(c) == pool.numel()
    return pool, c


def _rows(rng, t, h, d):
    """bf16 rows of very different sizes, with what a quantiser meets: values at a scale's
    border and between two codes, zeros of both signs, tiny ones, infinities, NaN and values
    past what the cache holds."""
    x = rng.normal(0, 1, (t, h, d)).astype(np.float32)
    x *= np.exp(rng.normal(0, 3, (t, h, 1))).astype(np.float32)
    flat = x.reshape(-1, 64)
    n, at = len(flat), np.arange(64)
    kinds = [lambda g: g * 0, lambda g: np.where(at % 2, 0.0, -0.0), lambda g: (at + 1) * 1.75, lambda g: (at + 1) / 16 * 7.03125,
             lambda g: g * 1e-6, lambda g: g * 1e-38, lambda g: np.where(at == 5, np.inf, g), lambda g: np.where(at == 63, np.nan, g),
             lambda g: np.where(at == 0, -np.inf, g), lambda g: np.where(at == 9, 57344., g), lambda g: np.where(at == 9, -57600., g),
             lambda g: np.where(at == 1, 3e38, g), lambda g: (2 * at + 1) * 2.0 ** -25, lambda g: np.where(at == 3, 448., g / 999)]
    for i, f in enumerate(kinds):
        if i < n:
            flat[(i * 7) % n] = f(flat[(i * 7) % n])
    return torch.from_numpy(x).bfloat16()


def _same_bytes(got, want):
    """Pools byte by byte (NaN codes among them)."""
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("t,hkv,dim,page", [(1, 1, 64, 16), (1, 2, 128, 64), (3, 3, 128, 16), (37, 5, 64, 32), (200, 8, 128, 64),
                                            (1031, 2, 64, 64), (21, 33, 128, 16), (5, 256, 64, 32)])
def test_append_writes_the_definition_bit_for_bit_and_read_returns_it(t, hkv, dim, page):
    """Whole requests from a page's start, K and V out of one fused buffer."""
    rng = np.random.default_rng(t * 7 + hkv)
    n_pages = -(-t // page) + 2
    pool, c = _cache(n_pages, page, hkv, dim)
    k, v = _rows(rng, t, hkv, dim), _rows(rng, t, hkv, dim)
    j = np.arange(t)
    slots = rng.permutation(n_pages)[j // page] * page + j % page
    fused = torch.randn(t, 2 * hkv + 1, dim + 8).bfloat16().cuda()
    fused[:, :hkv, :dim], fused[:, hkv:2 * hkv, :dim] = k.cuda(), v.cuda()
    hs.hs_kv8_append(c, fused[:, :hkv, :dim], fused[:, hkv:2 * hkv, :dim], torch.from_numpy(slots).cuda(), t)
    want = np.full(pool.shape, 0xFF, np.uint8)
    _kv8.append(want, page, dim, slots, k.float().numpy(), v.float().numpy())
    _same_bytes(pool, want)
    read = slots.copy()
    read[t // 2] = -1                      # no token there: zeros
    read = np.concatenate((read, [n_pages * page, -5]))
    sl = torch.from_numpy(read).cuda()
    shape = (t + 2, hkv, dim)
    kb, vb = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kf, vf = (torch.empty(shape, dtype=torch.float32, device="cuda") for _ in range(2))
    hs.hs_kv8_read(c, sl, t + 2, kb, vb, kf, vf)
    for ref, b, f in zip(_kv8.read(want, page, dim, read), (kb, vb), (kf, vf)):
        assert np.array_equal(f.cpu().numpy(), ref, equal_nan=True) and np.array_equal(b.double().cpu().numpy(), ref, equal_nan=True)
    only = torch.empty(shape, dtype=torch.float32, device="cuda")
    hs.hs_kv8_read(c, sl, t + 2, v_f32=only)
    assert torch.equal(only.nan_to_num(7), vf.nan_to_num(7))


@pytest.mark.parametrize("hkv,dim,page", [(1, 64, 16), (2, 128, 64), (3, 128, 16), (9, 64, 32)])
@pytest.mark.parametrize("steps", ["ones", "drafts", "chunks"])
def test_append_to_blocks_that_hold_tokens(hkv, dim, page, steps):
    """Requests that grow call by call: scales that grow under older codes, again and
    again, and such that stay; blocks begun anew; requests cut back.  Bit for bit."""
    rng = np.random.default_rng(hkv + dim)
    n, n_pages = 7, 24
    pool, c = _cache(n_pages, page, hkv, dim)
    want = np.full(pool.shape, 0xFF, np.uint8)
    width = n_pages // n
    table, length = rng.permutation(n_pages)[:n * width].reshape(n, width), np.zeros(n, int)
    for turn in range(20):
        most = {"ones": 1, "drafts": 5, "chunks": 40}[steps]
        new = np.minimum(rng.integers(0, most + 1, n), width * page - length)
        if turn % 5 == 4:                   # some are cut back, to the middle of a block or to nothing
            length = np.where(rng.random(n) < 0.5, np.maximum(length - rng.integers(0, 9, n), 0), length)
            length[turn % n] = 0
            new = np.minimum(new, width * page - length)
        slots = np.concatenate([table[i, np.arange(length[i], length[i] + new[i]) // page] * page +
                                np.arange(length[i], length[i] + new[i]) % page for i in range(n)]).astype(np.int64)
        t = len(slots)
        if not t:
            continue
        k, v = _rows(rng, t, hkv, dim), (_rows(rng, t, hkv, dim).float() * 2.0 ** int(rng.integers(-9, 9))).bfloat16()
        hs.hs_kv8_append(c, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), t)
        _kv8.append(want, page, dim, slots, k.float().numpy(), v.float().numpy())
        length += new
    _same_bytes(pool, want)


def test_append_takes_a_blocks_tokens_in_any_order_and_skips_slots_outside():
    page, hkv, dim = 32, 2, 128
    rng = np.random.default_rng(4)
    pool, c = _cache(6, page, hkv, dim)
    want = np.full(pool.shape, 0xFF, np.uint8)
    parts = [rng.permutation(16) + 16 * b for b in rng.permutation(12)]
    parts[3], parts[5] = np.array([-1, 6 * page, -(1 << 62)]), np.array([1 << 40])
    parts[7] = parts[7][:5]
    parts.insert(2, np.array([-1]))
    slots = np.concatenate(parts).astype(np.int64)
    t = len(slots)
    k, v = _rows(rng, t, hkv, dim), _rows(rng, t, hkv, dim)

    # (the block of five tokens may begin behind offset 0: it then holds "older" tokens of scale NaN,
    # read as the largest exponent; give it one that is sound)
    for p in (pool, want):
        p[:, :, 2 * page * dim:] = 0
        scales = torch.ones(4, dtype=torch.float32).view(torch.uint8)
        for b in range(2):
            p[:, :, 2 * page * dim + 16 * b:2 * page * dim + 16 * b + 8] = scales[:8].cuda() if p is pool else scales[:8].numpy()
    hs.hs_kv8_append(c, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), t)
    _kv8.append(want, page, dim, slots, k.float().numpy(), v.float().numpy())
    _same_bytes(pool, want)


def test_append_of_no_token_touches_nothing():
    pool, c = _cache(3, 16, 2, 64)
    k = torch.full((4, 2, 64), float("nan"), device="cuda").bfloat16()
    hs.hs_kv8_append(c, k, k, torch.tensor([-1, 48, 1 << 40, -(1 << 62)], device="cuda"), 4)
    hs.hs_kv8_append(c, k, k, torch.zeros(4, dtype=torch.int64, device="cuda"), 0)
    torch.cuda.synchronize()
    assert (pool == 0xFF).all()


def test_append_of_blocks_named_apart_touches_no_other_block():
    """What such blocks hold is undefined; every other one holds its own tokens."""
    page, hkv, dim, t = 16, 3, 128, 400
    rng = np.random.default_rng(5)
    pool, c = _cache(32, page, hkv, dim)
    k, v = _kv4.bf16(rng, (t, hkv, dim)), _kv4.bf16(rng, (t, hkv, dim))
    slots = np.arange(t)
    slots[100:200] = slots[7]                       # 101 tokens of one slot
    slots[200:240] = 16 + np.arange(40) % 2 * 48    # of two blocks in turn
    hs.hs_kv8_append(c, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), t)
    want = np.full(pool.shape, 0xFF, np.uint8)
    keep = np.r_[32:64, 80:96, 256:t]
    _kv8.append(want, page, dim, slots[keep], k[keep].float().numpy(), v[keep].float().numpy())
    whole = sorted({int(s) // page for s in slots[keep]})
    assert np.array_equal(pool.cpu().numpy()[whole], want[whole])
    assert (pool[25:] == 0xFF).all()


def test_append_of_many_tokens_and_of_the_most_heads():
    """Both ways in which the runs are given to warps, runs across their borders."""
    for t, hkv, dim, page, first in ((5000, 4, 128, 64, 5), (300, 256, 64, 16, 3), (9001, 1, 64, 32, 0), (70000, 1, 64, 64, 9)):
        rng = np.random.default_rng(t)
        n_pages = -(-(t + first) // page)
        pool, c = _cache(n_pages, page, hkv, dim, 0)
        k, v = (torch.randn((t, hkv, dim), generator=torch.Generator().manual_seed(s)).bfloat16() for s in (t, t + 1))
        j = np.arange(first, first + t)
        slots = rng.permutation(n_pages)[j // page].astype(np.int64) * page + j % page
        hs.hs_kv8_append(c, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), t)
        got = pool.cpu().numpy()
        want = np.zeros(got.shape, np.uint8)
        head = slots[:16 - first] if first else slots[:0]
        if first:                                   # the first block holds "older" tokens of scale 0: exponent -15
            p, o = divmod(int(slots[0]) // 16 * 16, page)
            for i in range(2):
                at = _kv8._scale_at(page, dim, o, i)
                want[p, :, at:at + 4] = np.array([2.0 ** -15], np.float32).view(np.uint8)
            _kv8.append(want, page, dim, head, k[:len(head)].float().numpy(), v[:len(head)].float().numpy())
        n = len(head)
        _kv8.fill(want, page, dim, slots[n:], k[n:].float().numpy(), v[n:].float().numpy())
        assert np.array_equal(got, want)


def test_pool_offsets_past_4_gigabytes():
    page, hkv, dim = 64, 8, 128
    n_pages = (5 << 30) // (hkv * _kv8.record_bytes(page, dim))
    pool, c = _cache(n_pages, page, hkv, dim)
    rng = np.random.default_rng(1)
    k, v = _kv4.bf16(rng, (70, hkv, dim)), _kv4.bf16(rng, (70, hkv, dim))
    pages = np.array([n_pages - 1, n_pages - 5])
    slots = pages[np.arange(70) // page].astype(np.int64) * page + np.arange(70) % page
    hs.hs_kv8_append(c, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), 70)
    kf = torch.empty((70, hkv, dim), dtype=torch.float32, device="cuda")
    hs.hs_kv8_read(c, torch.from_numpy(slots).cuda(), 70, k_f32=kf)
    kk, vv = _kv8.values(k.float().numpy()), _kv8.values(v.float().numpy())
    assert np.array_equal(kf.cpu().numpy(), kk)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for new in (1, 40):
        q = _kv4.bf16(rng, (new, hkv, dim))
        out = torch.empty_like(q, device="cuda")
        ws = torch.zeros(hs.hs_kv8_attention_workspace_size(c, 1, hkv), dtype=torch.uint8, device="cuda")
        hs.hs_kv8_attention(c, q.cuda(), i32([0, new]), i32([70]), i32(pages.reshape(1, 2)), 1, new, 0.1, 0, out, ws)
        _close(out, _kv4.attention(q.double().numpy(), kk, vv, new, 70, 0.1), 0.1)


# -------------------------------------------------------------- attention
def _close(out, ref, scale, vmax=6.5):
    """Bound of one output against the 64-bit one.

    Keys, values and queries are exact in fp16.  The last rounding is half a bf16
    step, 2^-8 of the value.  Before it, each probability is rounded to fp16 (2^-11
    of it), which moves an output, a mean of values, by 2^-11 * max|v| at most; the
    sum is not rounded so.  Scores are fp32 sums: 128 products of a size of at
    most 100 in all (in units of the exponent) lose 2^-23 of that at each of the
    products' 8 steps, 2^-13 of the probabilities, as much of their sum;
    exponentials 2^-22.  max|v|: of bf16 normal values and their rounding to e4m3."""
    got = out.float().cpu().double().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    bound = np.abs(ref) * 2.0 ** -8 + vmax * (2.0 ** -11 + 2 * 2.0 ** -13 + 2.0 ** -20)
    assert (err <= bound).all(), float((err / bound).max())
    norm = np.linalg.norm(ref)
    if norm > 0:  # in the mean: bf16's 2^-8 / sqrt(3) at worst, and the fp16 roundings next to it
        assert np.linalg.norm(got - ref) <= 2.0 ** -8 * norm


SHAPES = [  # cached, new, hq, hkv, dim, page
    ([0], [1], 1, 1, 64, 16),
    ([0], [1], 32, 2, 128, 64),
    ([76], [1], 32, 2, 128, 64),
    ([15, 16, 17, 63, 64, 65, 127], [1] * 7, 8, 8, 128, 16),
    ([4999], [1], 16, 1, 128, 64),
    ([4999, 3, 700], [1, 1, 1], 20, 4, 64, 32),
    ([100, 0, 31], [3, 3, 3], 32, 2, 128, 32),
    ([100, 900], [2, 0], 12, 4, 64, 64),
    ([1000], [5], 21, 3, 128, 16),
    ([333, 12, 0, 80], [8, 1, 7, 0], 56, 8, 128, 64),
    ([0, 5], [130, 77], 8, 2, 64, 16),
    ([260], [300], 7, 1, 128, 64),
    ([130, 0, 64], [257, 129, 64], 16, 1, 128, 32),
    ([10], [20], 64, 1, 64, 64),
    ([0], [513], 4, 4, 128, 64),
    ([5000, 2500], [20, 9], 16, 1, 128, 64),
    ([4000], [70], 6, 2, 64, 16),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("window", [0, 1, 50, 333])
def test_attention(case, window):
    cached, new, hq, hkv, dim, page = SHAPES[case]
    r = _kv8.Requests(case, cached, new, hq, hkv, dim, page)
    scale = dim ** -0.5
    out = r.run(hs, scale, window)
    _close(out, r.expected(scale, window), scale)


ROW_SHAPES = [  # new, hq, hkv: rows of a kv head at the ends of each row tile of the few-row kernel
    (9, 2, 2), (2, 9, 1), (3, 16, 4), (4, 8, 2), (2, 16, 2),          # 9, 18, 12, 16, 16
    (1, 17, 1), (17, 1, 1), (4, 8, 1), (8, 16, 4), (5, 24, 4), (3, 20, 2),  # 17, 17, 32, 32, 30, 30
    (3, 11, 1), (12, 8, 2), (1, 64, 1), (64, 2, 2),                   # 33, 48, 64, 64: four row warps in calls this small
]


@pytest.mark.parametrize("dim,page", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 64)])
@pytest.mark.parametrize("case", range(len(ROW_SHAPES)))
@pytest.mark.parametrize("window", [0, 1, 50, 333])
def test_attention_of_each_row_tile(case, dim, page, window):
    new, hq, hkv = ROW_SHAPES[case]
    r = _kv8.Requests(case + dim + page, [400, 0, 65], [new, new, min(new, 2)], hq, hkv, dim, page)
    scale = dim ** -0.5
    _close(r.run(hs, scale, window), r.expected(scale, window), scale)


@pytest.mark.parametrize("hq,long", [(2, 1), (40, 1), (2, 70)])
def test_attention_of_4096_requests(hq, long):
    """The most requests there may be, in the few-row kernel and in the chunk kernel (40 query
    heads of one kv head; 70 tokens); a third of them has no new token."""
    rng = np.random.default_rng(hq + long)
    cached = [int(x) for x in rng.integers(0, 20, 4096)]
    new = [int(x) for x in rng.integers(0, 3, 4096).clip(0, 1)]
    new[0], new[4095], new[2000] = 1, 1, long
    r = _kv8.Requests(hq, cached, new, hq, 1, 64, 16)
    _close(r.run(hs, 0.2), r.expected(0.2), 0.2)


@pytest.mark.parametrize("hq,hkv,dim", [(32, 8, 128), (24, 24, 64), (16, 2, 64)])
@pytest.mark.parametrize("bound", [None, 600])
def test_prompts_and_single_tokens_in_one_call(hq, hkv, dim, bound):
    """A step as the plan makes it: decoding requests, prompts, a request that waits; max_new
    is the step's own or a bound."""
    cached = [200, 0, 77, 1000, 0, 31, 64, 5, 0, 512]
    new = [1, 300, 1, 1, 7, 0, 1, 130, 1, 1]
    r = _kv8.Requests(hq, cached, new, hq, hkv, dim, 32)
    scale = dim ** -0.5
    _close(r.run(hs, scale, max_new=bound), r.expected(scale), scale)


@pytest.mark.parametrize("n,hkv,most", [(1, 1, 640), (1, 2, 1024), (1, 2, 1025), (5, 3, 600), (5, 3, 641), (31, 2, 300), (32, 4, 500), (32, 5, 200),
                                        (32, 2, 1000), (33, 2, 500), (32, 10, 90), (140, 1, 300)])
@pytest.mark.parametrize("group,new,dim", [(4, 1, 128), (16, 1, 64), (3, 6, 128), (12, 2, 64)])
def test_short_items_of_few_requests(n, hkv, most, group, new, dim):
    """Items that a CTA takes whole and such that are cut, at the lengths, numbers and tables at which
    one turns into the other; requests without rows, without keys and without pages among them."""
    rng = np.random.default_rng(n * most + group)
    cached = [int(x) for x in rng.integers(0, most, n)]
    cached[n // 2] = most - new
    fresh = [new if i == n // 2 or x > 0.2 else 0 for i, x in enumerate(rng.random(n))]
    r = _kv8.Requests(n + most, cached, fresh, hkv * group, hkv, dim, 64)
    out = r.run(hs, 0.1)
    _close(out, r.expected(0.1), 0.1)
    _close(r.run(hs, 0.1, max_new=1), r.expected(0.1), 0.1)   # (several row tiles a request)
    wide = torch.cat((torch.from_numpy(r.table), torch.full((n, 40), -1, dtype=torch.int32)), 1).cuda()
    _close(r.run(hs, 0.1, table=wide), r.expected(0.1), 0.1)


@pytest.mark.parametrize("n,hkv,most,window", [(32, 4, 384, 0), (32, 4, 385, 0), (33, 3, 768, 0), (33, 3, 769, 0), (24, 2, 2048, 0), (24, 2, 2049, 0),
                                               (25, 2, 1000, 0), (24, 2, 3000, 500), (150, 1, 700, 0), (4, 2, 5000, 333)])
@pytest.mark.parametrize("group,new,dim", [(4, 16, 128), (11, 3, 64), (13, 5, 128)])
def test_rows_of_short_items(n, hkv, most, window, group, new, dim):
    """33 to 65 rows a request, at the numbers, widths and windows at which they go from one kernel to the other;
    requests without rows among them, and a wide table that holds the same."""
    rng = np.random.default_rng(n * most + group)
    cached = [int(x) for x in rng.integers(0, most - new + 1, n)]
    cached[n // 2] = most - new
    fresh = [new if i == n // 2 or x > 0.2 else 0 for i, x in enumerate(rng.random(n))]
    r = _kv8.Requests(n + most, cached, fresh, hkv * group, hkv, dim, 16)
    ref = r.expected(0.1, window)
    _close(r.run(hs, 0.1, window), ref, 0.1)
    wide = torch.cat((torch.from_numpy(r.table), torch.full((n, 300), -1, dtype=torch.int32)), 1).cuda()
    _close(r.run(hs, 0.1, window, table=wide), ref, 0.1)


@pytest.mark.parametrize("n", [32, 33, 64, 100, 127, 128, 129, 300])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_of_many_requests(n, new):
    """The division of the work over one to four requests a lane and over more, some
    requests without new tokens, some with many."""
    rng = np.random.default_rng(n)
    fresh = [int(x) for x in rng.integers(0, new + 1, n)]
    fresh[n // 2] = 70 if new > 1 else 1
    cached = [int(x) for x in rng.integers(0, 90, n)]
    r = _kv8.Requests(n, cached, fresh, 4, 2, 64, 16)
    _close(r.run(hs, 0.2), r.expected(0.2), 0.2)


@pytest.mark.parametrize("new", [1, 5, 100])
def test_attention_rows_and_pages_that_are_not_there(new):
    """Missing pages drop out of the softmax, a request of absent pages gives
    zeros, an empty request has no row, and more new tokens than the length
    (rows before position 0) give zeros."""
    r = _kv8.Requests(3, [150, 40, 0, 90], [new, new, 0, new], 8, 2, 128, 32)
    table = r.table.copy()
    table[0, 1], table[0, 3] = -1, r.n_pages + 5
    table[1, :] = -1
    present = [np.ones(n, bool) for n in r.len]
    present[0][32:64] = present[0][96:128] = False
    present[1][:] = False
    got = r.run(hs, 0.1, table=torch.from_numpy(table).cuda())
    ref = r.expected(0.1, present=present)
    assert not ref[r.starts[1]:r.starts[2]].any()
    _close(got, ref, 0.1)
    r.len[3] = new // 2                     # rows at negative positions
    r.k[3], r.v[3] = r.k[3][:new // 2], r.v[3][:new // 2]
    _close(r.run(hs, 0.1), r.expected(0.1), 0.1)


@pytest.mark.parametrize("window", [(1 << 31) - 1, 1 << 30])
@pytest.mark.parametrize("new,dim", [(3, 128), (5, 64), (100, 128)])
def test_windows_of_any_size_and_rows_before_position_zero(new, dim, window):
    """A window past every length hides nothing, in a row tile that holds rows at
    negative positions too."""
    r = _kv8.Requests(4, [0, 70], [new, new], 8, 2, dim, 32)
    r.len[0] = new // 2
    r.k[0], r.v[0] = r.k[0][:new // 2], r.v[0][:new // 2]
    _close(r.run(hs, 0.1, window), r.expected(0.1), 0.1)


@pytest.mark.parametrize("new", [1, 40])
def test_contexts_past_two_to_the_thirty_without_a_window(new):
    """2^30 + 2^16 cached tokens, all in two pages: the oldest 2^16 tokens stand in
    one, whose keys lie nearer to the queries by as much as the others are more."""
    page, dim, old = 64, 64, 1 << 10
    length = (1 << 30) + (1 << 16) + 7
    rng = np.random.default_rng(12)
    q = _kv4.bf16(rng, (new, 1, dim))
    u = q.double().numpy()[:, 0].mean(0)
    u *= 1 / np.abs(u).max()
    q = torch.from_numpy(u[None, None] + rng.normal(0, 0.02, (new, 1, dim))).bfloat16()
    scale, k, v = 0.125, rng.normal(0, 0.2, (2 * page, 1, dim)), rng.normal(0, 1, (2 * page, 1, dim))
    k[:page, 0] += u * (14 * np.log(2) / scale / (u @ u))
    v[:page] += 2
    v[page:] -= 2
    k, v = (torch.from_numpy(x.astype(np.float32)).bfloat16() for x in (k, v))
    pool, c = _cache(2, page, 1, dim)
    slots = torch.arange(2 * page, device="cuda")
    hs.hs_kv8_append(c, k.cuda(), v.cuda(), slots, 2 * page)
    table = torch.ones((1, -(-length // page)), dtype=torch.int32, device="cuda")
    table[0, :old] = 0
    out = torch.empty_like(q, device="cuda")
    ws = torch.zeros(hs.hs_kv8_attention_workspace_size(c, 1, 1), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    hs.hs_kv8_attention(c, q.cuda(), i32([0, new]), i32([length]), table, 1, new, scale, 0, out, ws)
    torch.cuda.synchronize()
    assert hs.hs_device_status() == hs.HS_OK
    kk, vv, qq = _kv8.values(k.float().numpy())[:, 0], _kv8.values(v.float().numpy())[:, 0], q.double().numpy()[:, 0]
    ref = np.zeros((new, 1, dim))
    for i in range(new):
        seen = length - new + i + 1
        pages, rest = divmod(seen, page)
        times = np.concatenate((np.full(page, old), pages - old + (np.arange(page) < rest))).astype(float)
        s = kk @ qq[i] * scale
        e = times * np.exp(s - s.max())
        assert 0.2 < e[:page].sum() / e.sum() < 0.8
        ref[i, 0] = e / e.sum() @ vv
    # roundings as in _close, and 2^30 / 16 / 152 products added in turn, each sum cut off at 2^-23 of it at worst
    bound = np.abs(ref) * 2.0 ** -8 + 6 * (2.0 ** -11 * 2 + (1 << 30) / 16 / 152 * 2.0 ** -23)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.parametrize("new", [1, 3, 70])
def test_nan_in_hidden_places_does_not_spread(new):
    """NaN keys and values behind the causal border or before the window reach
    only the rows that see them."""
    def edit(i, k, v):
        n = len(k)
        k[n - 1], v[n - 1] = np.nan, np.inf      # the newest token's own
        k[2], v[2] = np.nan, np.nan              # far before the window
    r = _kv8.Requests(11, [200], [new], 4, 2, 128, 16, edit=edit)
    got = r.run(hs, 0.1, window=100).float().cpu().numpy()
    assert np.isnan(got[-1]).all()
    if new > 1:
        ref = r.expected(0.1, 100)
        _close(torch.from_numpy(got[:-1]), ref[:-1], 0.1)


@pytest.mark.parametrize("new,hq,dim", [(3, 4, 128), (3, 2, 64), (7, 8, 128), (20, 4, 64), (10, 4, 64), (16, 8, 64), (70, 4, 128)])
@pytest.mark.parametrize("window", [0, 90])
def test_a_nan_value_that_some_rows_see_and_some_do_not(new, hq, dim, window):
    """NaN in the values of one new token (half of its channels where there are 128) and of one
    token at the window's border: each row is NaN in those channels if it sees the token,
    and what it is without them if not."""
    where = 200 - new + new // 2

    def edit(i, k, v):
        v[where, 0, dim - 64:] = np.nan
        v[where - 91, 1, :64] = np.inf
    r = _kv8.Requests(17, [200 - new], [new], hq, 2, dim, 16, edit=edit)
    got = r.run(hs, 0.1, window).float().cpu().double().numpy()
    r.v[0] = np.nan_to_num(r.v[0])
    ref = r.expected(0.1, window)
    for i in range(new):
        p = 200 - new + i
        nan = np.zeros((hq, dim), bool)
        if p >= where:
            nan[:hq // 2, dim - 64:] = True
        if not window or p - window < where - 91:
            nan[hq // 2:, :64] = True
        assert np.array_equal(np.isnan(got[i]), nan), i
        got[i][nan] = ref[i][nan] = 0
    _close(torch.from_numpy(got), ref, 0.1)


@pytest.mark.parametrize("new", [1, 3, 70])
@pytest.mark.parametrize("far", [0, 40])
@pytest.mark.parametrize("where", [3, 199])
def test_a_visible_nan_value_reaches_its_rows_however_unlikely_its_key(new, far, where):
    """A value is NaN, in a step that all rows see whole or in the one where the rows'
    borders begin; with far > 0 its key's probability vanishes in fp32.  Every row sees
    it, and is NaN in its 64 channels and in them alone."""
    def edit(i, k, v):
        k[:] = np.abs(k)
        if far:
            k[where] = -far
        v[where, :, 64:] = np.nan
    r = _kv8.Requests(13, [200], [new], 4, 2, 128, 16, edit=edit)
    r.q = r.q.abs()
    got = r.run(hs, 0.1).float().cpu().double().numpy()
    assert np.isnan(got[..., 64:]).all()
    r.v[0] = np.nan_to_num(r.v[0])
    _close(torch.from_numpy(got[..., :64]), r.expected(0.1)[..., :64], 0.1)


@pytest.mark.parametrize("k_size,v_size,q_size", [(30., 1., 1.), (1., 300., 1.), (1., 1e-4, 1.), (1e-3, 1., 1e4), (1., 1., 1e-20),
                                                  (9000., 9000., 1e-4)])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_attention_sizes_of_values(k_size, v_size, q_size, new):
    """Peaked softmax, large and small values, large and tiny queries: the error
    stays relative to the values' size."""
    r = _kv8.Requests(5, [300], [new], 8, 2, 128, 64, k_size=k_size, v_size=v_size)
    r.q = (r.q.float() * q_size).bfloat16()
    ref = r.expected(0.05)
    got = r.run(hs, 0.05).float().cpu().double().numpy()
    # fp32 sums of scores lose 8 steps' 2^-23 of the products' sizes, whose sum is 128 * |q||k| at most
    err_s = 0.05 * 128 * 9 * k_size * q_size * 8 * 2.0 ** -23
    bound = 2.0 ** -8 * np.abs(ref) + np.abs(r.v[0]).max() * (2.0 ** -11 + 2 * err_s + 2.0 ** -20)
    assert (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_blocks_of_very_different_scales(new, dim):
    """Scales from one end of their range to the other among the keys and among the values, large
    values first, last and between: the output's error is that of the rounded
    probabilities, by the size of the values that carry weight."""
    size = 2.0 ** np.repeat([0, 6, -12, 3, 11, -14, 1, 8, -20, 0, 5, 0, -3], 16)[:200, None, None]

    def edit(i, k, v):
        v *= size[:len(v)]
        k *= 2.0 ** np.repeat(np.arange(13) % 5 - 3, 16)[:len(k), None, None]
    r = _kv8.Requests(16, [200 - new], [new], 8, 2, dim, 16, edit=edit)
    ref = r.expected(0.1)
    got = r.run(hs, 0.1).float().cpu().double().numpy()
    # as in _close, with max|v| * p of each key in place of the mean's bound: sum_j p_j |v_j| 2^-11, and for
    # single tokens the probabilities times 2^(e - largest e) below fp16's normal range, 2^-31 of the largest
    wide = _kv4.attention(r.q.double().numpy(), r.k[0], np.abs(r.v[0]), new, 200, 0.1)
    bound = 2.0 ** -8 * np.abs(ref) + wide * (2.0 ** -11 + 2.0 ** -12) + np.abs(r.v[0]).max() * 200 * 2.0 ** -31
    assert (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("spike", [0, 1, 77])
def test_attention_query_with_one_large_channel(new, spike):
    """The queries' common power of two follows their largest channel wherever it stands."""
    r = _kv8.Requests(6, [200], [new], 8, 2, 128, 64)
    q = r.q.float() * 0.01
    q[:, :, spike] = 300.0
    q[:, :, (spike + 2) % 128] = -0.03
    r.q = q.bfloat16()
    scale = 0.003  # scores of a few units
    bound = 2.0 ** -8 + 6.5 * (2.0 ** -11 + 2 * 300 * 6.5 * scale * 8 * 2.0 ** -23)
    ref = r.expected(scale)
    assert (np.abs(r.run(hs, scale).float().cpu().double().numpy() - ref) <= bound * np.maximum(1, np.abs(ref))).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 7, 12, 40])
def test_a_query_row_that_is_no_number_leaves_its_neighbours_alone(new, dim):
    """Of each kv head's four query heads one holds a NaN, one an infinity, the
    others values of about 20 and 300 (past 2^16 under a common scale of 1):
    the first two give NaN, the others what they give alone."""
    r = _kv8.Requests(8, [200], [new], 8, 2, dim, 32)
    kind = np.arange(8) % 4
    q = r.q.float() * torch.from_numpy(np.array([1., 1., 20., 300.], np.float32)[kind])[None, :, None]
    r.q = q.bfloat16()
    scale = 0.003
    ref = r.expected(scale)
    q[:, kind == 0, 5] = float("nan")
    q[:, kind == 1, 6] = float("inf")
    q[::2, kind == 1, 6] = -float("inf")
    r.q = q.bfloat16()
    got = r.run(hs, scale).float().cpu().double().numpy()
    assert np.isnan(got[:, kind < 2]).all()
    # as in test_attention_sizes_of_values, row by row
    err_s = scale * dim * 9 * np.array([20., 300.])[kind[kind > 1] - 2][None, :, None] * 8 * 2.0 ** -23
    bound = 2.0 ** -8 * np.abs(ref[:, kind > 1]) + 6.5 * (2.0 ** -11 + 2 * err_s + 2.0 ** -20)
    assert (np.abs(got - ref)[:, kind > 1] <= bound).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 7, 12, 40])
def test_query_rows_of_very_different_sizes(new, dim):
    """Rows 2^30 times smaller than their neighbours keep all their bits: their
    scores, of a few units at this scale, are those that they have alone."""
    r = _kv8.Requests(9, [200], [new], 8, 2, dim, 32)
    small = np.arange(8) % 4 > 1
    size = np.where(small, 2.0 ** -30, 1.0).astype(np.float32)
    r.q = (r.q.float() * torch.from_numpy(size)[None, :, None]).bfloat16()
    scale = 0.09 * 2.0 ** 30
    ref = r.expected(scale)
    got = r.run(hs, scale).float().cpu().double().numpy()
    assert np.isfinite(got).all()
    err_s = 0.09 * dim * 9 * 8 * 2.0 ** -23  # of the small rows; the others' softmax is one key's
    bound = 2.0 ** -8 * np.abs(ref[:, small]) + 6.5 * (2.0 ** -11 + 2 * err_s + 2.0 ** -20)
    assert (np.abs(got - ref)[:, small] <= bound).all()


@pytest.mark.parametrize("scale", [1e3, 1e30])
@pytest.mark.parametrize("sign", [0, -1])
@pytest.mark.parametrize("new,hq,dim", [(1, 2, 64), (1, 8, 128), (3, 8, 128), (7, 8, 64), (12, 8, 128), (40, 8, 128), (40, 8, 64)])
def test_scores_far_past_the_exponents_range(scale, sign, new, hq, dim):
    """Scores of 1e9 and 1e36 units, of both signs or all negative: the softmax is
    that of one key, and the output its value, wherever no other key comes near it."""
    def edit(i, k, v):
        if sign:
            k[:] = -np.abs(k)
    r = _kv8.Requests(10, [500], [new], hq, 2, dim, 16, k_size=30.0, edit=edit)
    q = r.q.float() * 1e4
    r.q = (q.abs() if sign else q).bfloat16()
    got = r.run(hs, scale).float().cpu().double().numpy()
    assert np.isfinite(got).all()
    q, seen = r.q.double().numpy(), 0
    for i in range(new):
        n = r.len[0] - new + i + 1
        for h in range(hq):
            k, v = r.k[0][:n, h // (hq // 2)], r.v[0][:n, h // (hq // 2)]
            s = k @ q[i, h]
            # fp32 sums (2^-20 of the products' sizes at most), scores levelled to 2^-20 of the largest
            err = (np.abs(k) @ np.abs(q[i, h])).max() * (2.0 ** -20 + 2.0 ** -20)
            order = np.argsort(s)
            if s[order[-1]] - s[order[-2]] <= 2 * err:
                continue
            seen += 1
            # the value and its rounding to bf16, beside the probability's to fp16
            top = v[order[-1]]
            assert (np.abs(got[i, h] - top) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) * np.abs(top)).all()
    assert seen >= new * hq // 3


@pytest.mark.parametrize("scale,q_size", [(1e-30, 1e-20), (1e-38, 1e-30), (1e30, 3e4), (1e30, 1e5)])
@pytest.mark.parametrize("new", [1, 3, 12, 40])
def test_scales_at_the_ends_of_their_range(scale, q_size, new):
    """Scores of nothing: the mean of the visible values, hidden keys and absent rows
    apart.  Scores of -10^36 and more, one key far above the others: its value."""
    def edit(i, k, v):
        k[:] = -10 - np.abs(k)
        k[17] = -0.5
    r = _kv8.Requests(14, [90, 30], [new, 2], 8, 2, 128, 32, edit=edit)
    r.q = ((r.q.float().abs() + 0.5) * q_size).bfloat16()
    ref = r.expected(scale)
    got = r.run(hs, scale).float().cpu().double().numpy()
    # probabilities rounded to fp16 (2^-11) before their product with values of up to 6.5
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + 6.5 * (2.0 ** -11 + 2.0 ** -20)).all()


@pytest.mark.parametrize("exponent", [-95, 105, 113, 120])
@pytest.mark.parametrize("new,dim", [(1, 128), (3, 64), (12, 128), (40, 128), (40, 64)])
def test_queries_of_any_exponent(exponent, new, dim):
    """Queries of 2^exponent with a scale that makes their scores the usual ones."""
    r = _kv8.Requests(15, [300, 20], [new, 1], 8, 2, dim, 64)
    r.q = (r.q.float() * 2.0 ** exponent).bfloat16()
    scale = dim ** -0.5 * 2.0 ** -exponent
    _close(r.run(hs, scale), r.expected(scale), scale)


def test_attention_strides_streams_and_reuse_of_the_workspace():
    r = _kv8.Requests(21, [700, 90], [2, 2], 16, 4, 128, 64)
    ref = r.expected(0.09)
    wide_q = torch.full((4, 19, 136), float("nan"), device="cuda").bfloat16()
    wide_o = torch.full((4, 17, 160), 7.0, device="cuda").bfloat16()
    wide_q[:, 2:18, :128] = r.q.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = wide_o[:, :16, :128]
    r.run(hs, 0.09, q=wide_q[:, 2:18, :128], out=out, stream=s)
    _close(out, ref, 0.09)
    assert (wide_o[:, 16] == 7).all() and (wide_o[:, :, 128:] == 7).all()
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    a = r.run(hs, 0.09, ws=ws)
    big = _kv8.Requests(22, [3000], [1], 32, 2, 128, 64)
    b0 = big.run(hs, 0.09, ws=ws)
    b1 = big.run(hs, 0.09, ws=ws)
    assert torch.equal(a, r.run(hs, 0.09, ws=ws)) and torch.equal(b0, b1)  # bit for bit, call after call
    _close(b0, big.expected(0.09), 0.09)


@pytest.mark.parametrize("ctx,new,hq,hkv,dim", [([900] * 5, [200] * 5, 16, 4, 128), ([1500, 40, 700], [1, 130, 333], 8, 2, 64),
                                                ([1500] * 24, [1] * 24, 32, 8, 128), ([2000] * 9, [3] * 9, 32, 2, 128),
                                                # one row tile: joins in shared memory (few pieces), from memory (many)
                                                ([1500] * 14, [3] * 14, 32, 2, 128), ([3000] * 6, [40] * 6, 4, 4, 64),
                                                ([700, 0, 65], [40, 128, 1], 8, 8, 128), ([20000], [9], 16, 4, 64),
                                                # sixteen rows on eight warps: two rounds, one round, items that a CTA begins and ends
                                                ([40000], [1], 32, 2, 128), ([9000], [4], 8, 2, 64), ([5000, 30], [1, 1], 16, 1, 128),
                                                ([15000, 200, 9000], [2, 1, 2], 16, 2, 128), ([3000] * 7, [1] * 7, 32, 2, 64)])
def test_joined_pieces_do_not_depend_on_who_comes_last(ctx, new, hq, hkv, dim):
    """Work on another stream delays some CTAs, so that an item's pieces arrive in other orders."""
    r = _kv8.Requests(77, ctx, new, hq, hkv, dim, 64)
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    first = r.run(hs, 0.09, ws=ws)
    _close(first, r.expected(0.09), 0.09)
    side, a = torch.cuda.Stream(), torch.ones(2048, 2048, device="cuda")
    for i in range(20):
        if i % 2:
            with torch.cuda.stream(side):
                a @ a
        assert torch.equal(first, r.run(hs, 0.09, ws=ws))
    torch.cuda.synchronize()


def test_rows_past_the_last_request_are_not_written_and_max_new_only_chooses():
    r = _kv8.Requests(31, [40, 500], [3, 2], 8, 2, 128, 64)
    q = torch.cat((r.q, torch.full((6, 8, 128), float("nan")).bfloat16())).cuda()
    out = torch.full_like(q, 5.0)
    got = r.run(hs, 0.1, q=q, out=out)
    assert (got[5:] == 5).all()
    ref = r.expected(0.1)
    _close(got[:5], ref, 0.1)
    for m in (1, 9, 4000):
        _close(r.run(hs, 0.1, max_new=m), ref, 0.1)


def test_step_in_a_captured_graph():
    """plan, append and attention of one decode step, captured once and replayed
    with other lengths: the host knows none of them."""
    page, hkv, hq, dim, n, width = 16, 2, 8, 64, 5, 12
    rng = np.random.default_rng(77)
    n_pages = n * width
    pool, c = _cache(n_pages, page, hkv, dim)
    dev = dict(device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, **dev)  # noqa: E731
    cached, new, table = i32(n), i32(n), torch.full((n, width), -1, dtype=torch.int32, **dev)
    ring = torch.from_numpy(rng.permutation(n_pages).astype(np.int32)).cuda()
    cin = torch.tensor([0, n_pages], dtype=torch.int64, **dev)
    cout, short, seq, qs, pos = torch.zeros_like(cin), i32(1), i32(n), i32(n + 1), i32(32)
    slot = torch.zeros(32, dtype=torch.int64, **dev)
    k, v = (torch.zeros((32, hkv, dim), **dev).bfloat16() for _ in range(2))
    q = torch.zeros((32, hq, dim), **dev).bfloat16()
    out = torch.zeros_like(q)
    ws = torch.zeros(hs.hs_kv8_attention_workspace_size(c, n, hq), dtype=torch.uint8, **dev)

    def step():
        hs.hs_kv4_plan(cached, new, n, page, n_pages, table, width, ring, cin, 32, table, seq, qs, slot, pos, cout, short)
        hs.hs_kv8_append(c, k, v, slot, 32)
        hs.hs_kv8_attention(c, q, qs, seq, table, n, 32, 0.2, 0, out, ws)
        cin.copy_(cout)
        cached.copy_(seq)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()  # nothing new: attributes are set, nothing changes
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    pool_np, length = np.full(pool.shape, 0xFF, np.uint8), [0] * n
    for turn in range(12):
        fresh = rng.integers(0, 7, n)
        if turn == 6:
            fresh[2] = -1
        total = int(fresh.clip(0).sum())
        kk, vv, qq = (_kv4.bf16(rng, (32, h, dim)) for h in (hkv, hkv, hq))
        k.copy_(kk), v.copy_(vv), q.copy_(qq)
        new.copy_(torch.from_numpy(fresh.astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        assert int(short) == 0 and int(qs[-1]) == total
        at, refs = 0, []
        for i, f in enumerate(fresh):
            if f < 0:
                length[i] = 0
                continue
            length[i] += int(f)
            row, j = table[i].cpu().numpy().astype(np.int64), np.arange(length[i])
            slots = row[j // page] * page + j % page
            _kv8.append(pool_np, page, dim, slots[length[i] - f:], kk[at:at + f].float().numpy(), vv[at:at + f].float().numpy())
            refs.append(_kv4.attention(qq[at:at + f].double().numpy(), *_kv8.read(pool_np, page, dim, slots), int(f), length[i], 0.2))
            at += f
        _close(out[:total], np.concatenate(refs), 0.2)
    free = int(cin[1] - cin[0])
    rows = table.cpu().numpy()
    assert free + int((rows >= 0).sum()) == n_pages


def test_a_workspace_shared_with_the_4_bit_cache():
    """Both kinds of attention on one workspace, in turn."""
    a, b = _kv8.Requests(41, [900, 3000], [1, 2], 16, 2, 128, 64), _kv4.Requests(42, [2500, 70], [1, 60], 8, 2, 128, 32)
    need = max(hs.hs_kv8_attention_workspace_size(hs.make_kv8_cache(None, 1, 64, 2, 128), 2, 16),
               hs.hs_kv4_attention_workspace_size(hs.make_kv4_cache(None, 1, 32, 2, 128), 2, 8))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = a.run(hs, 0.09, ws=ws), b.run(hs, 0.09, ws=ws)
    _close(first[0], a.expected(0.09), 0.09)
    for _ in range(3):
        assert torch.equal(a.run(hs, 0.09, ws=ws), first[0]) and torch.equal(b.run(hs, 0.09, ws=ws), first[1])


def test_requests_that_fork_decode_are_cut_back_and_move():
    """Samples of a prompt over the 8-bit cache, as a server runs them: plan, append, attention,
    fork, release and compact, mirrored byte by byte; every attention against 64 bits."""
    page, hkv, hq, dim, n_pages, width, rows = 32, 2, 8, 128, 40, 6, 6
    rng = np.random.default_rng(43)
    pool, c = _cache(n_pages, page, hkv, dim)
    mirror = np.full(pool.shape, 0xFF, np.uint8)
    dev = dict(device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, **dev)  # noqa: E731
    table, ring, shared = torch.full((rows, width), -1, dtype=torch.int32, **dev), torch.from_numpy(rng.permutation(n_pages)).int().cuda(), i32(n_pages)
    length, out_len, seq, qs, short, src, dst = i32(rows), i32(rows), i32(rows), i32(rows + 1), i32(1), i32(n_pages), i32(n_pages)
    counters, cout, slot = torch.tensor([0, n_pages], **dev), torch.zeros(2, dtype=torch.int64, **dev), torch.zeros(256, dtype=torch.int64, **dev)
    ws = torch.zeros(hs.hs_kv8_attention_workspace_size(c, rows, hq), dtype=torch.uint8, **dev)
    pages_ws = torch.zeros(hs.hs_kv_pages_workspace_size(n_pages), dtype=torch.uint8, **dev)
    size = hkv * _kv8.record_bytes(page, dim)

    def done(new_length):
        assert int(short) == 0
        length.copy_(new_length)
        counters.copy_(cout)

    def slots_of(i):
        j = np.arange(int(length[i]))
        return table[i].cpu().numpy().astype(np.int64)[j // page] * page + j % page

    def step(new):
        t = sum(new)
        hs.hs_kv4_plan(length, torch.tensor(new, dtype=torch.int32, **dev), rows, page, n_pages, table, width, ring, counters, 256, table, seq,
                       qs, slot, None, cout, short)
        size = 2.0 ** int(rng.integers(-3, 4))
        k, v, q = _kv4.bf16(rng, (t, hkv, dim), size), _kv4.bf16(rng, (t, hkv, dim)), _kv4.bf16(rng, (t, hq, dim), 1 / size)
        hs.hs_kv8_append(c, k.cuda(), v.cuda(), slot, t)
        out = torch.empty((t, hq, dim), dtype=torch.bfloat16, **dev)
        hs.hs_kv8_attention(c, q.cuda(), qs, seq, table, rows, max(new), 0.09, 0, out, ws)
        done(seq)
        _kv8.append(mirror, page, dim, slot[:t].cpu().numpy(), k.float().numpy(), v.float().numpy())
        at = 0
        for i, m in enumerate(new):
            if m:
                kk, vv = _kv8.read(mirror, page, dim, slots_of(i))
                _close(out[at:at + m], _kv4.attention(q[at:at + m].double().numpy(), kk, vv, m, len(kk), 0.09), 0.09)
            at += m
        _same_bytes(pool, mirror)

    def copied():
        hs.hs_kv_copy_pages([pool], size, n_pages, src, dst, n_pages)
        for x, y in zip(src.tolist(), dst.tolist()):
            if x >= 0:
                mirror[y] = mirror[x]
        _same_bytes(pool, mirror)

    def fork(p, ch, m):
        src.fill_(-1), dst.fill_(-1)
        a = [torch.tensor(x, dtype=torch.int32, **dev) for x in (p, ch, m)]
        hs.hs_kv_fork(*a, len(p), length, rows, page, n_pages, table, width, shared, ring, counters, table, out_len, src, dst, cout, short)
        done(out_len)
        copied()

    def keep(m):
        hs.hs_kv_release(length, torch.tensor(m, dtype=torch.int32, **dev), rows, page, n_pages, table, width, shared, ring, counters, table,
                         out_len, cout, pages_ws)
        done(out_len)
    step([45, 0, 0, 70, 0, 0])
    fork([0, 0, 3], [1, 2, 4], [45, 40, 64])
    for _ in range(3):
        step([1, 1, 1, 1, 1, 0])
    step([3, 2, 0, 0, 40, 0])               # drafts and a chunk
    keep([46, 1 << 30, 1 << 30, 1 << 30, 65, 0])   # drafts refused, a row cut back in a page of its own
    step([1, 1, 2, 0, 3, 0])
    keep([0, 1 << 30, 1 << 30, 0, 1 << 30, 0])     # the prompts end, what was forked off lives on
    hs.hs_kv_compact(length, rows, page, n_pages, table, width, shared, ring, counters, n_pages, table, shared, src, dst, cout, short, pages_ws)
    done(length)
    copied()
    fork([1], [0], [33])
    step([1, 1, 1, 90, 1, 0])
    keep([0] * rows)
    assert not shared.any() and int(counters[1] - counters[0]) == n_pages and hs.hs_device_status() == hs.HS_OK


def test_two_calls_at_once():
    """Appends, reads and attention on two streams, a workspace each: what each gives alone."""
    a, b = _kv8.Requests(44, [4000] * 6, [1] * 6, 32, 2, 128, 64), _kv8.Requests(45, [300, 2000], [200, 90], 8, 2, 64, 16)
    streams, ws = [torch.cuda.Stream() for _ in range(2)], []
    made = []
    for r in (a, b):
        c = hs.make_kv8_cache(None, r.n_pages, r.page, r.hkv, r.dim)
        ws.append(torch.zeros(hs.hs_kv8_attention_workspace_size(c, len(r.len), r.hq), dtype=torch.uint8, device="cuda"))
        first = r.run(hs, 0.09, ws=ws[-1])
        _close(first, r.expected(0.09), 0.09)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        made.append((hs.make_kv8_cache(r.pool, r.n_pages, r.page, r.hkv, r.dim), r.q.cuda(), i32(r.starts.tolist()), i32(r.len),
                     torch.from_numpy(r.table).cuda(), len(r.len), max(r.new), torch.empty_like(first), first))
    torch.cuda.synchronize()
    for turn in range(10):
        for s, w, (c, q, qs, ls, table, n, most, out, first) in zip(streams, ws, made):
            hs.hs_kv8_attention(c, q, qs, ls, table, n, most, 0.09, 0, out, w, stream=s)
    torch.cuda.synchronize()
    assert hs.hs_device_status() == hs.HS_OK
    for m in made:
        assert torch.equal(m[-1], m[-2])
