"""The 4-bit key/value cache on the GPU: plan, append, read and attention
against their 64-bit restatements (tests/_kv4.py)."""
import numpy as np
import pytest
import torch

import _kv4
from activation_sparse_moe_gb300 import hs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from activation_sparse_moe_gb300 import build
    build.build()
    hs.lib()


# ------------------------------------------------------------------ plan
def _plan(cached, new, page, n_pages, table, ring, counters, max_tokens, in_place=False):
    d = lambda a, t=torch.int32: torch.as_tensor(np.asarray(a)).to("cuda", t)  # noqa: E731
    n, w = table.shape
    tin, r = d(table).contiguous(), d(ring)
    tout = tin if in_place else torch.full_like(tin, -7)
    i32 = lambda m: torch.full((m,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    seq, qs, pos, short = i32(n), i32(n + 1), i32(max_tokens), i32(1)
    slot = torch.full((max_tokens,), -7, dtype=torch.int64, device="cuda")
    cout = torch.full((2,), -7, dtype=torch.int64, device="cuda")
    hs.hs_kv4_plan(d(cached), d(new), n, page, n_pages, tin, w, r, d(counters, torch.int64), max_tokens, tout, seq, qs,
                   slot, pos, cout, short)
    return {k: v.cpu().numpy() for k, v in dict(table=tout, ring=r, counters=cout, seq_len=seq, q_start=qs, slot=slot,
                                                position=pos, short=short).items()}


def _plan_case(seed, n, page, width, spare, head=None):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, width * page // 2, n)
    new = np.where(rng.random(n) < 0.5, 1, rng.integers(-1, max(2, width * page // 3), n)).clip(-1)
    new[rng.random(n) < 0.15] = -1
    cached[rng.random(n) < 0.1] = 0
    have = -(-cached // page)
    need = int(sum(max(0, -(-(c + x) // page) - h) for c, x, h in zip(cached, new, have) if x >= 0))
    n_pages = int(have.sum()) + max(need + spare, 1)
    perm = rng.permutation(n_pages)
    table = np.full((n, width), -1, np.int32)
    at = 0
    for i in range(n):
        table[i, :have[i]] = perm[at:at + have[i]]
        at += have[i]
    head = int(rng.integers(0, 1 << 40)) if head is None else head
    ring = np.full(n_pages, -1, np.int32)
    ring[(head + np.arange(n_pages - at)) % n_pages] = perm[at:]
    return cached, new, n_pages, table, ring, [head, head + n_pages - at]


@pytest.mark.parametrize("n,page,width,spare", [(1, 64, 3, 0), (2, 16, 1, 1), (8, 64, 64, 5), (33, 32, 9, 0), (300, 16, 70, 11),
                                                (4096, 16, 5, 3), (257, 64, 33, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(n, page, width, spare, in_place):
    cached, new, n_pages, table, ring, counters = _plan_case(n + page, n, page, width, spare)
    tokens = int(new.clip(0).sum())
    cap = tokens + 13
    ref = _kv4.plan(cached, new, page, n_pages, table, ring, counters, cap)
    got = _plan(cached, new, page, n_pages, table, ring, counters, cap, in_place)
    for name in ref:
        assert np.array_equal(np.atleast_1d(got[name]), np.atleast_1d(ref[name])), name


@pytest.mark.parametrize("why", ["pages", "width", "tokens"])
def test_plan_refuses_a_step_as_a_whole(why):
    cached, new, n_pages, table, ring, counters = _plan_case(5, 40, 16, 20, 4)
    cached, new = cached.copy(), new.copy()
    new[3], new[7], new[9] = -1, 30, 30
    cap = int(new.clip(0).sum()) + 5
    if why == "pages":
        counters = [counters[0], counters[0] + 2]
    elif why == "width":
        cached[11], new[11] = 0, 21 * 16
        cap += 21 * 16
    else:
        cap = int(new.clip(0).sum()) - 1
    ref = _kv4.plan(cached, new, 16, n_pages, table, ring, counters, cap)
    assert ref["short"] > 0 and ref["q_start"][-1] == 0
    got = _plan(cached, new, 16, n_pages, table, ring, counters, cap)
    for name in ref:
        assert np.array_equal(np.atleast_1d(got[name]), np.atleast_1d(ref[name])), name


# --------------------------------------------------------- append and read
def _cache(n_pages, page, hkv, dim):
    pool = torch.full((n_pages, hkv, _kv4.record_bytes(page, dim)), 0xFF, dtype=torch.uint8, device="cuda")
    c = hs.make_kv4_cache(pool, n_pages, page, hkv, dim)
    assert hs.hs_kv4_pool_bytes(c) == pool.numel()
    return pool, c


def _hard_rows(rng, t, h, d):
    """bf16 rows with what a quantiser meets: equal values, ties between codes,
    large and tiny ranges, signed zeros, infinities and NaN, fp16 overflow."""
    x = rng.normal(0, 1, (t, h, d)).astype(np.float32)
    x *= np.exp(rng.normal(0, 3, (t, h, 1))).astype(np.float32)
    flat = x.reshape(-1, 64)
    n = len(flat)
    kinds = [lambda g: g * 0 + 3.25, lambda g: g * 0, lambda g: np.where(np.arange(64) % 2, 0.0, -0.0),
             lambda g: np.arange(64) / 2 % 15.5, lambda g: g * 1e-6, lambda g: g * 1e5,
             lambda g: np.where(np.arange(64) == 5, np.inf, g), lambda g: np.where(np.arange(64) == 63, np.nan, g),
             lambda g: np.where(np.arange(64) == 0, -np.inf, g), lambda g: np.where(np.arange(64) == 9, 30000., g),
             lambda g: g * 1e-38]
    for i, f in enumerate(kinds):
        if i < n:
            flat[(i * 7) % n] = f(flat[(i * 7) % n])
    return torch.from_numpy(x).bfloat16()


@pytest.mark.parametrize("t,hkv,dim,page", [(1, 1, 64, 16), (1, 2, 128, 64), (3, 3, 128, 16), (37, 5, 64, 32), (200, 8, 128, 64),
                                            (1031, 2, 64, 64)])
def test_append_writes_the_definition_bit_for_bit_and_read_returns_it(t, hkv, dim, page):
    rng = np.random.default_rng(t * 7 + hkv)
    n_pages = -(-t // page) + 2
    pool, c = _cache(n_pages, page, hkv, dim)
    k, v = _hard_rows(rng, t, hkv, dim), _hard_rows(rng, t, hkv, dim)
    slots = rng.permutation(n_pages * page)[:t]
    # K and V from one fused buffer: other strides than the packed ones
    fused = torch.randn(t, 2 * hkv + 1, dim + 8).bfloat16().cuda()
    fused[:, :hkv, :dim], fused[:, hkv:2 * hkv, :dim] = k.cuda(), v.cuda()
    hs.hs_kv4_append(c, fused[:, :hkv, :dim], fused[:, hkv:2 * hkv, :dim], torch.from_numpy(slots).cuda(), t)
    want = np.full(pool.shape, 0xFF, np.uint8)
    _kv4.fill_pool(want, page, dim, slots, k.float().numpy(), v.float().numpy())
    half = page * dim // 2
    got = pool.cpu().numpy()
    assert np.array_equal(got[..., :2 * half], want[..., :2 * half])
    gp, wp = (np.ascontiguousarray(a[..., 2 * half:]).view(np.float16) for a in (got, want))
    assert np.array_equal(gp, wp, equal_nan=True)
    read = slots.copy()
    read[t // 2] = -1                      # no token there: zeros
    sl = torch.from_numpy(np.concatenate((read, [n_pages * page, -5]))).cuda()
    shape = (t + 2, hkv, dim)
    kb, vb = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kf, vf = (torch.empty(shape, dtype=torch.float32, device="cuda") for _ in range(2))
    hs.hs_kv4_read(c, sl, t + 2, kb, vb, kf, vf)
    for x, b, f in ((k, kb, kf), (v, vb, vf)):
        ref = np.concatenate((_kv4.values(x.float().numpy()), np.zeros((2, hkv, dim))))
        ref[t // 2] = 0
        # one fp32 rounding of scale * code + bias
        assert np.array_equal(f.cpu().numpy(), ref.astype(np.float32), equal_nan=True)
        assert torch.equal(b.cpu().view(torch.int16)[torch.isfinite(b.cpu())], f.cpu().bfloat16().view(torch.int16)[torch.isfinite(b.cpu())])
        assert torch.equal(torch.isnan(b), torch.isnan(f))


@pytest.mark.parametrize("t,hkv,dim,page", [(21, 33, 128, 16), (9, 65, 64, 32), (5, 256, 128, 16), (3, 129, 64, 16)])
def test_append_and_read_of_many_heads(t, hkv, dim, page):
    """More than 64 groups a row: several CTAs along it."""
    rng = np.random.default_rng(hkv)
    pool, c = _cache(4, page, hkv, dim)
    k, v = _hard_rows(rng, t, hkv, dim), _hard_rows(rng, t, hkv, dim)
    slots = rng.permutation(4 * page)[:t]
    sl = torch.from_numpy(slots).cuda()
    hs.hs_kv4_append(c, k.cuda(), v.cuda(), sl, t)
    want = np.full(pool.shape, 0xFF, np.uint8)
    _kv4.fill_pool(want, page, dim, slots, k.float().numpy(), v.float().numpy())
    half, got = page * dim // 2, pool.cpu().numpy()
    assert np.array_equal(got[..., :2 * half], want[..., :2 * half])
    gp, wp = (np.ascontiguousarray(a[..., 2 * half:]).view(np.float16) for a in (got, want))
    assert np.array_equal(gp, wp, equal_nan=True)
    kf, vf = (torch.empty((t, hkv, dim), dtype=torch.float32, device="cuda") for _ in range(2))
    vb = torch.empty((t, hkv, dim), dtype=torch.bfloat16, device="cuda")
    hs.hs_kv4_read(c, sl, t, k_f32=kf, v_f32=vf, v_bf16=vb)
    for x, f in ((k, kf), (v, vf)):
        assert np.array_equal(f.cpu().numpy(), _kv4.values(x.float().numpy()).astype(np.float32), equal_nan=True)
    assert torch.equal(vb.isnan(), vf.isnan()) and torch.equal(vb[~vb.isnan()], vf.bfloat16()[~vb.isnan()])


def test_append_of_a_slot_given_twice_touches_no_other():
    """What such a slot holds is undefined where its tokens differ; where they are
    equal it holds them, and every other slot holds its own token bit for bit."""
    page, hkv, dim, t = 16, 3, 128, 400
    rng = np.random.default_rng(5)
    pool, c = _cache(32, page, hkv, dim)
    k, v = _kv4.bf16(rng, (t, hkv, dim)), _kv4.bf16(rng, (t, hkv, dim))
    slots = rng.permutation(32 * page)[:t]
    slots[100:200] = slots[7]                       # 101 tokens of different values
    slots[200:250], k[200:250], v[200:250] = slots[8], k[8], v[8]
    hs.hs_kv4_append(c, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), t)
    keep = np.r_[0:7, 8:100, 250:t]
    want = np.full(pool.shape, 0xFF, np.uint8)
    _kv4.fill_pool(want, page, dim, slots[keep], k[keep].float().numpy(), v[keep].float().numpy())
    got = pool.cpu().numpy()
    p, o = divmod(int(slots[7]), page)
    for a in (got, want):
        half, pairs = page * dim // 2, page * dim // 16
        for x in (0, 1):
            a[p, :, x * half + o * (dim // 2):x * half + (o + 1) * (dim // 2)] = 0
            a[p, :, 2 * half + x * pairs + o * (dim // 16):2 * half + x * pairs + (o + 1) * (dim // 16)] = 0
    assert np.array_equal(got, want)


def test_append_skips_slots_outside_the_pool_and_zero_tokens():
    pool, c = _cache(3, 16, 2, 64)
    k = torch.full((4, 2, 64), float("nan"), device="cuda").bfloat16()
    hs.hs_kv4_append(c, k, k, torch.tensor([-1, 48, 1 << 40, -(1 << 62)], device="cuda"), 4)
    hs.hs_kv4_append(c, k, k, torch.zeros(4, dtype=torch.int64, device="cuda"), 0)
    torch.cuda.synchronize()
    assert (pool == 0xFF).all()


def test_pool_offsets_past_4_gigabytes():
    page, hkv, dim = 64, 8, 128
    n_pages = (5 << 30) // (hkv * _kv4.record_bytes(page, dim))
    pool, c = _cache(n_pages, page, hkv, dim)
    rng = np.random.default_rng(1)
    k, v = _kv4.bf16(rng, (70, hkv, dim)), _kv4.bf16(rng, (70, hkv, dim))
    pages = np.array([n_pages - 1, n_pages - 5])
    slots = pages[np.arange(70) // page].astype(np.int64) * page + np.arange(70) % page
    hs.hs_kv4_append(c, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), 70)
    kf = torch.empty((70, hkv, dim), dtype=torch.float32, device="cuda")
    hs.hs_kv4_read(c, torch.from_numpy(slots).cuda(), 70, k_f32=kf)
    assert np.array_equal(kf.cpu().numpy(), _kv4.values(k.float().numpy()).astype(np.float32))
    q = _kv4.bf16(rng, (1, hkv, dim))
    out = torch.empty_like(q, device="cuda")
    ws = torch.zeros(hs.hs_kv4_attention_workspace_size(c, 1, hkv), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    hs.hs_kv4_attention(c, q.cuda(), i32([0, 1]), i32([70]), i32(pages.reshape(1, 2)), 1, 1, 0.1, 0, out, ws)
    ref = _kv4.attention(q.double().numpy(), _kv4.values(k.float().numpy()), _kv4.values(v.float().numpy()), 1, 70, 0.1)
    _close(out, ref, 0.1)


# -------------------------------------------------------------- attention
def _close(out, ref, scale):
    """Bound of one output against the 64-bit one, in units of the row's size.

    The last rounding is half a bf16 step, 2^-8 of the value.  Before it, the
    probabilities are rounded to fp16 (2^-11 each; in chunks also keys and
    values, 2^-11 each of their size), the exponentials and fp32 sums add a few
    2^-22.  An output is a mean of values weighted by the probabilities, so the
    roundings of p and v move it by at most 2 * 2^-11 * max|v|, and those of k by
    2^-11 * |scale * q . k| <= 2^-11 * 32 here at most once for p and its sum
    (2 * 32 * 2^-11 * max|v| in the worst alignment, never seen; the mean over
    channels' random signs is 1/10 of it).  max|v| over a row's output is not
    known to the reader of the output, its root mean square is: for these
    normal values max|v| <= 6 and a row's outputs spread around sqrt(sum p^2)."""
    got = out.float().cpu().double().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    vmax = 6.0
    bound = np.abs(ref) * 2.0 ** -8 + vmax * 2.0 ** -11 * (2 + 6.4)
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
    r = _kv4.Requests(case, cached, new, hq, hkv, dim, page)
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
    r = _kv4.Requests(case + dim + page, [400, 0, 65], [new, new, min(new, 2)], hq, hkv, dim, page)
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
    r = _kv4.Requests(hq, cached, new, hq, 1, 64, 16)
    _close(r.run(hs, 0.2), r.expected(0.2), 0.2)


@pytest.mark.parametrize("hq,hkv,dim", [(32, 8, 128), (24, 24, 64), (16, 2, 64)])
@pytest.mark.parametrize("bound", [None, 600])
def test_prompts_and_single_tokens_in_one_call(hq, hkv, dim, bound):
    """A step as the plan makes it: decoding requests, prompts, a request that waits; max_new
    is the step's own or a bound."""
    cached = [200, 0, 77, 1000, 0, 31, 64, 5, 0, 512]
    new = [1, 300, 1, 1, 7, 0, 1, 130, 1, 1]
    r = _kv4.Requests(hq, cached, new, hq, hkv, dim, 32)
    scale = dim ** -0.5
    _close(r.run(hs, scale, max_new=bound), r.expected(scale), scale)


@pytest.mark.parametrize("n", [32, 33, 64, 100, 127, 128, 129, 300])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_of_many_requests(n, new):
    """The division of the work over one to four requests a lane and over more, some
    requests without new tokens, some with many."""
    rng = np.random.default_rng(n)
    fresh = [int(x) for x in rng.integers(0, new + 1, n)]
    fresh[n // 2] = 70 if new > 1 else 1
    cached = [int(x) for x in rng.integers(0, 90, n)]
    r = _kv4.Requests(n, cached, fresh, 4, 2, 64, 16)
    _close(r.run(hs, 0.2), r.expected(0.2), 0.2)


@pytest.mark.parametrize("new", [1, 5, 100])
def test_attention_rows_and_pages_that_are_not_there(new):
    """Missing pages drop out of the softmax, a request of absent pages gives
    zeros, an empty request has no row, and more new tokens than the length
    (rows before position 0) give zeros."""
    r = _kv4.Requests(3, [150, 40, 0, 90], [new, new, 0, new], 8, 2, 128, 32)
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
    r = _kv4.Requests(4, [0, 70], [new, new], 8, 2, dim, 32)
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
    hs.hs_kv4_append(c, k.cuda(), v.cuda(), slots, 2 * page)
    table = torch.ones((1, -(-length // page)), dtype=torch.int32, device="cuda")
    table[0, :old] = 0
    out = torch.empty_like(q, device="cuda")
    ws = torch.zeros(hs.hs_kv4_attention_workspace_size(c, 1, 1), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    hs.hs_kv4_attention(c, q.cuda(), i32([0, new]), i32([length]), table, 1, new, scale, 0, out, ws)
    torch.cuda.synchronize()
    assert hs.hs_device_status() == hs.HS_OK
    kk, vv, qq = _kv4.values(k.float().numpy())[:, 0], _kv4.values(v.float().numpy())[:, 0], q.double().numpy()[:, 0]
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
    bound = np.abs(ref) * 2.0 ** -8 + 6 * (2.0 ** -11 * 8.4 + (1 << 30) / 16 / 152 * 2.0 ** -23)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.parametrize("new", [1, 3, 70])
def test_nan_in_hidden_places_does_not_spread(new):
    """NaN keys and values behind the causal border or before the window reach
    only the rows that see them."""
    def edit(i, k, v):
        n = len(k)
        k[n - 1], v[n - 1] = np.nan, np.inf      # the newest token's own
        k[2], v[2] = np.nan, np.nan              # far before the window
    r = _kv4.Requests(11, [200], [new], 4, 2, 128, 16, edit=edit)
    got = r.run(hs, 0.1, window=100).float().cpu().numpy()
    assert np.isnan(got[-1]).all()
    if new > 1:
        ref = r.expected(0.1, 100)
        _close(torch.from_numpy(got[:-1]), ref[:-1], 0.1)


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
    r = _kv4.Requests(13, [200], [new], 4, 2, 128, 16, edit=edit)
    r.q = r.q.abs()
    got = r.run(hs, 0.1).float().cpu().double().numpy()
    assert np.isnan(got[..., 64:]).all()
    r.v[0] = np.nan_to_num(r.v[0])
    _close(torch.from_numpy(got[..., :64]), r.expected(0.1)[..., :64], 0.1)


@pytest.mark.parametrize("k_size,v_size,q_size", [(30., 1., 1.), (1., 300., 1.), (1., 1e-4, 1.), (1e-3, 1., 1e4), (1., 1., 1e-20)])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_sizes_of_values(k_size, v_size, q_size, new):
    """Peaked softmax, large and small values, large and tiny queries: the error
    stays relative to the values' size."""
    r = _kv4.Requests(5, [300], [new], 8, 2, 128, 64, k_size=k_size, v_size=v_size)
    r.q = (r.q.float() * q_size).bfloat16()
    ref = r.expected(0.05)
    got = r.run(hs, 0.05).float().cpu().double().numpy()
    # a peaked softmax turns the fp16 rounding of a chunk's keys (2^-11 of each
    # product, in the mean over 128 channels 2^-11 * |q||k| / sqrt(128)) into that error of p
    err_s = 0.05 * 128 ** 0.5 * k_size * q_size * 2.0 ** -11
    bound = 2.0 ** -8 * np.abs(ref) + v_size * 6 * (2 * 2.0 ** -11 + 8 * err_s)
    assert (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("spike", [0, 1, 77])
def test_attention_query_with_one_large_channel(new, spike):
    """The queries' common power of two follows their largest channel wherever it stands."""
    r = _kv4.Requests(6, [200], [new], 8, 2, 128, 64)
    q = r.q.float() * 0.01
    q[:, :, spike] = 300.0
    q[:, :, (spike + 2) % 128] = -0.03
    r.q = q.bfloat16()
    scale = 0.003  # scores of a few units
    # in chunks the keys' fp16 rounding (2^-11) times 300 * 4 * scale moves a probability by 0.002
    bound = 2.0 ** -8 + 6 * (2 * 2.0 ** -11 + 300 * 4 * scale * 2.0 ** -11)
    ref = r.expected(scale)
    assert (np.abs(r.run(hs, scale).float().cpu().double().numpy() - ref) <= bound * np.maximum(1, np.abs(ref))).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 7, 12, 40])
def test_a_query_row_that_is_no_number_leaves_its_neighbours_alone(new, dim):
    """Of each kv head's four query heads one holds a NaN, one an infinity, the
    others values of about 20 and 300 (past 2^16 under a common scale of 1):
    the first two give NaN, the others what they give alone."""
    r = _kv4.Requests(8, [200], [new], 8, 2, dim, 32)
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
    err_s = scale * dim ** 0.5 * np.array([20., 300.])[kind[kind > 1] - 2][None, :, None] * 2.0 ** -11
    bound = 2.0 ** -8 * np.abs(ref[:, kind > 1]) + 6 * (2 * 2.0 ** -11 + 8 * err_s)
    assert (np.abs(got - ref)[:, kind > 1] <= bound).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 7, 12, 40])
def test_query_rows_of_very_different_sizes(new, dim):
    """Rows 2^30 times smaller than their neighbours keep all their bits: their
    scores, of a few units at this scale, are those that they have alone."""
    r = _kv4.Requests(9, [200], [new], 8, 2, dim, 32)
    small = np.arange(8) % 4 > 1
    size = np.where(small, 2.0 ** -30, 1.0).astype(np.float32)
    r.q = (r.q.float() * torch.from_numpy(size)[None, :, None]).bfloat16()
    scale = 0.09 * 2.0 ** 30
    ref = r.expected(scale)
    got = r.run(hs, scale).float().cpu().double().numpy()
    assert np.isfinite(got).all()
    err_s = 0.09 * dim ** 0.5 * 2.0 ** -11  # of the small rows; the others' softmax is one key's
    bound = 2.0 ** -8 * np.abs(ref[:, small]) + 6 * (2 * 2.0 ** -11 + 8 * err_s)
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
    r = _kv4.Requests(10, [500], [new], hq, 2, dim, 16, k_size=30.0, edit=edit)
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
            # keys rounded to fp16 in chunks (2^-11 of each product) and fp32 sums (2^-20 of the products' sizes at most)
            err = (np.abs(k) @ np.abs(q[i, h])).max() * (2.0 ** -11 + 2.0 ** -20)
            order = np.argsort(s)
            if s[order[-1]] - s[order[-2]] <= 2 * err:
                continue
            seen += 1
            # the value, fp16-rounded in chunks, and its rounding to bf16
            top = v[order[-1]]
            assert (np.abs(got[i, h] - top) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(top) + 2.0 ** -12).all()
    assert seen >= new * hq // 3


@pytest.mark.parametrize("scale,q_size", [(1e-30, 1e-20), (1e-38, 1e-30), (1e30, 3e4), (1e30, 1e5)])
@pytest.mark.parametrize("new", [1, 3, 12, 40])
def test_scales_at_the_ends_of_their_range(scale, q_size, new):
    """Scores of nothing: the mean of the visible values, hidden keys and absent rows
    apart.  Scores of -10^36 and more, one key far above the others: its value."""
    def edit(i, k, v):
        k[:] = -10 - np.abs(k)
        k[17] = -0.5
    r = _kv4.Requests(14, [90, 30], [new, 2], 8, 2, 128, 32, edit=edit)
    r.q = ((r.q.float().abs() + 0.5) * q_size).bfloat16()
    ref = r.expected(scale)
    got = r.run(hs, scale).float().cpu().double().numpy()
    # probabilities rounded to fp16 (2^-11) before their product with codes of values up to 6 wide, values too in chunks
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + 6 * 2 * 2.0 ** -11).all()


@pytest.mark.parametrize("exponent", [-95, 105, 113, 120])
@pytest.mark.parametrize("new,dim", [(1, 128), (3, 64), (12, 128), (40, 128), (40, 64)])
def test_queries_of_any_exponent(exponent, new, dim):
    """Queries of 2^exponent with a scale that makes their scores the usual ones."""
    r = _kv4.Requests(15, [300, 20], [new, 1], 8, 2, dim, 64)
    r.q = (r.q.float() * 2.0 ** exponent).bfloat16()
    scale = dim ** -0.5 * 2.0 ** -exponent
    _close(r.run(hs, scale), r.expected(scale), scale)


def test_attention_strides_streams_and_reuse_of_the_workspace():
    r = _kv4.Requests(21, [700, 90], [2, 2], 16, 4, 128, 64)
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
    big = _kv4.Requests(22, [3000], [1], 32, 2, 128, 64)
    b0 = big.run(hs, 0.09, ws=ws)
    b1 = big.run(hs, 0.09, ws=ws)
    assert torch.equal(a, r.run(hs, 0.09, ws=ws)) and torch.equal(b0, b1)  # bit for bit, call after call
    _close(b0, big.expected(0.09), 0.09)


@pytest.mark.parametrize("ctx,new,hq,hkv,dim", [([900] * 5, [200] * 5, 16, 4, 128), ([1500, 40, 700], [1, 130, 333], 8, 2, 64),
                                                ([3000] * 40, [1] * 40, 32, 8, 128), ([2000] * 9, [3] * 9, 32, 2, 128),
                                                # one row tile: joins in shared memory (few pieces), from memory (many)
                                                ([1500] * 14, [3] * 14, 32, 2, 128), ([3000] * 6, [40] * 6, 4, 4, 64),
                                                ([700, 0, 65], [40, 128, 1], 8, 8, 128), ([20000], [9], 16, 4, 64)])
def test_joined_pieces_do_not_depend_on_who_comes_last(ctx, new, hq, hkv, dim):
    """Work on another stream delays some CTAs, so that an item's pieces arrive in other orders."""
    r = _kv4.Requests(77, ctx, new, hq, hkv, dim, 64)
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
    r = _kv4.Requests(31, [40, 500], [3, 2], 8, 2, 128, 64)
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
    ws = torch.zeros(hs.hs_kv4_attention_workspace_size(c, n, hq), dtype=torch.uint8, **dev)

    def step():
        hs.hs_kv4_plan(cached, new, n, page, n_pages, table, width, ring, cin, 32, table, seq, qs, slot, pos, cout, short)
        hs.hs_kv4_append(c, k, v, slot, 32)
        hs.hs_kv4_attention(c, q, qs, seq, table, n, 32, 0.2, 0, out, ws)
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
    held = [[np.zeros((0, hkv, dim))] * 2 for _ in range(n)]
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
                held[i] = [np.zeros((0, hkv, dim))] * 2
                continue
            add = [_kv4.values(x[at:at + f].float().numpy()) for x in (kk, vv)]
            held[i] = [np.concatenate((a, b)) for a, b in zip(held[i], add)]
            refs.append(_kv4.attention(qq[at:at + f].double().numpy(), *held[i], int(f), len(held[i][0]), 0.2))
            at += f
        _close(out[:total], np.concatenate(refs), 0.2)
    free = int(cin[1] - cin[0])
    rows = table.cpu().numpy()
    assert free + int((rows >= 0).sum()) == n_pages
