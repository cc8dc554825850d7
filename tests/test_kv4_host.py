"""The 4-bit key/value cache without a GPU: refusals of its entry points, and
pins of the tests' 64-bit restatement (tests/_kv4.py) to hand-worked values."""
import ctypes as C

import numpy as np
import pytest

import _kv4
from activation_sparse_moe_gb300 import build as hsbuild
from activation_sparse_moe_gb300 import hs

A = 0x100000  # a fake, aligned device address: validation fails before it is touched


@pytest.fixture(scope="module")
def lib():
    hsbuild.build()
    return hs.lib()


def _cache(pool=A, n_pages=8, page=64, heads=2, dim=128):
    return hs.hs_kv4_cache(pool, n_pages, page, heads, dim)


def test_pool_bytes(lib):
    assert hs.hs_kv4_pool_bytes(_cache()) == 8 * 2 * 64 * (128 + 16)
    assert hs.hs_kv4_pool_bytes(_cache(None, 1 << 20, 16, 8, 64)) == (1 << 20) * 8 * 16 * 72  # past 32 bits
    for bad in (dict(n_pages=0), dict(page=48), dict(page=128), dict(heads=0), dict(heads=257), dict(dim=96), dict(dim=256)):
        assert hs.hs_kv4_pool_bytes(_cache(**bad)) == 0
    assert lib.hs_kv4_pool_bytes(None) == 0


def test_plan_refusals(lib):
    ok = [A, A, 4, 64, 100, A, 8, A, A, 64, A, A, A, A, A, A + 64, A, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.hs_kv4_plan(*a)
    for i in (0, 1, 5, 7, 8, 10, 11, 12, 13, 15, 16):
        assert call(**{f"a{i}": None}) == hs.HS_ERR_INVALID_ARG
    for i in (2, 4, 6, 9):
        assert call(**{f"a{i}": 0}) == hs.HS_ERR_INVALID_ARG
    assert call(a15=A) == hs.HS_ERR_INVALID_ARG            # counters in and out are one
    for p in (0, 8, 48, 128):
        assert call(a3=p) == hs.HS_ERR_UNSUPPORTED_SHAPE
    assert call(a2=4097) == hs.HS_ERR_UNSUPPORTED_SHAPE
    assert call(a2=4096, a6=1 << 18) == hs.HS_ERR_UNSUPPORTED_SHAPE
    assert call(a2=1, a6=1 << 25) == hs.HS_ERR_UNSUPPORTED_SHAPE
    assert call(a4=1 << 30) == hs.HS_ERR_UNSUPPORTED_SHAPE
    assert call(a9=1 << 30) == hs.HS_ERR_UNSUPPORTED_SHAPE
    for i in (0, 1, 5, 7, 10, 11, 12, 14, 16):
        assert call(**{f"a{i}": A + 2}) == hs.HS_ERR_MISALIGNED
    for i in (8, 13, 15):
        assert call(**{f"a{i}": A + 4}) == hs.HS_ERR_MISALIGNED


def test_plan_refuses_outputs_that_overlap(lib):
    """4 requests, 8 entries a row, 100 pages, 64 tokens; each buffer 4096 bytes
    from the next.  The lengths updated in place would be read after they were written."""
    names = "cached new n page pages table_in width ring counters_in tokens table_out seq_len q_start slot position counters_out short stream"
    names = names.split()
    size = dict(cached=16, new=16, table_in=128, ring=400, counters_in=16, table_out=128, seq_len=16, q_start=20, slot=512, position=256,
                counters_out=16, short=4)
    written = ("ring", "table_out", "seq_len", "q_start", "slot", "position", "counters_out", "short")
    ok = {x: A + 4096 * i for i, x in enumerate(size)}

    def call(**kw):
        a = {**dict(n=4, page=64, pages=100, width=8, tokens=64, stream=None), **ok, **kw}
        return lib.hs_kv4_plan(*(a[x] for x in names))
    for x in written:
        for y in size:
            if y == x or {x, y} == {"table_in", "table_out"}:
                continue
            wide = 8  # both ends: y's last bytes and x's first ones, and the other way round
            for at in (ok[x], ok[x] + (size[x] - 1) // wide * wide, ok[x] - (size[y] - 1) // wide * wide):
                assert call(**{y: at}) == hs.HS_ERR_INVALID_ARG, (x, y, at - ok[x])
    for at in (4, 124, -124):
        assert call(table_out=ok["table_in"] + at) == hs.HS_ERR_INVALID_ARG


def _bad_caches():
    yield _cache(pool=None), hs.HS_ERR_INVALID_ARG
    yield _cache(pool=A + 8), hs.HS_ERR_MISALIGNED
    for bad in (dict(n_pages=0), dict(page=24), dict(heads=0), dict(dim=32)):
        yield _cache(**bad), hs.HS_ERR_UNSUPPORTED_SHAPE


def test_plan_gives_no_slot_twice_and_the_header_asks_for_that():
    """The append of a slot given twice is undefined: the plan must not ask for it."""
    rng = np.random.default_rng(6)
    for _ in range(20):
        n, page, width = int(rng.integers(1, 30)), int(rng.choice([16, 32, 64])), 12
        cached = rng.integers(0, 4 * page, n)
        new = rng.integers(-1, 5 * page, n)
        have = -(-cached // page)
        need = int(sum(-(-(c + f) // page) - h for c, f, h in zip(cached, new, have) if f >= 0))
        pages = rng.permutation(int(have.sum()) + need + 3).astype(np.int32)
        table = np.full((n, width), -1, np.int32)
        at = 0
        for i in range(n):
            table[i, :have[i]] = pages[at:at + have[i]]
            at += have[i]
        ring = np.concatenate((pages[at:], np.full(at, -1, np.int32)))
        r = _kv4.plan(cached, new, page, len(pages), table, ring, [0, len(pages) - at], int(new.clip(0).sum()) + 1)
        slots = [s for s in r["slot"] if s >= 0]
        assert r["short"] == 0 and len(set(slots)) == len(slots) == int(new.clip(0).sum())
    text = " ".join(open(hs.HEADER).read().replace("\n *", " ").split())
    assert "what a slot given to tokens of different values holds afterwards is undefined" in text
    assert "leave one of the two in it" not in text


def test_append_and_read_refusals(lib):
    def app(c, k=A, ks=256, kh=128, v=A, vs=256, vh=128, s=A, n=4):
        return lib.hs_kv4_append(C.byref(c) if c else None, k, ks, kh, v, vs, vh, s, n, None)

    def read(c, s=A, n=4, o=(A, A, A, A)):
        return lib.hs_kv4_read(C.byref(c) if c else None, s, n, *o, None)
    for c, st in _bad_caches():
        assert app(c) == st and read(c) == st
    assert app(None) == read(None) == hs.HS_ERR_INVALID_ARG
    c = _cache()
    for kw in (dict(k=None), dict(v=None), dict(s=None), dict(n=-1)):
        assert app(c, **kw) == hs.HS_ERR_INVALID_ARG
    for kw in (dict(k=A + 2), dict(v=A + 8), dict(s=A + 4), dict(ks=260), dict(kh=4), dict(vs=1), dict(vh=-12)):
        assert app(c, **kw) == hs.HS_ERR_MISALIGNED
    assert app(c, n=(1 << 20) + 1) == hs.HS_ERR_UNSUPPORTED_SHAPE
    assert app(c, n=0) == hs.HS_OK and read(c, n=0) == hs.HS_OK      # nothing to do: no launch
    for kw in (dict(s=None), dict(n=-1), dict(o=(None,) * 4)):
        assert read(c, **kw) == hs.HS_ERR_INVALID_ARG
    for kw in (dict(s=A + 4), dict(o=(A + 2, A, A, A)), dict(o=(None, None, None, A + 4))):
        assert read(c, **kw) == hs.HS_ERR_MISALIGNED
    assert read(c, n=(1 << 20) + 1) == hs.HS_ERR_UNSUPPORTED_SHAPE


def test_attention_refusals(lib):
    need = hs.hs_kv4_attention_workspace_size(_cache(), 4, 32)
    assert need > 0
    names = "cache q qs qh start len table width n tokens hq new scale window out os oh ws nb stream".split()
    ok = dict(q=A, qs=4096, qh=128, start=A, len=A, table=A, width=16, n=4, tokens=4, hq=32, new=1, scale=0.1, window=0, out=A,
              os=4096, oh=128, ws=A, nb=need, stream=None)

    def call(c=None, **kw):
        a = {**ok, "cache": C.byref(c or _cache()), **kw}
        return lib.hs_kv4_attention(*(a[x] for x in names))
    for c, st in _bad_caches():
        assert call(c) == st
    for x in ("q", "start", "len", "table", "out"):
        assert call(**{x: None}) == hs.HS_ERR_INVALID_ARG
    for kw in (dict(width=0), dict(n=0), dict(tokens=-1), dict(new=-1), dict(window=-1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**kw) == hs.HS_ERR_INVALID_ARG
    for kw in (dict(hq=1), dict(hq=33), dict(hq=2 * 65), dict(n=4097), dict(width=1 << 25)):
        assert call(**kw) == hs.HS_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(q=A + 2), dict(out=A + 8), dict(qs=4100), dict(qh=2), dict(os=1), dict(oh=-3), dict(start=A + 1),
               dict(len=A + 2), dict(table=A + 3), dict(ws=A + 4)):
        assert call(**kw) == hs.HS_ERR_MISALIGNED
    assert call(ws=None) == call(nb=need - 1) == hs.HS_ERR_WORKSPACE
    assert call(tokens=0) == hs.HS_OK
    for bad in ((_cache(dim=32), 4, 32), (_cache(), 0, 32), (_cache(), 4097, 32), (_cache(), 4, 33), (_cache(), 4, 1), (_cache(), 4, 130)):
        assert hs.hs_kv4_attention_workspace_size(*bad) == 0


def test_attention_refuses_tables_whose_keys_leave_no_room_in_32_bits(lib):
    need = hs.hs_kv4_attention_workspace_size(_cache(page=16, heads=1), 1, 1)

    def call(width):
        return lib.hs_kv4_attention(C.byref(_cache(page=16, heads=1)), A, 128, 128, A, A, A, width, 1, 0, 1, 1, 0.1, 0, A, 128, 128,
                                    A, need, None)
    assert call((1 << 27) - (1 << 9)) == hs.HS_OK                    # (no token: no launch)
    assert call((1 << 27) - (1 << 9) + 1) == call((1 << 27) - 1) == hs.HS_ERR_UNSUPPORTED_SHAPE


def test_binding_wants_contiguous_channels(lib):
    import torch
    k = torch.zeros(4, 2, 256).bfloat16()[:, :, ::2]
    with pytest.raises(hs.HsError):
        hs.hs_kv4_append(_cache(), k, k, 0, 4)


def test_binding_refuses_tensors_that_do_not_fit(lib):
    """What the pointers do not tell the library: each of these was launched on
    other data than the tensors hold.  (A call that the binding passes on ends on the CPU
    in HS_ERR_CUDA at the launch; here none may get there.)"""
    import torch
    b16, i32, i64, f32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
    c = _cache(pool=A, n_pages=8, page=64, heads=2, dim=128)
    z = lambda *s, t=b16: torch.zeros(s, dtype=t)  # noqa: E731

    def refused(f, base, bads):
        for name, values in bads.items():
            for bad in values:
                with pytest.raises(hs.HsError) as e:
                    f(**{**base, name: bad})
                assert e.value.status == hs.HS_ERR_INVALID_ARG, (name, bad.shape if hasattr(bad, "shape") else bad)
    slots = [z(4, t=i32), z(3, t=i64), z(8, t=i64)[::2]]
    refused(hs.hs_kv4_append, dict(cache=c, k=z(4, 2, 128), v=z(4, 2, 128), slots=z(4, t=i64), n_tokens=4, stream=0),
            dict(k=[z(4, 2, 64), z(4, 1, 128), z(3, 2, 128), z(4, 2, 256)[:, :, ::2]], v=[z(4, 2, 64), z(4, 1, 128), z(3, 2, 128)],
                 slots=slots, n_tokens=[5]))
    refused(hs.hs_kv4_read, dict(cache=c, slots=z(4, t=i64), n_tokens=4, k_bf16=z(4, 2, 128), v_bf16=z(4, 2, 128),
                                 k_f32=z(4, 2, 128, t=f32), v_f32=z(4, 2, 128, t=f32), stream=0),
            dict(slots=slots, k_bf16=[z(3, 2, 128)], v_bf16=[z(4, 2, 256)[:, :, :128]], k_f32=[z(4, 2, 64, t=f32)],
                 v_f32=[z(8, 2, 128, t=f32)[::2]]))
    refused(hs.hs_kv4_attention, dict(cache=c, q=z(4, 8, 128), q_start=z(4, t=i32), seq_len=z(3, t=i32), table=z(3, 16, t=i32), n_seqs=3,
                                      max_new=2, scale=0.1, window=0, out=z(4, 8, 128), workspace=z(1, t=torch.uint8),
                                      workspace_bytes=1 << 30, stream=0),
            dict(q=[z(4, 8, 64), z(3, 8, 128), z(4, 4, 128), z(4, 8, 256)[:, :, ::2]], out=[z(4, 8, 64), z(3, 8, 128)],
                 q_start=[z(3, t=i32)], seq_len=[z(2, t=i32)], table=[z(3, 32, t=i32)[:, :16], z(2, 16, t=i32), z(16, 3, t=i32).T]))
    plan = dict(cached_len=z(4, t=i32), new_len=z(4, t=i32), n_seqs=4, page_tokens=64, n_pages=100, table_in=z(4, 8, t=i32),
                table_width=8, ring=z(100, t=i32), counters_in=z(2, t=i64), max_tokens=64, table_out=z(4, 8, t=i32), seq_len=z(4, t=i32),
                q_start=z(5, t=i32), slot=z(64, t=i64), position=z(64, t=i32), counters_out=z(2, t=i64), short=z(1, t=i32), stream=0)
    refused(hs.hs_kv4_plan, plan, dict(table_in=[z(4, 16, t=i32)[:, :8]], table_out=[z(4, 16, t=i32)[:, :8]], slot=[z(64, t=i32)]))


# ------------------------------------------------ pins of the restatement
def test_quantiser_by_hand():
    x = np.zeros((1, 64), np.float32)
    x[0, :16] = np.arange(16) - 8                      # -8 .. 7: scale 1, bias -8, exact
    codes, scale, bias = _kv4.quantise(x)
    assert scale[0, 0] == 1 and bias[0, 0] == -8
    assert list(codes[0, :17]) == list(range(16)) + [8]
    assert np.array_equal(_kv4.values(x), x)
    flat = np.full((1, 64), 2.5, np.float32)            # one value: scale 0
    assert np.array_equal(_kv4.values(flat), flat) and not _kv4.quantise(flat)[0].any()
    half = np.zeros((1, 64), np.float32)
    half[0, :3] = (15, 0.5, 1.5)                       # ties go to the even code
    assert list(_kv4.quantise(half)[0][0, :4]) == [15, 0, 2, 0]
    x[0, 3] = np.inf
    assert np.isnan(_kv4.values(x)).all()


def test_quantiser_error_is_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.normal(0, 1, (50, 128)).astype(np.float32)
    _, scale, bias = _kv4.quantise(x)
    err = np.abs(_kv4.values(x) - x).reshape(50, 2, 64)
    # half a step, the rounding of bias (2^-11 of it) and of the scale (15 * 2^-11 of a step)
    bound = scale[..., None].astype(float) * (0.5 + 15 * 2.0 ** -11) + np.abs(bias[..., None].astype(float)) * 2.0 ** -11
    assert (err <= bound).all()


def test_pool_layout_by_hand():
    page, dim = 16, 64
    pool = np.zeros((2, 1, _kv4.record_bytes(page, dim)), np.uint8)
    k = np.zeros((1, 1, 64), np.float32)
    k[0, 0, :2] = (15, 3)
    v = np.full((1, 1, 64), -1, np.float32)
    _kv4.fill_pool(pool, page, dim, [16 + 5], k, v)
    rec = pool[1, 0]
    assert rec[5 * 32] == 15 | 3 << 4 and not rec[:5 * 32].any()
    pairs = rec[2 * 16 * 32:].view(np.float16)
    assert pairs[5 * 2] == 1 and pairs[5 * 2 + 1] == 0
    assert pairs[32 + 5 * 2] == 0 and pairs[32 + 5 * 2 + 1] == -1
    assert not pool[0].any()


def test_attention_restatement_closed_forms():
    rng = np.random.default_rng(3)
    k, v = np.zeros((9, 1, 64)), rng.normal(0, 1, (9, 1, 64))
    q = rng.normal(0, 1, (2, 2, 64))
    out = _kv4.attention(q, k, v, 2, 9, 1.0)            # equal scores: the mean of what is seen
    assert np.allclose(out[0], v[:8].mean(0)) and np.allclose(out[1], v.mean(0))
    out = _kv4.attention(q, k, v, 2, 9, 1.0, window=1)  # the token itself
    assert np.allclose(out[0], v[7]) and np.allclose(out[1], v[8])
    assert not _kv4.attention(q, k, v, 2, 9, 1.0, present=np.zeros(9, bool)).any()


def test_plan_restatement_by_hand():
    table = np.array([[4, 2, -1], [7, -1, -1], [1, -1, -1]], np.int32)
    ring = np.array([0, 3, 5, 6, 8, 9, -1, -1, -1, -1], np.int32)
    r = _kv4.plan([32, 3, 16], [1, -1, 17], 16, 10, table, ring, [10, 16], 20)
    assert r["short"] == 0 and r["counters"] == [13, 17]
    assert r["table"].tolist() == [[4, 2, 0], [-1] * 3, [1, 3, 5]]
    assert r["ring"].tolist() == [0, 3, 5, 6, 8, 9, 7, -1, -1, -1]
    assert r["seq_len"] == [33, 0, 33] and r["q_start"] == [0, 1, 1, 18]
    assert r["slot"] == [0] + list(range(48, 64)) + [80, -1, -1]
    assert r["position"] == [32] + list(range(16, 33)) + [-1, -1]
    short = _kv4.plan([32, 3, 16], [1, -1, 17], 16, 10, table, ring, [10, 12], 20)
    assert short["short"] == 1 and short["q_start"] == [0] * 4 and short["counters"] == [10, 13]
