"""The 8-bit key/value cache without a GPU: refusals of its entry points, pins of
the tests' 64-bit restatement (tests/_kv8.py) to hand-worked values, and the waits
of its attention kernels."""
import ctypes as C
import math
import pathlib
import re

import numpy as np
import pytest

import _kv8
import test_kv4_drains as drains
from activation_sparse_moe_gb300 import build as hsbuild
from activation_sparse_moe_gb300 import hs

A = 0x100000  # a fake, aligned device address: validation fails before it is touched


@pytest.fixture(scope="module")
def lib():
    hsbuild.build()
    return hs.lib()


def _cache(pool=A, n_pages=8, page=64, heads=2, dim=128):
    return hs.hs_kv8_cache(pool, n_pages, page, heads, dim)


def _bad_caches():
    yield _cache(pool=None), hs.HS_ERR_INVALID_ARG
    yield _cache(pool=A + 8), hs.HS_ERR_MISALIGNED
    for bad in (dict(n_pages=0), dict(page=24), dict(page=128), dict(heads=0), dict(heads=257), dict(dim=32), dict(dim=96)):
        yield _cache(**bad), hs.HS_ERR_UNSUPPORTED_SHAPE


def test_pool_bytes(lib):
    assert hs.hs_kv8_pool_bytes(_cache()) == 8 * 2 * 64 * 257
    assert hs.hs_kv8_pool_bytes(_cache(None, 1 << 20, 16, 8, 64)) == (1 << 20) * 8 * 16 * 129  # past 32 bits
    for c, st in list(_bad_caches())[2:]:
        assert hs.hs_kv8_pool_bytes(c) == 0
    assert lib.hs_kv8_pool_bytes(None) == 0
    for page in (16, 32, 64):
        for dim in (64, 128):
            assert _kv8.record_bytes(page, dim) % 16 == 0 and hs.hs_kv8_pool_bytes(_cache(None, 1, page, 1, dim)) == _kv8.record_bytes(page, dim)


def test_append_and_read_refusals(lib):
    def app(c, k=A, ks=256, kh=128, v=A, vs=256, vh=128, s=A, n=4):
        return lib.hs_kv8_append(C.byref(c) if c else None, k, ks, kh, v, vs, vh, s, n, None)

    def read(c, s=A, n=4, o=(A, A, A, A)):
        return lib.hs_kv8_read(C.byref(c) if c else None, s, n, *o, None)
    for c, st in _bad_caches():
        assert app(c) == st and read(c) == st
    assert app(None) == read(None) == hs.HS_ERR_INVALID_ARG
    c = _cache()
    for kw in (dict(k=None), dict(v=None), dict(s=None), dict(n=-1)):
        assert app(c, **kw) == hs.HS_ERR_INVALID_ARG
    for kw in (dict(k=A + 2), dict(v=A + 8), dict(s=A + 4), dict(ks=260), dict(kh=4), dict(vs=1), dict(vh=-12)):
        assert app(c, **kw) == hs.HS_ERR_MISALIGNED
    assert app(c, n=(1 << 20) + 1) == read(c, n=(1 << 20) + 1) == hs.HS_ERR_UNSUPPORTED_SHAPE
    assert app(c, n=0) == hs.HS_OK and read(c, n=0) == hs.HS_OK      # nothing to do: no launch
    for kw in (dict(s=None), dict(n=-1), dict(o=(None,) * 4)):
        assert read(c, **kw) == hs.HS_ERR_INVALID_ARG
    for kw in (dict(s=A + 4), dict(o=(A + 2, A, A, A)), dict(o=(None, None, None, A + 4))):
        assert read(c, **kw) == hs.HS_ERR_MISALIGNED


def test_attention_refusals(lib):
    need = hs.hs_kv8_attention_workspace_size(_cache(), 4, 32)
    assert need > 0
    names = "cache q qs qh start len table width n tokens hq new scale window out os oh ws nb stream".split()
    ok = dict(q=A, qs=4096, qh=128, start=A, len=A, table=A, width=16, n=4, tokens=4, hq=32, new=1, scale=0.1, window=0, out=A,
              os=4096, oh=128, ws=A, nb=need, stream=None)

    def call(c=None, **kw):
        a = {**ok, "cache": C.byref(c or _cache()), **kw}
        return lib.hs_kv8_attention(*(a[x] for x in names))
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
        assert hs.hs_kv8_attention_workspace_size(*bad) == 0


def test_binding_refuses_tensors_that_do_not_fit(lib):
    import torch
    b16, i32, i64, f32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
    c = _cache(pool=A, n_pages=8, page=64, heads=2, dim=128)
    z = lambda *s, t=b16: torch.zeros(s, dtype=t)  # noqa: E731

    def refused(f, base, bads):
        for name, items in bads.items():
            for bad in items:
                with pytest.raises(hs.HsError) as e:
                    f(**{**base, name: bad})
                assert e.value.status == hs.HS_ERR_INVALID_ARG, (name, bad.shape if hasattr(bad, "shape") else bad)
    slots = [z(4, t=i32), z(3, t=i64), z(8, t=i64)[::2]]
    half, wide = torch.float16, f32
    refused(hs.hs_kv8_append, dict(cache=c, k=z(4, 2, 128), v=z(4, 2, 128), slots=z(4, t=i64), n_tokens=4, stream=0),
            dict(k=[z(4, 2, 64), z(4, 1, 128), z(3, 2, 128), z(4, 2, 256)[:, :, ::2], z(4, 2, 128, t=half)],
                 v=[z(4, 2, 64), z(4, 1, 128), z(3, 2, 128), z(4, 2, 128, t=wide)], slots=slots, n_tokens=[5]))
    refused(hs.hs_kv8_read, dict(cache=c, slots=z(4, t=i64), n_tokens=4, k_bf16=z(4, 2, 128), v_bf16=z(4, 2, 128),
                                 k_f32=z(4, 2, 128, t=f32), v_f32=z(4, 2, 128, t=f32), stream=0),
            dict(slots=slots, k_bf16=[z(3, 2, 128)], v_bf16=[z(4, 2, 256)[:, :, :128]], k_f32=[z(4, 2, 64, t=f32)],
                 v_f32=[z(8, 2, 128, t=f32)[::2]]))
    refused(hs.hs_kv8_attention, dict(cache=c, q=z(4, 8, 128), q_start=z(4, t=i32), seq_len=z(3, t=i32), table=z(3, 16, t=i32), n_seqs=3,
                                      max_new=2, scale=0.1, window=0, out=z(4, 8, 128), workspace=z(1, t=torch.uint8),
                                      workspace_bytes=1 << 30, stream=0),
            dict(q=[z(4, 8, 64), z(3, 8, 128), z(4, 4, 128), z(4, 8, 256)[:, :, ::2], z(4, 8, 128, t=half)],
                 out=[z(4, 8, 64), z(3, 8, 128), z(4, 8, 128, t=wide)], q_start=[z(3, t=i32)], seq_len=[z(2, t=i32)],
                 table=[z(3, 32, t=i32)[:, :16], z(2, 16, t=i32), z(16, 3, t=i32).T]))


def test_binding_refuses_other_types(lib):
    """What the library would write past the end of (floats into bf16 rows) or misread (64-bit offsets, every other word)."""
    import torch
    b16, i32, i64, f32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
    c = _cache(pool=A, n_pages=8, page=64, heads=2, dim=128)
    rows = lambda t: torch.zeros(4, 2, 128, dtype=t)  # noqa: E731
    read = dict(cache=c, slots=torch.zeros(4, dtype=i64), n_tokens=4, stream=0)
    for name, bad in (("k_bf16", f32), ("v_bf16", torch.float16), ("k_f32", b16), ("v_f32", b16), ("k_f32", torch.float64)):
        with pytest.raises(hs.HsError) as e:
            hs.hs_kv8_read(**read, **{name: rows(bad)})
        assert e.value.status == hs.HS_ERR_INVALID_ARG
    words = lambda n, t: torch.zeros(n, dtype=t)  # noqa: E731
    base = dict(cache=c, q=torch.zeros(4, 8, 128, dtype=b16), q_start=words(4, i32), seq_len=words(3, i32), table=torch.zeros(3, 16, dtype=i32),
                n_seqs=3, max_new=2, scale=0.1, window=0, out=torch.zeros(4, 8, 128, dtype=b16), workspace=words(1, torch.uint8),
                workspace_bytes=1 << 30, stream=0)
    for name, bad in (("q_start", words(4, i64)), ("q_start", words(8, i32)[::2]), ("seq_len", words(3, i64)), ("seq_len", words(6, i32)[::2]),
                      ("table", torch.zeros(3, 16, dtype=i64)), ("table", torch.zeros(3, 16, dtype=torch.int16))):
        with pytest.raises(hs.HsError) as e:
            hs.hs_kv8_attention(**{**base, name: bad})
        assert e.value.status == hs.HS_ERR_INVALID_ARG


# ------------------------------------------------ pins of the restatement
def test_codes_by_hand():
    t = _kv8.TABLE
    assert t[0x7E] == 448 and t[0x08] == 2.0 ** -6 and t[0x01] == 2.0 ** -9 and t[0xC0] == -2 and math.isnan(t[0xFF])
    assert (np.diff(t[:127]) > 0).all()
    assert _kv8.codes_of([0.0, -0.0, 448, 1, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, -17]).tolist() == \
        [0, 128, 0x7E, 0x38, 0x38, 0x3A, 0, 2, 128 | 0x58]                                  # ties to the even byte
    for b in (0, 1, 7, 8, 0x40, 0x7E, 0x81, 0xFE):
        assert _kv8.codes_of(t[b]) == b
    import torch
    x = np.random.default_rng(0).normal(0, 1, 20000) * np.exp(np.random.default_rng(1).normal(0, 3, 20000))
    x = x[np.abs(x) <= 448].astype(np.float32)
    assert np.array_equal(_kv8.codes_of(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scale_by_hand():
    assert _kv8.exponent(448) == 0 and _kv8.exponent(448.5) == 1 and _kv8.exponent(0) == -15 and _kv8.exponent(57344) == 7
    assert _kv8.exponent(224) == -1 and _kv8.exponent(1.75) == -8 and _kv8.exponent(1.7578125) == -7


@pytest.mark.parametrize("dim", [64, 128])
def test_append_by_hand(dim):
    pool = np.full((2, 1, _kv8.record_bytes(32, dim)), 0xFF, np.uint8)
    k, v = np.zeros((2, 1, dim)), np.full((2, 1, dim), 7.0)
    k[0, 0, 17], k[1, 0, 3] = 448.0, -2.0
    _kv8.append(pool, 32, dim, [32 + 16, 32 + 17], k, v)      # page 1, its second block
    rec = pool[1, 0]
    o = 16 * dim
    turn1 = 2 if dim == 128 else 0                              # of offset 17
    assert rec[o + 17] == 0x7E and rec[o + dim + 16 * turn1 + 3] == 0xC0 and not rec[o:o + 17].any()
    scales = rec[2 * 32 * dim:].view(np.float32)
    assert scales[4] == 1 and scales[5] == 2.0 ** -6 and scales[6] == scales[7] == 0 and np.isnan(scales[0])
    # a token of twice the size: the scale grows by two, older codes by one less in their exponent
    k2 = np.zeros((1, 1, dim))
    k2[0, 0, 0] = 896
    _kv8.append(pool, 32, dim, [32 + 18], k2, v[:1])
    assert scales[4] == 2 and rec[o + 17] == 0x76 and rec[o + dim + 16 * turn1 + 3] == 0xB8
    got, _ = _kv8.read(pool, 32, dim, [48, 49, 50, -1])
    assert got[0, 0, 17] == 448 and got[1, 0, 3] == -2 and got[2, 0, 0] == 896 and not got[3].any()
    # a smaller one leaves it; what is no number takes its 64 channels and no others
    k2[0, 0, 0], k2[0, 0, dim - 64] = 1, np.inf
    _kv8.append(pool, 32, dim, [32 + 19], k2, v[:1])
    got, _ = _kv8.read(pool, 32, dim, [51])
    assert scales[4] == 2 and np.isnan(got[0, 0, dim - 64:]).all() and (dim == 64 or got[0, 0, 0] == 1)
    _kv8.append(pool, 32, dim, [32 + 16], np.ones_like(k2), v[:1])  # the block begins anew
    assert scales[4] == 2.0 ** -8


def test_whole_requests_are_appended_as_block_by_block():
    rng = np.random.default_rng(3)
    for page, dim, n in ((16, 64, 33), (64, 128, 50), (32, 128, 16)):
        k, v = rng.normal(0, 1, (2, n, 2, dim)) * np.exp(rng.normal(0, 2, (2, n, 1, 1)))
        k[5, 0, 3], v[n - 1, 1, dim - 1] = np.nan, 1e6
        slots = rng.permutation(-(-n // page) + 1)[np.arange(n) // page] * page + np.arange(n) % page
        a, b = (np.zeros((-(-n // page) + 1, 2, _kv8.record_bytes(page, dim)), np.uint8) for _ in range(2))
        _kv8.append(a, page, dim, slots, k, v)
        _kv8.fill(b, page, dim, slots, k, v)
        assert np.array_equal(a, b)
        for x, y in zip(_kv8.read(a, page, dim, slots), (k, v)):
            assert np.array_equal(x, _kv8.values(y), equal_nan=True)
            fine = np.isfinite(x)
            # half a step of e4m3 (2^-4), or half its smallest one at the block's scale
            e = _kv8._blocks(y)[1][..., None] + np.zeros(x.shape)
            assert (np.abs(x - y)[fine] <= np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** (e - 10))[fine]).all()


def test_every_held_value_is_exact_in_fp16_and_bf16():
    import torch
    for e in (_kv8.LOW, -3, 0, _kv8.HIGH):
        x = torch.from_numpy(_kv8.TABLE[np.isfinite(_kv8.TABLE)] * 2.0 ** e)
        assert torch.equal(x.half().double(), x) and torch.equal(x.bfloat16().double(), x)


# -------------------------------------------------------------- the waits
CSRC = pathlib.Path(hs.PKG) / "csrc"


def test_few_row_kernel_waits_for_its_copies():
    src = drains._squeeze("hs_kv8_attn.cu")
    depths = [int(x) for x in re.search(r"kSlots = D == 128 \? (\d+) : (\d+);", src).groups()]
    end = ("if (phase >= 2) { do { mbar_wait(full + slot, phase & 1); if (++slot == C::kSlots) slot = 0, phase ^= 1; } "
           "while (slot != in_slot); }") in src
    for slots in depths:
        for steps in range(1, 4 * slots + 2):
            for give_up in [None, *range(steps)]:
                left, wrong = drains.few_row_waits(steps, give_up, slots, end)
                assert not wrong and not left, (slots, steps, give_up, left)


def test_chunk_kernel_waits_for_its_copies_and_products():
    src = drains._squeeze("hs_kv8_prefill.cu")
    slots = int(re.search(r"kPfPacked = (\d+)", src)[1])
    end = ("for (uint32_t i = f > kPfPacked ? f - kPfPacked : 0; i < f; ++i) "
           "mbar_wait(sh.packed_full + i % kPfPacked, (i / kPfPacked) & 1);") in src
    for fills in range(0, 5 * slots):
        for taken in range(max(0, fills - slots), fills + 1):
            assert not drains.chunk_waits(fills, taken, slots, end), (fills, taken)
    assert re.search(r"umma_commit\(&sh\.products_done\); __syncwarp\(\); mbar_wait\(&sh\.products_done, 0\);",
                     src[:src.index("tmem_dealloc(tmem, 512)")])
    # the joins' copies: none is asked for after a wait gave up, and those of that round and the next are waited for
    assert ("if (given_up >= 0) { for (int k = given_up; k < min(given_up + 2, rounds); ++k) "
            "mbar_wait(bars + (k & 1), k >> 1 & 1); }") in src
    assert "if (warp == 7 && k + 2 < rounds && given_up < 0) fetch(k + 2);" in src


@pytest.mark.parametrize("name,decided", [("hs_kv8_attn.cu", 0), ("hs_kv8_prefill.cu", 0)])
def test_every_wait_is_bounded_and_given_up_by_a_warp_as_one(name, decided):
    src = drains._squeeze(name)
    assert "mbarrier.try_wait" not in src and "mbarrier.test_wait" not in src and not re.search(r"while \(!mbar_(try_wait|test)", src)
    uses = [m.start() for m in re.finditer(r"\bmbar_wait\(", src)]
    assert uses and sum(1 for at in uses if not re.search(r"[;{})] $", src[:at])) == decided


@pytest.mark.parametrize("packed", [2, 3])
def test_stages_and_tiles_of_the_chunk_kernel_keep_step(packed):
    """The loader, the converting warps and the products count halves and tiles apart:
    every wait's parity is that of the phase it is for."""
    src = drains._squeeze("hs_kv8_prefill.cu")
    assert "slot = (f >> 1) % kPfSlots" in src and "(f / kPfPacked + 1) & 1" in src and "((f >> 1) / kPfSlots + 1) & 1" in src
    slots, fills = 3, 60
    full, empty, kv_full, kv_empty = [0] * packed, [0] * packed, [0] * slots, [0] * slots
    done = 0                                        # tiles whose products are done

    def passed(phases, parity):                     # a wait on a parity passes once that phase is complete
        return phases % 2 != parity
    for f in range(fills):
        st, tile = f % packed, f >> 1
        if f >= packed:
            assert passed(empty[st], (f // packed + 1) & 1)
        full[st] += 1
        assert passed(full[st], (f // packed) & 1)
        empty[st] += 1
        if f % 2 == 0 and tile >= slots:
            while not passed(kv_empty[tile % slots], (tile // slots + 1) & 1):
                assert passed(kv_full[done % slots], (done // slots) & 1)
                kv_empty[done % slots] += 1
                done += 1
            assert done >= tile - slots + 1
        if f % 2:
            kv_full[tile % slots] += 1


def test_eight_lanes_of_the_converting_warps_meet_no_bank_twice():
    """What the layout's turned chunks and the order of the work are for."""
    for dim in (64, 128):
        ng = dim // 64
        for first in range(0, 64 * dim // 16, 8):
            reads, writes = set(), [set(), set()]
            for i in range(first, first + 8):
                r = i >> 3 if ng == 1 else i >> 4
                key = (r >> 1) << 2 | ((r & 1) ^ (3 if i & 4 else 0))
                c = i & 3 if ng == 1 else (i & 3) | (i >> 1 & 4)
                turn = ((2 * (key & 3)) ^ (key & 4)) if dim == 128 else key & 2
                reads.add((key * dim + (c ^ turn) * 16) % 128 // 16)
                for x in range(2):
                    writes[x].add((key * 128 + ((((c & 3) * 2 + x) ^ (key & 7)) << 4)) % 128 // 16)
            assert len(reads) == 8 and all(len(w) == 8 for w in writes)
        places = set()
        for i in range(64 * dim // 16):
            r = i >> 3 if ng == 1 else i >> 4
            places.add(((r >> 1) << 2 | ((r & 1) ^ (3 if i & 4 else 0)), i & 3 if ng == 1 else (i & 3) | (i >> 1 & 4)))
        assert places == {(k, c) for k in range(64) for c in range(dim // 16)}


def test_lanes_of_the_few_row_kernel_meet_no_bank_twice():
    for first in range(0, 32, 8):
        for i in range(2):
            keys, vals = set(), set()
            for lane in range(first, first + 8):
                g, t = lane >> 2, lane & 3
                kr = (g >> 1) + 4 * (g & 1)
                turn = lambda o: (2 * (o & 3)) ^ (o & 4)  # noqa: E731
                keys.add((kr * 128 + ((t + 4 * i) ^ turn(kr)) * 16) % 128)
                vals.add(((t + 4 * i) * 128 + (g ^ turn(t + 4 * i)) * 16) % 128)
            assert len(keys) == 8 and len(vals) == 8
