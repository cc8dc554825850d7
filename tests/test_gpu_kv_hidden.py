"""A row of attention does not depend on what it does not see: on the size of values
before its window or behind its causal border, nor on memory before every row's
window that no token was ever written to.  Both caches, both kernels of each."""
import numpy as np
import pytest

import _kv4
import _kv8
from activation_sparse_moe_gb300 import hs

pytestmark = pytest.mark.gpu

KIND = {4: _kv4, 8: _kv8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from activation_sparse_moe_gb300 import build
    build.build()
    hs.lib()


def _bounded(r, bits, got, scale, window):
    """Every row within its own bound, of what it sees: the last rounding, half a bf16 step,
    2^-8 of the value; each probability's rounding to fp16 (2^-11) and the scores' (two times
    2^-13, as in test_gpu_kv8._close), of the sum of the products' sizes; and of the few-row kernels'
    products below fp16's normal range, 2^-25 by 2^-6 of the largest scale that
    the row sees for each key.  Sizes: of a product with a code of 8 bits the value's, of 4 bits at
    most its group's range."""
    ref = r.expected(scale, window)
    got = got.float().cpu().double().numpy()
    assert np.isfinite(got).all()
    at, q, worst = 0, r.q.double().numpy(), 0.0
    for i, new in enumerate(r.new):
        n, v = r.len[i], r.v[i]
        groups = v.reshape(n, v.shape[1], -1, 64)
        size = np.abs(v) if bits == 8 else np.repeat(np.ptp(groups, -1), 64, -1).reshape(v.shape)
        wide = _kv4.attention(q[at:at + new], r.k[i], size, new, n, scale, window)
        for j in range(new):
            p = n - new + j
            lo = max(0, p - window + 1) if window else 0
            if bits == 8:           # a scale is that of all its 16 tokens, of at least half of 448 times it
                top = max(2 * np.abs(v[lo // 16 * 16:p // 16 * 16 + 16]).max(), 448 * 2.0 ** -15)
            else:
                top = max(2 * size[lo:p + 1].max(), 15 * 2.0 ** -14)
            bound = np.abs(ref[at + j]) * 2.0 ** -8 + wide[j] * (2.0 ** -11 + 2.0 ** -12) + top * (p + 1 - lo) * 2.0 ** -31
            worst = max(worst, float((np.abs(got[at + j] - ref[at + j]) / bound).max()))
        at += new
    assert worst <= 1, worst


SMALL, BIG = 0.003, 50000.0


def _sizes(big):
    def edit(i, k, v):
        v *= SMALL
        for a, b in big:
            v[a:b] = np.where(v[a:b] < 0, -BIG, BIG)
    return edit


ROWS = [(1, 2, 64), (1, 16, 128), (3, 8, 128), (4, 16, 64), (8, 8, 64), (8, 8, 128)]


# (of 4 bits only what never goes to the chunk kernel, whose keys are rounded to fp16)
@pytest.mark.parametrize("bits,new,hq,dim", [(b, *x) for b in (4, 8) for x in ROWS] + [(8, 12, 8, 128), (8, 16, 8, 128)])
@pytest.mark.parametrize("page", [16, 64])
def test_large_values_before_the_window(bits, new, hq, dim, page):
    """A block of 16 that no row sees, in a step of 32 keys that the rows' windows begin in: key 112."""
    length = 210
    window = length - new - 112 + 1
    r = KIND[bits].Requests(new + dim, [length - new, 40], [new, 1], hq, 2, dim, page, edit=lambda i, k, v: _sizes([] if i else [(96, 112)])(i, k, v))
    _bounded(r, bits, r.run(hs, 0.1, window), 0.1, window)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hq,dim", [(2, 64), (4, 128), (8, 64), (8, 128), (16, 128)])
@pytest.mark.parametrize("window", [0, 60])
def test_large_values_behind_a_rows_border(bits, hq, dim, window):
    """Drafts whose last two tokens hold large values, in a block of 16 of their own in the step's second half:
    the rows before them do not see it."""
    r = KIND[bits].Requests(hq + dim, [204], [6], hq, 2, dim, 16, edit=_sizes([(208, 210)]))
    _bounded(r, bits, r.run(hs, 0.1, window), 0.1, window)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hq,dim", [(2, 64), (4, 128), (8, 64), (8, 128), (16, 128)])
def test_large_values_that_only_the_first_rows_windows_reach(bits, hq, dim):
    """The window's border passes key 112 between the fourth row and the fifth; key 111 is large."""
    r = KIND[bits].Requests(hq + dim, [207], [6], hq, 2, dim, 16, edit=_sizes([(111, 112)]))
    _bounded(r, bits, r.run(hs, 0.1, 100), 0.1, 100)


@pytest.mark.parametrize("kind", ["ones", "infinite", "largest", "negative"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new,hq,dim", [(1, 4, 128), (3, 8, 64), (8, 8, 128), (40, 8, 128), (70, 4, 64), (300, 2, 128)])
def test_memory_before_every_window_that_was_never_written(kind, bits, new, hq, dim):
    """Tokens before the window that were not appended (slots of -1): their blocks hold codes and
    scales that no append writes."""
    length = 300 + new
    window = 93
    first = length - new - window + 1               # the first key that some row sees: 208, in the middle of a step of 32
    r = KIND[bits].Requests(new + dim, [length - new, 40], [new, 1], hq, 2, dim, 64)
    rows = r.table[0].astype(np.int64)
    f16 = {"ones": 0xFFFF, "infinite": 0x7C00, "largest": 0x7BFF, "negative": 0xFBFF}[kind]
    f32 = {"ones": 0xFFFFFFFF, "infinite": 0x7F800000, "largest": 0x7F7FFFFF, "negative": 0xFF000000}[kind]
    for t in range(first // 16 * 16):
        rec, o = r.pool_np[rows[t // 64]], t % 64
        if bits == 4:
            at, n = 64 * dim + o * (dim // 16), dim // 16
            for x in (0, 64 * (dim // 16)):         # pairs of (scale, bias), K's and V's
                pair = np.array([f16, 0], np.uint16).view(np.uint8)
                rec[:, at + x:at + x + n] = np.tile(pair, n // 4)
            for x in (0, 64 * dim // 2):
                rec[:, x + o * dim // 2:x + (o + 1) * dim // 2] = 0xFF
        else:
            at = 2 * 64 * dim + o // 16 * 16
            rec[:, at:at + 16] = np.array([f32] * 4, np.uint32).view(np.uint8)
            for x in (0, 64 * dim):
                rec[:, x + o * dim:x + (o + 1) * dim] = 0xFF if kind == "ones" else 0x7E
    ref = r.expected(0.1, window)
    got = r.run(hs, 0.1, window).float().cpu().double().numpy()
    assert np.isfinite(got).all()
    # the roundings of tests/test_gpu_kv8.py's _close; keys and values of 4 bits are rounded to fp16 in chunks: as much again,
    # and scores of 100 units at most by 2^-11 of keys, half that in the mean of 64 and more channels
    err = np.abs(got - ref)
    vmax = max(np.abs(v).max() for v in r.v)
    chunk = 2.0 ** -11 + 2.0 ** -8 if bits == 4 and new * hq // 2 > 64 else 0
    assert (err <= np.abs(ref) * 2.0 ** -8 + vmax * (2.0 ** -11 + 2 * 2.0 ** -13 + 2.0 ** -20 + chunk)).all(), float(err.max())
