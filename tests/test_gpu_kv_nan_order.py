"""NaN values in the chunk kernels of both caches where a CTA goes from an item of two row tiles to one
of a single one: what is known of the last tile's NaN is looked at late there (tests/test_kv_nan_order.py)."""
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


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 128])
def test_nan_of_items_of_two_row_tiles_before_items_of_one(bits, dim):
    """Requests of 160 rows whose last tile of keys holds a NaN value that some rows see, and longer ones of 80
    rows behind them in a CTA's run."""
    n, hkv = 120, 4
    new = [20 if i % 2 == 0 else 10 for i in range(n)]
    length = [260 + i % 7 * 20 if i % 2 == 0 else 700 + i for i in range(n)]

    def edit(i, k, v):
        if i % 2 == 0:
            v[length[i] - 9, i // 2 % hkv, dim - 64:] = np.nan
    r = KIND[bits].Requests(dim, [a - b for a, b in zip(length, new)], new, 8 * hkv, hkv, dim, 64, edit=edit)
    got = r.run(hs, 0.1).float().cpu().double().numpy()
    for i in range(0, n, 2):
        rows = got[r.starts[i]:r.starts[i + 1]]
        want = np.zeros(rows.shape, bool)
        h = i // 2 % hkv
        want[new[i] - 9:, 8 * h:8 * h + 8, dim - 64:] = True
        assert np.array_equal(np.isnan(rows), want), i
        r.v[i] = np.nan_to_num(r.v[i])
    ref = r.expected(0.1)
    ok = ~np.isnan(got)
    assert ok[np.concatenate([np.arange(r.starts[i], r.starts[i + 1]) for i in range(1, n, 2)])].all()
    # the roundings of tests/test_gpu_kv8.py's _close; keys and values of 4 bits are rounded to fp16: as much again, and scores of
    # 100 units at most by 2^-11 of keys, half that in the mean of 64 and more channels
    vmax = max(np.abs(v).max() for v in r.v)
    bound = np.abs(ref) * 2.0 ** -8 + vmax * (2.0 ** -11 + 2 * 2.0 ** -13 + 2.0 ** -20 + (2.0 ** -11 + 2.0 ** -8 if bits == 4 else 0))
    assert (np.abs(got - ref) <= bound)[ok].all()
