"""Attention at the end of the longest rows that a table may have, over both caches: what
the kernels look ahead stays within 32 bits."""
import numpy as np
import pytest
import torch

import _kv4
import _kv8
from activation_sparse_moe_gb300 import hs

pytestmark = pytest.mark.gpu

KIND = {4: _kv4, 8: _kv8}
MOST = (1 << 31) - (1 << 13)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from activation_sparse_moe_gb300 import build
    build.build()
    hs.lib()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new,hq,dim", [(1, 4, 128), (1, 16, 64), (3, 4, 64), (5, 4, 128), (40, 4, 128)])
@pytest.mark.parametrize("short", [0, 1, 77])
def test_the_longest_rows_by_a_window(bits, page, new, hq, dim, short):
    """A window of 300 at the end of 2^31 - 2^13 keys (less some): every page before it is not there."""
    window, length = 300, MOST - short
    rng = np.random.default_rng(new + hq)
    first = (length - new - window + 1) // page * page      # its page's first key
    held = length - first
    k, v, q = _kv4.bf16(rng, (held, 1, dim)), _kv4.bf16(rng, (held, 1, dim)), _kv4.bf16(rng, (new, hq, dim))
    pages = -(-held // page)
    pool = np.full((pages, 1, KIND[bits].record_bytes(page, dim)), 0xFF, np.uint8)
    (_kv4.fill_pool if bits == 4 else _kv8.fill)(pool, page, dim, np.arange(held), k.float().numpy(), v.float().numpy())
    table = torch.full((1, MOST // page), -1, dtype=torch.int32, device="cuda")
    table[0, first // page:first // page + pages] = torch.arange(pages, dtype=torch.int32, device="cuda")
    make, size, call = ((hs.make_kv4_cache, hs.hs_kv4_attention_workspace_size, hs.hs_kv4_attention) if bits == 4 else
                        (hs.make_kv8_cache, hs.hs_kv8_attention_workspace_size, hs.hs_kv8_attention))
    on = torch.from_numpy(pool).cuda()
    c = make(on, pages, page, 1, dim)
    ws = torch.zeros(size(c, 1, hq), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"), device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    call(c, q.cuda(), i32([0, new]), i32([length]), table, 1, new, 0.09, window, out, ws)
    torch.cuda.synchronize()
    assert hs.hs_device_status() == hs.HS_OK
    kk, vv = (KIND[bits].values(x.float().numpy()) for x in (k, v))
    got = out.double().cpu().numpy()
    ref = _kv4.attention(q.double().numpy(), kk, vv, new, held, 0.09, window)
    # half a step of bf16, probabilities to fp16, scores: as tests/test_gpu_kv8.py's _close; 4 bits in chunks as in tests/test_gpu_kv_hidden.py
    chunk = 2.0 ** -11 + 2.0 ** -8 if bits == 4 and new * hq > 64 else 0
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + np.abs(vv).max() * (2.0 ** -11 + 2 * 2.0 ** -13 + 2.0 ** -20 + chunk)).all()
