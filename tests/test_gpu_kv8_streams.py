"""The calls of the 8-bit cache on streams of the caller's, at once and behind work that those
streams still have to do."""
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


@pytest.mark.parametrize("hkv,dim,page,t", [(2, 128, 64, 300), (8, 64, 16, 41), (1, 64, 32, 1)])
def test_appends_and_reads_on_two_streams_at_once(hkv, dim, page, t):
    """A pool and outputs a stream.  Each stream fills the rows that it appends, after some tens of
    milliseconds of other work: a call that went to another stream would take what stood there before."""
    rng = np.random.default_rng(t)
    n_pages = -(-t // page) + 1
    streams = [torch.cuda.Stream() for _ in range(2)]
    sides = []
    for s in streams:
        slots = (rng.permutation(n_pages)[np.arange(t) // page] * page + np.arange(t) % page).astype(np.int64)
        k, v = _kv4.bf16(rng, (t, hkv, dim)), _kv4.bf16(rng, (t, hkv, dim), 3.0)
        pool = torch.full((n_pages, hkv, _kv8.record_bytes(page, dim)), 0xFF, dtype=torch.uint8, device="cuda")
        sides.append(dict(s=s, slots=slots, k=k, v=v, pool=pool, c=hs.make_kv8_cache(pool, n_pages, page, hkv, dim),
                          on=torch.from_numpy(slots).cuda(), src=(k.cuda(), v.cuda()), rows=[torch.zeros_like(k, device="cuda") for _ in range(2)],
                          out=[torch.zeros_like(k, device="cuda") for _ in range(2)], f32=[torch.zeros(k.shape, device="cuda") for _ in range(2)]))
    torch.cuda.synchronize()
    for x in sides:
        with torch.cuda.stream(x["s"]):
            torch.cuda._sleep(50_000_000)
            for row, src in zip(x["rows"], x["src"]):
                row.copy_(src)
    for x in sides:
        hs.hs_kv8_append(x["c"], *x["rows"], x["on"], t, stream=x["s"])
    for x in sides:
        hs.hs_kv8_read(x["c"], x["on"], t, *x["out"], *x["f32"], stream=x["s"])
    torch.cuda.synchronize()
    for x in sides:
        want = np.full(x["pool"].shape, 0xFF, np.uint8)
        _kv8.append(want, page, dim, x["slots"], x["k"].float().numpy(), x["v"].float().numpy())
        assert np.array_equal(x["pool"].cpu().numpy(), want)
        for i, ref in enumerate(_kv8.read(want, page, dim, x["slots"])):
            assert np.array_equal(x["f32"][i].cpu().numpy(), ref) and np.array_equal(x["out"][i].double().cpu().numpy(), ref)


@pytest.mark.parametrize("new", [1, 40])
def test_a_step_on_the_current_stream_and_on_a_named_one(new):
    """Append, read and attention in turn, without a stream's name (the current one) and with it, give the same."""
    page, hkv, hq, dim, length = 32, 2, 8, 128, 200
    rng = np.random.default_rng(new)
    k, v, q = _kv4.bf16(rng, (length, hkv, dim)), _kv4.bf16(rng, (length, hkv, dim)), _kv4.bf16(rng, (new, hq, dim))
    n_pages = -(-length // page)
    table = torch.from_numpy(rng.permutation(n_pages).astype(np.int32)).cuda().view(1, n_pages)
    slots = table[0].long()[torch.arange(length, device="cuda") // page] * page + torch.arange(length, device="cuda") % page
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    starts, lens = i32([0, new]), i32([length])
    got = []
    for named in (False, True):
        pool = torch.zeros((n_pages, hkv, _kv8.record_bytes(page, dim)), dtype=torch.uint8, device="cuda")
        c = hs.make_kv8_cache(pool, n_pages, page, hkv, dim)
        ws = torch.zeros(hs.hs_kv8_attention_workspace_size(c, 1, hq), dtype=torch.uint8, device="cuda")
        rows = [torch.zeros_like(x, device="cuda") for x in (k, v, q)]
        out, back = torch.zeros_like(rows[2]), torch.zeros(k.shape, device="cuda")
        src = [x.cuda() for x in (k, v, q)]
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(50_000_000)
            for row, x in zip(rows, src):
                row.copy_(x)
            if not named:
                hs.hs_kv8_append(c, rows[0], rows[1], slots, length)
                hs.hs_kv8_attention(c, rows[2], starts, lens, table, 1, new, 0.09, 0, out, ws)
                hs.hs_kv8_read(c, slots, length, v_f32=back)
        if named:
            hs.hs_kv8_append(c, rows[0], rows[1], slots, length, stream=s)
            hs.hs_kv8_attention(c, rows[2], starts, lens, table, 1, new, 0.09, 0, out, ws, stream=s)
            hs.hs_kv8_read(c, slots, length, v_f32=back, stream=s)
        torch.cuda.synchronize()
        got.append((pool, out, back))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    kk, vv = _kv8.values(k.float().numpy()), _kv8.values(v.float().numpy())
    assert np.array_equal(got[0][2].cpu().numpy(), vv)
    ref = _kv4.attention(q.double().numpy(), kk, vv, new, length, 0.09)
    # half a step of bf16, probabilities to fp16, scores: as tests/test_gpu_kv8.py's _close
    assert (np.abs(got[0][1].double().cpu().numpy() - ref) <= np.abs(ref) * 2.0 ** -8 + np.abs(vv).max() * (2.0 ** -11 + 2 * 2.0 ** -13 + 2.0 ** -20)).all()
