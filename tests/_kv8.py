"""Plain 64-bit restatement of the 8-bit key/value cache for its tests (numpy,
no code shared with the library), and builders of caches on the GPU."""
import math

import numpy as np
import torch

import _kv4

LARGEST, LOW, HIGH, BLOCK = 57344.0, -15, 7, 16


def _table():
    out = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        x = math.ldexp(1 + m / 8, e - 7) if e else math.ldexp(m, -9)
        out.append(math.nan if b & 127 == 127 else -x if b & 128 else x)
    return np.array(out)


TABLE = _table()          # what each byte stands for


def codes_of(y):
    """Bytes of e4m3 next to values of at most 448 (ties: the even one)."""
    y = np.asarray(y, np.float64)
    a, up = np.abs(y), TABLE[:127]
    lo = np.clip(np.searchsorted(up, a, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    d, u = a - up[lo], up[hi] - a
    pick = np.where((u < d) | ((u == d) & (lo % 2 == 1)), hi, lo).astype(np.uint8)
    return pick | np.where(np.signbit(y), 128, 0).astype(np.uint8)


def exponent(largest):
    for e in range(LOW, HIGH + 1):
        if largest <= 448 * 2.0 ** e:
            return e
    raise ValueError(largest)


def record_bytes(page, dim):
    return page * (2 * dim + 1)


def places(o, dim):
    turn = ((2 * (o % 4)) ^ (o & 4)) if dim == 128 else o & 2
    d = np.arange(dim)
    return ((d // 16) ^ turn) * 16 + d % 16


def _scale_at(page, dim, o, i):
    return 2 * page * dim + o // BLOCK * 16 + 4 * i


def append(pool, page, dim, slots, k, v):
    """Tokens into a numpy pool [n_pages][heads][record], block by block (see hs_kv8_append)."""
    n_pages, heads, _ = pool.shape
    slots = [int(s) if 0 <= int(s) < n_pages * page else -1 for s in slots]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        end = t
        while end < len(slots) and slots[end] >= 0 and slots[end] // BLOCK == slots[t] // BLOCK:
            end += 1
        p, base = divmod(slots[t] // BLOCK * BLOCK, page)
        off = [s % BLOCK for s in slots[t:end]]
        for i, x in enumerate((k, v)):
            x = np.asarray(x[t:end], np.float64)
            with np.errstate(invalid="ignore"):
                bad = (~(np.abs(x) <= LARGEST)).reshape(*x.shape[:-1], -1, 64).any(-1).repeat(64, -1)
            fine = np.where(bad, 0, x)
            at = _scale_at(page, dim, base, i)
            for h in range(heads):
                rec = pool[p, h]
                e = exponent(np.abs(fine[:, h]).max())
                if min(off):
                    old = int(round(math.log2(rec[at:at + 4].view(np.float32)[0])))
                    e = max(e, old)
                    for o in range(min(off) if e > old else 0):
                        where = i * page * dim + (base + o) * dim + np.arange(dim)
                        c = TABLE[rec[where]] * 2.0 ** (old - e)
                        rec[where] = np.where(np.isnan(c), 0x7F, codes_of(np.nan_to_num(c)))
                for j, o in enumerate(off):
                    c = np.where(bad[j, h], 0x7F, codes_of(fine[j, h] * 2.0 ** -e))
                    rec[i * page * dim + (base + o) * dim + places(base + o, dim)] = c
                rec[at:at + 4] = np.array([2.0 ** e], np.float32).view(np.uint8)
                rec[_scale_at(page, dim, base, 2):_scale_at(page, dim, base, 4)] = 0
        t = end
    return pool


def read(pool, page, dim, slots):
    """Keys and values of slots in 64 bits, [tokens][heads][dim]; zeros outside the pool."""
    n_pages, heads, _ = pool.shape
    out = np.zeros((2, len(slots), heads, dim))
    for t, s in enumerate(slots):
        if not 0 <= int(s) < n_pages * page:
            continue
        p, o = divmod(int(s), page)
        for i in range(2):
            at = _scale_at(page, dim, o, i)
            scale = np.ascontiguousarray(pool[p, :, at:at + 4]).view(np.float32).astype(np.float64)
            out[i, t] = TABLE[pool[p][:, i * page * dim + o * dim + places(o, dim)]] * scale
    return out[0], out[1]


class Requests(_kv4.Requests):
    """As _kv4.Requests over the 8-bit cache: everything that no request owns is 0xFF
    (NaN codes, NaN scales)."""

    def __init__(self, seed, cached, new, hq, hkv, dim, page, spare=3, k_size=1.0, v_size=1.0, edit=None):
        rng = np.random.default_rng(seed)
        self.new, self.len = list(new), [c + n for c, n in zip(cached, new)]
        self.hq, self.hkv, self.dim, self.page, n = hq, hkv, dim, page, len(self.len)
        used = [-(-length // page) for length in self.len]
        self.n_pages = sum(used) + spare
        perm = rng.permutation(self.n_pages)
        self.width = max(max(used), 1)
        self.table = np.full((n, self.width), -1, np.int32)
        pool = np.full((self.n_pages, hkv, record_bytes(page, dim)), 0xFF, np.uint8)
        self.k, self.v, at = [], [], 0
        for i, length in enumerate(self.len):
            self.table[i, :used[i]] = perm[at:at + used[i]]
            at += used[i]
            k, v = (_kv4.bf16(rng, (length, hkv, dim), s).float().numpy() for s in (k_size, v_size))
            if edit:
                edit(i, k, v)
            j = np.arange(length)
            where = self.table[i, j // page].astype(np.int64) * page + j % page
            fill(pool, page, dim, where, k, v)
            k, v = values(k), values(v)
            self.k.append(k)
            self.v.append(v)
        self.pool_np = pool
        self.q = _kv4.bf16(rng, (sum(self.new), hq, dim))
        self.starts = np.concatenate(([0], np.cumsum(self.new))).astype(np.int32)

    def run(self, hs, scale, window=0, max_new=None, q=None, out=None, table=None, stream=None, ws=None):
        dev = "cuda"
        self.pool = torch.from_numpy(self.pool_np).to(dev)
        cache = hs.make_kv8_cache(self.pool, self.n_pages, self.page, self.hkv, self.dim)
        n = len(self.len)
        q = self.q.to(dev) if q is None else q
        out = torch.full_like(q, float("nan")) if out is None else out
        if ws is None:
            ws = torch.zeros(hs.hs_kv8_attention_workspace_size(cache, n, self.hq), dtype=torch.uint8, device=dev)
        table = torch.from_numpy(self.table).to(dev) if table is None else table
        hs.hs_kv8_attention(cache, q, torch.from_numpy(self.starts).to(dev),
                            torch.tensor(self.len, dtype=torch.int32, device=dev), table, n,
                            max(self.new + [0]) if max_new is None else max_new, scale, window, out, ws, stream=stream)
        torch.cuda.synchronize()
        assert hs.hs_device_status() == hs.HS_OK
        return out


def _blocks(x):
    """A request's tokens [length][heads][dim] appended in one call: codes and each
    token's scale exponent [length][heads]."""
    x = np.asarray(x, np.float64)
    n, heads, dim = x.shape
    with np.errstate(invalid="ignore"):
        bad = (~(np.abs(x) <= LARGEST)).reshape(n, heads, -1, 64).any(-1).repeat(64, -1)
    fine = np.where(bad, 0, x)
    pad = -n % BLOCK
    most = np.concatenate((np.abs(fine).max(-1), np.zeros((pad, heads)))).reshape(-1, BLOCK, heads).max(1)
    e = np.full(most.shape, LOW)
    for k in range(LOW, HIGH):
        e += most > 448 * 2.0 ** k
    e = e.repeat(BLOCK, 0)[:n]
    return np.where(bad, 0x7F, codes_of(fine * 2.0 ** -e[..., None])).astype(np.uint8), e


def values(x):
    """What a reader gets for a request's tokens that were appended in one call."""
    if not len(x):
        return np.zeros(x.shape)
    codes, e = _blocks(x)
    return TABLE[codes] * 2.0 ** e[..., None]


def fill(pool, page, dim, slots, k, v):
    """As append, of a whole request at once (its slots in order, from a block's start on)."""
    if not len(slots):
        return
    page_of, o = np.asarray(slots) // page, np.asarray(slots) % page
    at = np.stack([places(x, dim) for x in o]) + o[:, None] * dim
    for i, x in enumerate((k, v)):
        codes, e = _blocks(x)
        for h in range(pool.shape[1]):
            pool[page_of[:, None], h, i * page * dim + at] = codes[:, h]
            b = (2.0 ** e[:, h]).astype(np.float32)[:, None].view(np.uint8)
            pool[page_of[:, None], h, _scale_at(page, dim, o, i)[:, None] + np.arange(4)] = b
            pool[page_of[:, None], h, _scale_at(page, dim, o, 2)[:, None] + np.arange(8)] = 0
