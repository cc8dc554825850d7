"""Plain 64-bit restatement of the 4-bit key/value cache for its tests (numpy,
no code shared with the library), and builders of caches on either device."""
import numpy as np
import torch


def quantise(x):
    """Codes, scale, bias of groups of 64 along the last axis: the definition's
    fp32 steps (numpy float32 rounds each operation to nearest even)."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    with np.errstate(all="ignore"):
        scale = ((hi - lo) / np.float32(15)).astype(np.float16)
        bias = lo.astype(np.float16)
        s, b = scale.astype(np.float32), bias.astype(np.float32)
        codes = np.where(s > 0, np.clip(np.rint((g - b) / s), 0, 15), 0)
    bad = ~((np.abs(lo) < 65536) & (np.abs(hi) < 65536))
    scale = np.where(bad, np.float16(0), scale)
    bias = np.where(bad, np.float16("nan"), bias)
    codes = np.where(bad, 0, codes)
    return codes.reshape(x.shape).astype(np.uint8), scale[..., 0], bias[..., 0]


def values(x):
    """What a reader of the cache gets for x, exact in 64 bits."""
    codes, scale, bias = quantise(x)
    c = codes.astype(np.float64).reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    return (scale.astype(np.float64)[..., None] * c + bias.astype(np.float64)[..., None]).reshape(x.shape)


def record_bytes(page, dim):
    return page * dim + page * (dim // 64) * 8


def fill_pool(pool, page, dim, slots, k, v):
    """Writes tokens into a numpy pool [n_pages][heads][record] as declared in hs.h."""
    half, pairs = page * dim // 2, page * (dim // 64) * 4
    for i, x in enumerate((k, v)):
        codes, scale, bias = quantise(x)
        packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
        sb = np.stack((scale, bias), -1).reshape(*scale.shape[:-1], 2 * scale.shape[-1]).view(np.uint8)
        for t, s in enumerate(slots):
            if s < 0:
                continue
            p, o = divmod(int(s), page)
            pool[p, :, i * half + o * (dim // 2):i * half + (o + 1) * (dim // 2)] = packed[t]
            n = dim // 64 * 4
            at = 2 * half + i * pairs + o * n
            pool[p, :, at:at + n] = sb[t]
    return pool


def attention(q, k, v, new, length, scale, window=0, present=None):
    """One request in 64 bits: q [new][hq][dim], k and v [length][hkv][dim] fp64
    values; present: truth per key (False: its page is not there)."""
    group = q.shape[1] // k.shape[1]
    out = np.zeros(q.shape, np.float64)
    for i in range(new):
        p = length - new + i
        lo = max(0, p - window + 1) if window else 0
        seen = np.arange(lo, p + 1) if p >= lo else np.zeros(0, np.int64)
        if present is not None and len(seen):
            seen = seen[present[seen]]
        if not len(seen):
            continue
        for h in range(q.shape[1]):
            s = (k[seen, h // group] @ q[i, h].astype(np.float64)) * scale
            e = np.exp(s - s.max())
            out[i, h] = (e / e.sum()) @ v[seen, h // group]
    return out


def plan(cached, new, page, n_pages, table, ring, counters, max_tokens):
    """The step plan, request by request (see hs_kv4_plan)."""
    n, width = table.shape
    table, ring = table.copy(), ring.copy()
    head, tail = int(counters[0]), int(counters[1])
    c = [max(int(x), 0) for x in cached]
    up = lambda x: -(-x // page)  # noqa: E731
    need = sum(up(c[i] + int(new[i])) - up(c[i]) for i in range(n) if new[i] >= 0)
    over = sum(max(0, up(c[i] + int(new[i])) - width) for i in range(n) if new[i] >= 0)
    tokens = sum(int(x) for x in new if x > 0)
    short = over + max(0, need - (tail - head)) + max(0, tokens - max_tokens)
    starts, seq, slots, pos = [0], [], [], []
    out = np.full_like(table, -1)
    for i in range(n):
        have = up(c[i])
        if new[i] < 0:
            for w in range(have):
                ring[tail % n_pages] = table[i, w]
                tail += 1
            seq.append(0)
            starts.append(starts[-1])
            continue
        out[i, :have] = table[i, :have]
        fresh = int(new[i]) if not short else 0
        for w in range(have, up(c[i] + fresh)):
            out[i, w] = ring[head % n_pages]
            head += 1
        for p in range(c[i], c[i] + fresh):
            slots.append(int(out[i, p // page]) * page + p % page)
            pos.append(p)
        seq.append(c[i] + fresh)
        starts.append(starts[-1] + fresh)
    pad = [-1] * (max_tokens - len(slots))
    return dict(table=out, ring=ring, counters=[head, tail], seq_len=seq, q_start=starts, slot=slots + pad,
                position=pos + pad, short=short)


def bf16(rng, shape, size=1.0):
    return torch.from_numpy(rng.normal(0, size, shape).astype(np.float32)).bfloat16()


class Requests:
    """A cache on the GPU holding requests of given lengths, its pages in a
    random order, everything that no request owns set to 0xFF (NaN pairs)."""

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
            k, v = (bf16(rng, (length, hkv, dim), s).float().numpy() for s in (k_size, v_size))
            if edit:
                edit(i, k, v)
            if length:
                where = self.table[i, np.arange(length) // page].astype(np.int64) * page + np.arange(length) % page
                fill_pool(pool, page, dim, where, k, v)
            self.k.append(values(k))
            self.v.append(values(v))
        self.pool_np = pool
        self.q = bf16(rng, (sum(self.new), hq, dim))
        self.starts = np.concatenate(([0], np.cumsum(self.new))).astype(np.int32)

    def expected(self, scale, window=0, present=None):
        q = self.q.double().numpy()
        return np.concatenate([attention(q[self.starts[i]:self.starts[i + 1]], self.k[i], self.v[i], self.new[i],
                                         self.len[i], scale, window, None if present is None else present[i])
                               for i in range(len(self.len))])

    def run(self, hs, scale, window=0, max_new=None, q=None, out=None, table=None, stream=None, ws=None):
        dev = "cuda"
        self.pool = torch.from_numpy(self.pool_np).to(dev)
        cache = hs.make_kv4_cache(self.pool, self.n_pages, self.page, self.hkv, self.dim)
        n = len(self.len)
        q = self.q.to(dev) if q is None else q
        out = torch.full_like(q, float("nan")) if out is None else out
        if ws is None:
            ws = torch.zeros(hs.hs_kv4_attention_workspace_size(cache, n, self.hq), dtype=torch.uint8, device=dev)
        table = torch.from_numpy(self.table).to(dev) if table is None else table
        hs.hs_kv4_attention(cache, q, torch.from_numpy(self.starts).to(dev),
                            torch.tensor(self.len, dtype=torch.int32, device=dev), table, n,
                            max(self.new + [0]) if max_new is None else max_new, scale, window, out, ws, stream=stream)
        torch.cuda.synchronize()
        assert hs.hs_device_status() == hs.HS_OK
        return out
