"""The 4-bit key/value cache operators on real work: their cases, plain forms and 64-bit definitions.

The cache holds one attention layer's keys and values in pages of `page` tokens.  One (page, kv head)
record holds, in this order, K codes [page][dim/2], V codes [page][dim/2], K (scale, bias) fp16 pairs
[page][dim/64] and V pairs [page][dim/64]; two codes a byte, the even channel in the low nibble; a group of
64 channels of one token stands for scale * code + bias.  The pool is [pages][kv heads][record].  A token's
slot is page * page_tokens + offset, -1 for none.

Three passes are measured:
  plan       block tables, slot map, positions and row starts of one step, from the requests' lengths
  append     new keys and values into their slots (4 bits), and those slots read back (bf16)
  attention  causal attention of each request's newest tokens over its cached keys and values
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of eight requests: every request gets one token, a few get a new page
        {"name": "plan-step-8", "op": "plan", "requests": 8, "page": 64, "width": 64, "pattern": "step", "lens": 1},
        # a large scheduler's step: half decode, some prompts come in, some requests end
        {"name": "plan-mixed-1000", "op": "plan", "requests": 1000, "page": 16, "width": 515, "pattern": "mixed",
         "lens": 2},
        # one token of one sequence: the smallest write there is, latency counts
        {"name": "append-1", "op": "append", "tokens": 1, "hkv": 2, "dim": 128, "page": 64, "strided": False},
        # a decode batch of 64 (the largest decode batch of this library), K and V cut out of a fused projection
        {"name": "append-64", "op": "append", "tokens": 64, "hkv": 8, "dim": 64, "page": 16, "strided": True},
        # the library's largest prompt chunk, doubled, over 8 heads: bandwidth counts
        {"name": "append-8191", "op": "append", "tokens": 8191, "hkv": 8, "dim": 128, "page": 64, "strided": False},
        # the first steps of one conversation: a handful of cached tokens, nothing but latency
        {"name": "decode-1x77", "op": "attention", "requests": 1, "new": 1, "ctx": 77, "ragged": False, "hq": 32, "hkv": 2,
         "dim": 128, "page": 64, "window": 0, "lens": 3},
        # one user with a very long context: the key axis has to be split
        {"name": "decode-1x131071", "op": "attention", "requests": 1, "new": 1, "ctx": 131071, "ragged": False, "hq": 32,
         "hkv": 2, "dim": 128, "page": 64, "window": 0, "lens": 4},
        # a full decode batch of unequal requests
        {"name": "decode-64-ragged", "op": "attention", "requests": 64, "new": 1, "ctx": 8192, "ragged": True, "hq": 32,
         "hkv": 8, "dim": 128, "page": 64, "window": 0, "lens": 5},
        # a sliding-window layer with narrow heads and small pages
        {"name": "decode-33-window", "op": "attention", "requests": 33, "new": 1, "ctx": 6000, "ragged": True, "hq": 24,
         "hkv": 4, "dim": 64, "page": 16, "window": 1000, "lens": 6},
        # verification of two drafted tokens and the next one (3 rows of each sequence)
        {"name": "verify-16x3", "op": "attention", "requests": 16, "new": 3, "ctx": 4096, "ragged": True, "hq": 32,
         "hkv": 2, "dim": 128, "page": 32, "window": 0, "lens": 7},
        # prompt chunks of several requests behind contexts of unequal lengths
        {"name": "chunk-5-ragged", "op": "attention", "requests": 5, "new": 1111, "ctx": 5000, "ragged": True, "hq": 28,
         "hkv": 4, "dim": 128, "page": 64, "window": 0, "lens": 8},
        # the library's largest prompt chunk from an empty cache
        {"name": "prompt-4096", "op": "attention", "requests": 1, "new": 4096, "ctx": 0, "ragged": False, "hq": 32,
         "hkv": 8, "dim": 128, "page": 64, "window": 0, "lens": 9},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["plan", "append", "decode", "decode", "verify", "chunk", "chunk"])
    page, lens = rng.choice([16, 32, 64]), rng.randrange(1 << 30)
    if kind == "plan":
        return {"op": "plan", "requests": _log_int(rng, 1, 1000), "page": page, "width": rng.randint(64, 600),
                "pattern": rng.choice(["step", "mixed"]), "lens": lens}
    hkv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if kind == "append":
        return {"op": "append", "tokens": _log_int(rng, 1, 8191), "hkv": hkv, "dim": dim, "page": page,
                "strided": rng.random() < 0.5}
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    group = min(group, 32 // hkv)
    new = {"decode": 1, "verify": rng.randint(2, 8), "chunk": _log_int(rng, 9, 4096)}[kind]
    requests = _log_int(rng, 1, 64 if new < 9 else 8)
    # the plain form pads to the longest request: its scores and its rows stay within the largest listed cases'
    requests = max(1, min(requests, 4096 // new)) if new >= 9 else requests
    most = min(131071, 64 * 8192 * 8 * 128 // (requests * hkv * dim), 32 * 4096 * 4096 // (requests * new * hkv * group) - new)
    ctx = _log_int(rng, 1, max(1, most)) if rng.random() < 0.9 else 0
    window = 0 if rng.random() < 0.75 else _log_int(rng, 1, 4096)
    return {"op": "attention", "requests": requests, "new": new, "ctx": ctx, "ragged": rng.random() < 0.7,
            "hq": hkv * group, "hkv": hkv, "dim": dim, "page": page, "window": window, "lens": lens}


def _lengths(case):
    """Cached and new tokens of each request (numpy int64), from the case alone."""
    r = np.random.default_rng(case["lens"])
    n = case["requests"]
    if case["op"] == "plan":
        longest = (case["width"] - 1) * case["page"]
        cached = r.integers(0, max(1, longest // 2), n)
        new = np.ones(n, np.int64)
        if case["pattern"] == "mixed":
            what = r.random(n)
            prompt = what < 0.1
            cached[prompt] = 0
            new[prompt] = r.integers(1, min(700, longest), int(prompt.sum()))
            new[(what >= 0.1) & (what < 0.2)] = -1
            new[(what >= 0.2) & (what < 0.3)] = 0
        return cached, new
    cached = np.full(n, case["ctx"], np.int64)
    new = np.full(n, case["new"], np.int64)
    if case["ragged"]:
        cached = r.integers(case["ctx"] // 16, case["ctx"] + 1, n)
        cached[0] = case["ctx"]
        if case["new"] > 8:
            new = r.integers(1, case["new"] + 1, n)
            new[0] = case["new"]
    return cached, new


def _visible(case):
    """Keys each new token may look at, over all new tokens, and cached rows any of them looks at, per request."""
    cached, new = _lengths(case)
    pairs = rows = 0
    for c, n in zip(cached.tolist(), new.tolist()):
        seen = np.arange(c + 1, c + n + 1)
        lo = np.maximum(0, seen - case["window"]) if case["window"] else np.zeros_like(seen)
        pairs += int((seen - lo).sum())
        rows += int(c + n - lo[0]) if n else 0
    return pairs, rows, int(new.sum())


def work(case):
    if case["op"] == "plan":
        n, p, w = case["requests"], case["page"], case["width"]
        cached, new = _lengths(case)
        tokens = int(new.clip(0).sum())
        # lengths in, old and new table, row starts and lengths out, slot (8 bytes) and position (4) a token
        return {"bytes": 8 * n + 8 * n * w + 8 * n + 12 * _capacity(tokens), "flops": 0}
    if case["op"] == "append":
        t, values = case["tokens"], 2 * case["tokens"] * case["hkv"] * case["dim"]
        # bf16 in, codes and pairs written, read back, bf16 out
        return {"bytes": 4 * values + 2 * (values // 2 + values // 16) + 8 * t, "flops": 8 * values}
    pairs, rows, tokens = _visible(case)
    row = 2 * case["hkv"] * (case["dim"] // 2 + case["dim"] // 16)
    return {"bytes": rows * row + 4 * tokens * case["hq"] * case["dim"] + 4 * (rows // case["page"] + 1),
            "flops": 4 * case["dim"] * case["hq"] * pairs}


# --------------------------------------------------------------------------------------------- inputs
def _capacity(tokens):
    """Tokens a step's buffers are padded to (captured graphs run at fixed sizes)."""
    return -(-max(tokens, 1) // 64) * 64


def _quantise(x):
    """fp32 [..., dim] to codes [..., dim] (0..15) and fp16 scale, bias [..., dim / 64]."""
    g = x.unflatten(-1, (-1, 64))
    lo, hi = g.amin(-1), g.amax(-1)
    scale = ((hi - lo) / 15).half()
    bias = lo.half()
    s, b = scale.float()[..., None], bias.float()[..., None]
    codes = torch.where(s > 0, ((g - b) / s).round().clamp(0, 15), torch.zeros_like(g))
    return codes.flatten(-2), scale, bias


def _pack(codes):
    c = codes.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _kv(shape, gen):
    """Keys or values as a projection leaves them: normal, some channels several times larger."""
    x = torch.randn(shape, generator=gen, device="cuda")
    size = torch.exp(0.5 * torch.randn(shape[-2:], generator=gen, device="cuda"))
    return (x * size).bfloat16()


def _record(case):
    return case["page"] * case["dim"] + case["page"] * case["dim"] // 64 * 8


def _fill(pool, case, pages, k, v):
    """Writes whole pages: k, v fp32 [n, page, hkv, dim] into the records of `pages`; NaN where a value is NaN."""
    half, pairs = case["page"] * case["dim"] // 2, case["page"] * case["dim"] // 64 * 4
    for i, x in enumerate((k, v)):
        none = torch.isnan(x[..., 0])
        codes, scale, bias = _quantise(torch.nan_to_num(x))
        bias = torch.where(none[..., None], torch.full_like(bias, float("nan")), bias)
        packed = _pack(codes).permute(0, 2, 1, 3).flatten(2)
        sb = torch.stack((scale, bias), -1).permute(0, 2, 1, 3, 4).flatten(2).contiguous().view(torch.uint8)
        pool[pages, :, i * half:(i + 1) * half] = packed
        pool[pages, :, 2 * half + i * pairs:2 * half + (i + 1) * pairs] = sb


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = torch.device("cuda")
    state = {"case": case, "buffers": {}}
    if case["op"] == "plan":
        cached, new = (torch.from_numpy(a) for a in _lengths(case))
        # other lengths for another seed, of the same sizes: the requests in another order
        order = torch.randperm(case["requests"], generator=torch.Generator().manual_seed(seed))
        cached, new = cached[order].to(dev, torch.int32), new[order].to(dev, torch.int32)
        p, w = case["page"], case["width"]
        have = (cached + p - 1) // p
        need = int((torch.where(new > 0, cached + new + p - 1, 0) // p - have).clamp(min=0).sum())
        held = int(have.sum())
        n_pages = held + need + 37
        perm = torch.randperm(n_pages, generator=gen, device=dev).int()
        table = torch.full((case["requests"], w), -1, dtype=torch.int32, device=dev)
        cols = torch.arange(w, device=dev)
        table[cols < have[:, None]] = perm[:held]
        head = int(torch.randint(1, 3 * n_pages, (1,), generator=gen, device=dev))
        at = (head + torch.arange(n_pages - held, device=dev)) % n_pages
        ring = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        ring[at] = perm[held:]
        state.update(cached=cached, new=new, table=table, ring=ring, n_pages=n_pages,
                     counters=torch.tensor([head, head + n_pages - held], dtype=torch.int64, device=dev),
                     capacity=_capacity(int(new.clamp(min=0).sum())))
        return state
    if case["op"] == "append":
        t, h, d, p = case["tokens"], case["hkv"], case["dim"], case["page"]
        n_pages = -(-t // p) + 5
        if case["strided"]:  # columns of a fused query-key-value projection
            fused = torch.randn((t, (2 * h + 5) * d), generator=gen, device=dev).bfloat16()
            k = fused[:, 3 * d:(3 + h) * d].unflatten(1, (h, d))
            v = fused[:, (3 + h) * d:(3 + 2 * h) * d].unflatten(1, (h, d))
        else:
            k, v = _kv((t, h, d), gen), _kv((t, h, d), gen)
        pages = torch.randperm(n_pages, generator=gen, device=dev)[:-(-t // p)]
        at = torch.arange(t, device=dev)
        state.update(k=k, v=v, slots=pages[at // p] * p + at % p, n_pages=n_pages,
                     pool=torch.zeros((n_pages, h, _record(case)), dtype=torch.uint8, device=dev))
        return state
    cached, new = _lengths(case)
    h, d, p = case["hkv"], case["dim"], case["page"]
    lens = torch.from_numpy(cached + new).to(dev)
    width = int((lens.max() + p - 1) // p)
    used = (lens + p - 1) // p
    held = int(used.sum())
    n_pages = held + 3
    pool = torch.full((n_pages, h, _record(case)), 0xFF, dtype=torch.uint8, device=dev)
    perm = torch.randperm(n_pages, generator=gen, device=dev)[:held].int()
    table = torch.full((case["requests"], width), -1, dtype=torch.int32, device=dev)
    cols = torch.arange(width, device=dev)
    table[cols < used[:, None]] = perm
    # tokens of each held page that its request has filled; the rest of a last page holds NaN
    full = (lens[:, None] - cols * p).clamp(0, p)[cols < used[:, None]]
    step = max(1, (1 << 26) // (p * h * d))
    for a in range(0, held, step):
        n = min(step, held - a)
        k, v = (_kv((n, p, h, d), gen).float() for _ in range(2))
        gone = torch.arange(p, device=dev) >= full[a:a + n, None]
        nan = torch.full((), float("nan"), device=dev)
        _fill(pool, case, perm[a:a + n].long(), torch.where(gone[..., None, None], nan, k),
              torch.where(gone[..., None, None], nan, v))
    tokens = int(new.sum())
    starts = torch.zeros(case["requests"] + 1, dtype=torch.int32, device=dev)
    starts[1:] = torch.from_numpy(new).to(dev).cumsum(0)
    q = torch.randn((tokens, case["hq"], d), generator=gen, device=dev).bfloat16()
    state.update(q=q, starts=starts, seq_len=lens.int(), table=table, pool=pool, n_pages=n_pages, tokens=tokens,
                 max_new=int(new.max()), scale=1.0 / math.sqrt(d))
    return state


# ----------------------------------------------------------------------------------------- plain forms
def _plan(s):
    case, dev = s["case"], s["cached"].device
    p, w, n_pages = case["page"], case["width"], s["n_pages"]
    cached, ended, new = s["cached"].clamp(min=0).long(), s["new"] < 0, s["new"].clamp(min=0).long()
    table, ring = s["table"], s["ring"].clone()
    head, tail = s["counters"][0], s["counters"][1]
    have = (cached + p - 1) // p
    want = torch.where(ended, have, (cached + new + p - 1) // p)
    need = want - have
    short = (want - w).clamp(min=0).sum() + (need.sum() - (tail - head)).clamp(min=0)
    ok = short == 0
    need, new = need * ok, new * ok
    want = torch.minimum(have + need, torch.full_like(have, w))
    before = need.cumsum(0) - need
    cols = torch.arange(w, device=dev)
    fresh = ring[(head + before[:, None] + cols - have[:, None]).clamp(min=0) % n_pages]
    out = torch.where(cols < have[:, None], table, torch.where(cols < want[:, None], fresh, torch.full_like(table, -1)))
    out = torch.where(ended[:, None], torch.full_like(out, -1), out)
    seq_len = torch.where(ended, torch.zeros_like(cached), cached + new)
    starts = torch.cat((new.new_zeros(1), new.cumsum(0)))
    j = torch.arange(s["capacity"], device=dev)
    r = torch.searchsorted(starts[1:], j, right=True).clamp(max=case["requests"] - 1)
    live = j < starts[-1]
    pos = cached[r] + j - starts[r]
    page = out[r, (pos // p).clamp(0, w - 1)].long()
    none = torch.full_like(pos, -1)
    slot = torch.where(live & (page >= 0), page * p + pos % p, none)
    pos = torch.where(live, pos, none)
    # pages of ended requests go to the ring's tail, request by request
    back = torch.where(ended, have, torch.zeros_like(have))
    gone = ended[:, None] & (cols < have[:, None])
    at = (tail + (back.cumsum(0) - back)[:, None] + cols) % n_pages
    spare = torch.cat((ring, ring.new_zeros(1)))
    spare[torch.where(gone, at, torch.full_like(at, n_pages))] = table
    counters = torch.stack((head + need.sum(), tail + back.sum()))
    return {"table": out, "seq_len": seq_len.int(), "starts": starts.int(), "slot": slot, "position": pos.int(),
            "ring": spare[:-1], "counters": counters, "short": short.int().reshape(1)}


def _append(s):
    case, pool = s["case"], s["pool"]
    p, d = case["page"], case["dim"]
    half, pairs = p * d // 2, p * d // 64 * 4
    page, off = s["slots"] // p, s["slots"] % p
    codes_at = torch.arange(d // 2, device=pool.device) + off[:, None] * (d // 2)
    pairs_at = torch.arange(d // 16, device=pool.device) + off[:, None] * (d // 16)
    heads = torch.arange(case["hkv"], device=pool.device)[None, :, None]
    out = {}
    for i, name in enumerate("kv"):
        codes, scale, bias = _quantise(s[name].float())
        at = (page[:, None, None], heads, i * half + codes_at[:, None])
        sb_at = (page[:, None, None], heads, 2 * half + i * pairs + pairs_at[:, None])
        pool[at] = _pack(codes)
        pool[sb_at] = torch.stack((scale, bias), -1).flatten(-2).view(torch.uint8)
        out[name] = _value(pool[at], pool[sb_at].view(torch.half)).bfloat16()
    return out


def _value(packed, sb):
    """Packed codes [..., dim/2] and fp16 pairs [..., dim/32] to fp32 values [..., dim]."""
    codes = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).float().unflatten(-1, (-1, 64))
    sb = sb.float().unflatten(-1, (-1, 2))
    return (sb[..., 0:1] * codes + sb[..., 1:2]).flatten(-2)


def _attention(s):
    case, pool, dev = s["case"], s["pool"], s["pool"].device
    p, d, h, n = case["page"], case["dim"], case["hkv"], case["requests"]
    group, rows = case["hq"] // h, s["max_new"]
    half, pairs = p * d // 2, p * d // 64 * 4
    rec = pool[s["table"].clamp(min=0).long()]  # [n, width, h, record], padded to the longest request
    length = rec.shape[1] * p
    key = torch.arange(length, device=dev)
    held = (key < s["seq_len"][:, None])[:, None, :, None]

    def rows_of(i):
        packed = rec[..., i * half:(i + 1) * half].unflatten(-1, (p, d // 2))
        sb = rec[..., 2 * half + i * pairs:2 * half + (i + 1) * pairs].contiguous().view(torch.half).unflatten(-1, (p, d // 32))
        x = _value(packed, sb).permute(0, 2, 1, 3, 4).flatten(2, 3)
        return torch.where(held, x, torch.zeros((), device=dev))

    starts = s["starts"].long()
    new = starts[1:] - starts[:-1]
    row = torch.arange(rows, device=dev)
    token = (starts[:-1, None] + row).clamp(max=s["tokens"] - 1)
    q = s["q"][token].float().unflatten(2, (h, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = torch.matmul(q, rows_of(0).transpose(-1, -2)).mul_(s["scale"]).unflatten(2, (group, rows))
    at = (s["seq_len"] - new)[:, None] + row  # position of each new token
    see = key <= at[..., None]
    if case["window"]:
        see &= key > at[..., None] - case["window"]
    score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    prob = score.sub_(top).exp_()
    total = prob.sum(-1, keepdim=True).flatten(2, 3)
    o = torch.matmul(prob.flatten(2, 3), rows_of(1))
    o = torch.where(total > 0, o / total, torch.zeros((), device=dev)).unflatten(2, (group, rows))
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [n, rows, hq, dim]
    request = torch.repeat_interleave(torch.arange(n, device=dev), new, output_size=s["tokens"])
    return o[request, torch.arange(s["tokens"], device=dev) - starts[request]].bfloat16()


# ---------------------------------------------------------------------------------------------- passes
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"plan": _plan, "append": _append, "attention": _attention}[op](state)
    from activation_sparse_moe_gb300 import hs
    s, case, keep = state, state["case"], state["buffers"]
    if op == "plan":
        n, w, dev = case["requests"], case["width"], s["table"].device
        if not keep:
            keep.update(table=torch.empty_like(s["table"]), seq_len=torch.empty(n, dtype=torch.int32, device=dev),
                        starts=torch.empty(n + 1, dtype=torch.int32, device=dev),
                        slot=torch.empty(s["capacity"], dtype=torch.int64, device=dev),
                        position=torch.empty(s["capacity"], dtype=torch.int32, device=dev),
                        counters=torch.empty_like(s["counters"]), short=torch.empty(1, dtype=torch.int32, device=dev))
        hs.hs_kv4_plan(s["cached"], s["new"], n, case["page"], s["n_pages"], s["table"], w, s["ring"], s["counters"],
                       s["capacity"], keep["table"], keep["seq_len"], keep["starts"], keep["slot"], keep["position"],
                       keep["counters"], keep["short"])
        return {"table": keep["table"], "seq_len": keep["seq_len"], "starts": keep["starts"], "slot": keep["slot"],
                "position": keep["position"], "ring": s["ring"], "counters": keep["counters"], "short": keep["short"]}
    if "cache" not in keep:
        keep["cache"] = hs.make_kv4_cache(s["pool"], s["n_pages"], case["page"], case["hkv"], case["dim"])
    if op == "append":
        if "k" not in keep:
            shape = (case["tokens"], case["hkv"], case["dim"])
            keep.update({name: torch.empty(shape, dtype=torch.bfloat16, device=s["pool"].device) for name in "kv"})
        hs.hs_kv4_append(keep["cache"], s["k"], s["v"], s["slots"], case["tokens"])
        hs.hs_kv4_read(keep["cache"], s["slots"], case["tokens"], keep["k"], keep["v"])
        return {"k": keep["k"], "v": keep["v"]}
    if "out" not in keep:
        size = hs.hs_kv4_attention_workspace_size(keep["cache"], case["requests"], case["hq"])
        keep.update(out=torch.empty_like(s["q"]), ws=torch.zeros(size, dtype=torch.uint8, device=s["pool"].device))
    hs.hs_kv4_attention(keep["cache"], s["q"], s["starts"], s["seq_len"], s["table"], case["requests"], s["max_new"],
                        s["scale"], case["window"], keep["out"], keep["ws"])
    return keep["out"]


# -------------------------------------------------------------------------------- definitions, 64 bits
def exact(case, seed):
    if case["op"] == "plan":  # whole numbers only
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        # the codes are decided in fp32 by definition; the values they stand for are exact
        out = {}
        for name in "kv":
            x = s[name].float().cpu().numpy()
            g = x.reshape(x.shape[0], x.shape[1], -1, 64)
            lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
            scale = ((hi - lo) / np.float32(15)).astype(np.float16).astype(np.float32)
            bias = lo.astype(np.float16).astype(np.float32)
            with np.errstate(divide="ignore", invalid="ignore"):
                code = np.where(scale > 0, np.clip(np.rint((g - bias) / scale), 0, 15), 0)
            out[name] = (scale.astype(np.float64) * code + bias.astype(np.float64)).reshape(x.shape)
        return out
    p, d, h = case["page"], case["dim"], case["hkv"]
    group = case["hq"] // h
    half, pairs = p * d // 2, p * d // 64 * 4
    out = torch.zeros((s["tokens"], case["hq"], d), dtype=torch.float64, device="cuda")
    starts, lens = s["starts"].tolist(), s["seq_len"].tolist()
    shift = torch.tensor([0, 4], device="cuda", dtype=torch.uint8)
    for i in range(case["requests"]):
        n, total = starts[i + 1] - starts[i], lens[i]
        first = max(0, total - n + 1 - case["window"]) if case["window"] else 0
        pos = torch.arange(first, total, device="cuda")
        page = s["table"][i, pos // p].long()
        at = pos % p
        for j in range(h):
            rec = s["pool"][page, j]

            def values(k):
                c = rec.gather(1, k * half + at[:, None] * (d // 2) + torch.arange(d // 2, device="cuda"))
                c = ((c[:, :, None] >> shift) & 15).reshape(len(pos), d).double()
                e = rec.gather(1, 2 * half + k * pairs + at[:, None] * (d // 16) + torch.arange(d // 16, device="cuda"))
                e = e.contiguous().view(torch.half).double().reshape(len(pos), d // 64, 2).repeat_interleave(64, 1)
                return e[..., 0] * c + e[..., 1]

            k, v = values(0), values(1)
            for a in range(0, n, 512):
                m = min(512, n - a)
                q = s["q"][starts[i] + a:starts[i] + a + m, j * group:(j + 1) * group].double()
                score = torch.einsum("mgd,ld->gml", q, k) * s["scale"]
                last = total - n + a + torch.arange(m, device="cuda")[:, None]
                hide = pos > last
                if case["window"]:
                    hide |= pos <= last - case["window"]
                score = torch.softmax(score.masked_fill(hide, -math.inf), -1)
                out[starts[i] + a:starts[i] + a + m, j * group:(j + 1) * group] = torch.einsum("gml,ld->mgd", score, v)
    return out
