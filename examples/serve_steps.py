"""A small server loop on the library's entry points: attention layers over the
4-bit or the 8-bit key/value cache between activation-sparse MoE layers.

Requests come with prompts of unequal lengths, decode token by token and end; a
step is one call of hs_kv4_plan (which gives pages, slots and row starts on the
device, from the lengths alone) and, for every layer, hs_kv4_append,
hs_kv4_attention (or those of the 8-bit cache), hs_router_logits and
hs_moe_layer_decode.  Between steps a request is forked into several samples, which
share its pages (hs_kv_fork, hs_kv_copy_pages), requests end or are cut back
(hs_kv_release), and the pages in use are moved to the pool's front
(hs_kv_compact).  The weights are synthetic; the projections around the attention
are plain matrix products.

    python examples/serve_steps.py [8]
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import synth
from activation_sparse_moe_gb300 import hs
from activation_sparse_moe_gb300.layer import DeviceLayer, from_synth_expert, from_synth_stack

HIDDEN, HEADS, KV_HEADS, DIM = 512, 8, 2, 64
EXPERTS, TOP_K, ROUTED, SHARED = 8, 3, 128, 256


class Layer:
    """One attention layer with its cache, and the MoE layer behind it."""

    def __init__(self, index: int, n_pages: int, page: int, bits: int):
        g = torch.Generator(device="cuda")
        g.manual_seed(100 + index)
        w = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[0] ** -0.5).bfloat16()  # noqa: E731
        self.qkv, self.out, self.router = w(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM), w(HEADS * DIM, HIDDEN), w(HIDDEN, EXPERTS).T.contiguous()
        up, down = synth.gen_routed_stack((0, f"serve{index}", "routed"), EXPERTS, ROUTED, hidden=HIDDEN)
        shared = synth.gen_expert((0, f"serve{index}", "shared"), SHARED, hidden=HIDDEN, p=0.2)
        self.moe = DeviceLayer(from_synth_stack(up, down, synth.stack_offsets(up, 0.2)), from_synth_expert(shared), top_k=TOP_K)
        make, size = (hs.make_kv4_cache, hs.hs_kv4_pool_bytes) if bits == 4 else (hs.make_kv8_cache, hs.hs_kv8_pool_bytes)
        self.pool = torch.zeros(size(make(None, n_pages, page, KV_HEADS, DIM)), dtype=torch.uint8, device="cuda")
        self.cache = make(self.pool, n_pages, page, KV_HEADS, DIM)


class Server:
    def __init__(self, rows: int = 4, layers: int = 2, n_pages: int = 64, page: int = 16, width: int = 32, max_tokens: int = 256,
                 bits: int = 4):
        self.rows, self.page, self.n_pages, self.width, self.max_tokens = rows, page, n_pages, width, max_tokens
        self.layers = [Layer(i, n_pages, page, bits) for i in range(layers)]
        self.append, self.attention = (hs.hs_kv4_append, hs.hs_kv4_attention) if bits == 4 else (hs.hs_kv8_append, hs.hs_kv8_attention)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        i64 = lambda *s: torch.zeros(s, dtype=torch.int64, device="cuda")  # noqa: E731
        self.length, self.table = i32(rows), torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.ring, self.counters = torch.arange(n_pages, dtype=torch.int32, device="cuda"), i64(2)
        self.counters[1] = n_pages                       # every page is free
        self.counters_out, self.short = i64(2), i32(1)
        self.seq_len, self.q_start, self.slot, self.position = i32(rows), i32(rows + 1), i64(max_tokens), i32(max_tokens)
        # for pages that several rows hold, that are given back, and that move
        self.shared, self.length_out = i32(n_pages), i32(rows)
        self.copy_src, self.copy_dst = i32(n_pages), i32(n_pages)
        self.pools = hs.make_kv_pools([layer.pool for layer in self.layers])
        self.page_bytes = self.pools.nbytes // n_pages
        self.pages_ws = torch.zeros(hs.hs_kv_pages_workspace_size(n_pages), dtype=torch.uint8, device="cuda")
        size = hs.hs_kv4_attention_workspace_size if bits == 4 else hs.hs_kv8_attention_workspace_size
        self.ws = torch.zeros(size(self.layers[0].cache, rows, HEADS), dtype=torch.uint8, device="cuda")
        moe = max(layer.moe.workspace_size(t) for layer in self.layers for t in (1, 2, 8, 50, max_tokens))
        self.moe_ws = torch.zeros(moe, dtype=torch.uint8, device="cuda")

    def step(self, new: list, x: torch.Tensor) -> torch.Tensor:
        """new: each row's new tokens (-1: its request has ended); x: their hidden
        states [sum of new][HIDDEN] bf16.  Returns the hidden states behind the
        last layer.  The host knows the tokens' number, not where they are cached."""
        t, most = x.shape[0], max(new + [1])
        fresh = torch.tensor(new, dtype=torch.int32, device="cuda")
        hs.hs_kv4_plan(self.length, fresh, self.rows, self.page, self.n_pages, self.table, self.width, self.ring, self.counters,
                       self.max_tokens, self.table, self.seq_len, self.q_start, self.slot, self.position, self.counters_out, self.short)
        for layer in self.layers:
            qkv = (norm(x) @ layer.qkv).view(t, HEADS + 2 * KV_HEADS, DIM)
            q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
            self.append(layer.cache, k, v, self.slot, t)
            o = torch.empty((t, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
            self.attention(layer.cache, q, self.q_start, self.seq_len, self.table, self.rows, most, DIM ** -0.5, 0, o, self.ws)
            x = x + o.view(t, HEADS * DIM) @ layer.out
            h = norm(x)
            logits, y = torch.empty((t, EXPERTS), device="cuda"), torch.empty_like(h)
            hs.hs_router_logits(h, layer.router, t, HIDDEN, EXPERTS, logits)
            self.moe_ws.zero_()
            hs.hs_moe_layer_decode(layer.moe.c, h, logits, t, y, workspace=self.moe_ws)
            x = x + norm(y)
        self.length.copy_(self.seq_len)
        self.counters.copy_(self.counters_out)
        return x

    def fork(self, parents: list, children: list, lengths: list):
        """Rows `children` (empty ones) begin with the first `lengths` tokens of rows `parents`."""
        p, c, m = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (parents, children, lengths))
        hs.hs_kv_fork(p, c, m, len(parents), self.length, self.rows, self.page, self.n_pages, self.table, self.width, self.shared,
                      self.ring, self.counters, self.table, self.length_out, self.copy_src, self.copy_dst, self.counters_out, self.short)
        hs.hs_kv_copy_pages(self.pools, self.page_bytes, self.n_pages, self.copy_src, self.copy_dst, len(parents))
        self.length.copy_(self.length_out)
        self.counters.copy_(self.counters_out)

    def keep(self, lengths: list):
        """Every row's first tokens that it keeps (0: its request has ended).  Where rows
        share pages requests end here, not with a step's -1."""
        m = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        hs.hs_kv_release(self.length, m, self.rows, self.page, self.n_pages, self.table, self.width, self.shared, self.ring,
                         self.counters, self.table, self.length_out, self.counters_out, self.pages_ws)
        self.length.copy_(self.length_out)
        self.counters.copy_(self.counters_out)

    def compact(self):
        hs.hs_kv_compact(self.length, self.rows, self.page, self.n_pages, self.table, self.width, self.shared, self.ring, self.counters,
                         self.n_pages, self.table, self.shared, self.copy_src, self.copy_dst, self.counters_out, self.short, self.pages_ws)
        hs.hs_kv_copy_pages(self.pools, self.page_bytes, self.n_pages, self.copy_src, self.copy_dst, self.n_pages)
        self.counters.copy_(self.counters_out)

    def free_pages(self) -> int:
        return int(self.counters[1] - self.counters[0])


def norm(x: torch.Tensor) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


def hidden(tokens: int, seed: int) -> torch.Tensor:
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((tokens, HIDDEN), generator=g, device="cuda").bfloat16()


def main(bits: int = 4):
    s = Server(bits=bits)
    print("free pages", s.free_pages())
    s.step([37, 5, 130, 0], hidden(172, 0))
    print("three prompts in:", s.length.tolist(), "free", s.free_pages())
    for i in range(4):
        y = s.step([1, 1, 1, 0], hidden(3, 1 + i))
    print("four tokens each:", s.length.tolist(), "free", s.free_pages())
    y = s.step([1, -1, 1, 60], hidden(62, 9))
    print("one ended, one came:", s.length.tolist(), "free", s.free_pages(), "|y|", float(y.float().norm()))
    s.keep([1 << 30, 0, 0, 1 << 30])
    s.fork([0, 0], [1, 2], [int(s.length[0]), 32])
    for i in range(3):
        s.step([1, 1, 1, 1], hidden(4, 20 + i))
    print("two samples of the first:", s.length.tolist(), "free", s.free_pages())
    s.keep([0, 1 << 30, 0, 50])
    s.compact()
    s.step([0, 1, 20, 1], hidden(22, 30))
    print("ended, cut back, compacted:", s.length.tolist(), "free", s.free_pages(), "last page", int(s.table.max()))
    assert hs.hs_device_status() == hs.HS_OK and int(s.short) == 0


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 4)
