"""A small server loop on the library's entry points: attention layers over the
4-bit key/value cache between activation-sparse MoE layers.

Requests come with prompts of unequal lengths, decode token by token and end; a
step is one call of hs_kv4_plan (which gives pages, slots and row starts on the
device, from the lengths alone) and, for every layer, hs_kv4_append,
hs_kv4_attention, hs_router_logits and hs_moe_layer_decode.  The weights are
synthetic; the projections around the attention are plain matrix products.

    python examples/serve_steps.py
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

    def __init__(self, index: int, n_pages: int, page: int):
        g = torch.Generator(device="cuda")
        g.manual_seed(100 + index)
        w = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[0] ** -0.5).bfloat16()  # noqa: E731
        self.qkv, self.out, self.router = w(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM), w(HEADS * DIM, HIDDEN), w(HIDDEN, EXPERTS).T.contiguous()
        up, down = synth.gen_routed_stack((0, f"serve{index}", "routed"), EXPERTS, ROUTED, hidden=HIDDEN)
        shared = synth.gen_expert((0, f"serve{index}", "shared"), SHARED, hidden=HIDDEN, p=0.2)
        self.moe = DeviceLayer(from_synth_stack(up, down, synth.stack_offsets(up, 0.2)), from_synth_expert(shared), top_k=TOP_K)
        sizes = hs.make_kv4_cache(None, n_pages, page, KV_HEADS, DIM)
        self.pool = torch.zeros(hs.hs_kv4_pool_bytes(sizes), dtype=torch.uint8, device="cuda")
        self.cache = hs.make_kv4_cache(self.pool, n_pages, page, KV_HEADS, DIM)


class Server:
    def __init__(self, rows: int = 4, layers: int = 2, n_pages: int = 64, page: int = 16, width: int = 32, max_tokens: int = 256):
        self.rows, self.page, self.n_pages, self.width, self.max_tokens = rows, page, n_pages, width, max_tokens
        self.layers = [Layer(i, n_pages, page) for i in range(layers)]
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        i64 = lambda *s: torch.zeros(s, dtype=torch.int64, device="cuda")  # noqa: E731
        self.length, self.table = i32(rows), torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.ring, self.counters = torch.arange(n_pages, dtype=torch.int32, device="cuda"), i64(2)
        self.counters[1] = n_pages                       # every page is free
        self.counters_out, self.short = i64(2), i32(1)
        self.seq_len, self.q_start, self.slot, self.position = i32(rows), i32(rows + 1), i64(max_tokens), i32(max_tokens)
        c = self.layers[0].cache
        self.ws = torch.zeros(hs.hs_kv4_attention_workspace_size(c, rows, HEADS), dtype=torch.uint8, device="cuda")
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
            hs.hs_kv4_append(layer.cache, k, v, self.slot, t)
            o = torch.empty((t, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
            hs.hs_kv4_attention(layer.cache, q, self.q_start, self.seq_len, self.table, self.rows, most, DIM ** -0.5, 0, o, self.ws)
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

    def free_pages(self) -> int:
        return int(self.counters[1] - self.counters[0])


def norm(x: torch.Tensor) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


def hidden(tokens: int, seed: int) -> torch.Tensor:
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((tokens, HIDDEN), generator=g, device="cuda").bfloat16()


def main():
    s = Server()
    print("free pages", s.free_pages())
    s.step([37, 5, 130, 0], hidden(172, 0))
    print("three prompts in:", s.length.tolist(), "free", s.free_pages())
    for i in range(4):
        y = s.step([1, 1, 1, 0], hidden(3, 1 + i))
    print("four tokens each:", s.length.tolist(), "free", s.free_pages())
    y = s.step([1, -1, 1, 60], hidden(62, 9))
    print("one ended, one came:", s.length.tolist(), "free", s.free_pages(), "|y|", float(y.float().norm()))
    assert hs.hs_device_status() == hs.HS_OK and int(s.short) == 0


if __name__ == "__main__":
    main()
