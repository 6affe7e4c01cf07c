"""Prompts through one full-attention layer, then decode steps on the same paged cache,
with 4-bit projections throughout.

A step, whether it brings prompts or one token a request:
  slot_map                 offsets, positions and slots of the step's tokens, new blocks
                           off the free list
  linear_w4                the fused projection q | k | v | gate of every token
  kv_append                norms and rotation, keys and values into their slots
  PagedAttention.attend    the step's queries over their requests' pages, gated
  linear_w4                out projection, added to the residual stream

The prompts here are short. A server keeps bf16 weights beside the codes for long ones, whose
projections `linear` does in one pass, where linear_w4 reads the weights again for each 32 rows
at most.

    python examples/serve_attention_layer.py [decode steps]
"""
from __future__ import annotations

import os
import sys
from collections import namedtuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_deltanet_layer_gb300 import PagedAttention, kv_append, linear_w4, slot_map  # noqa: E402

Layer = namedtuple("Layer", "hidden q_heads kv_heads head_dim rotary block")
TINY = Layer(hidden=512, q_heads=8, kv_heads=2, head_dim=64, rotary=32, block=16)


def make_weights(layer, seed, group=64):
    """Codes, scales and zeros of both projections, norm weights and frequencies."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cols = (2 * layer.q_heads + 2 * layer.kv_heads) * layer.head_dim

    def packed(n, k):
        byte = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)
        scales = (0.5 + torch.rand(n, k // group, generator=g, device="cuda")) * 0.2 * k ** -0.5
        return byte(n, k // 2), scales.to(torch.bfloat16), byte(n, k // group) % 16

    norm = lambda: (torch.randn(layer.head_dim, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    r = layer.rotary
    freq = (1e4 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()
    return dict(proj=packed(cols, layer.hidden), out=packed(layer.hidden, layer.q_heads * layer.head_dim), q_norm=norm(),
                k_norm=norm(), freq=freq)


class Server:
    """The layer's cache, its free blocks, and what each request holds of them."""

    def __init__(self, layer, weights, *, blocks, max_blocks, requests, max_tokens):
        self.layer, self.w = layer, weights
        shape = (blocks * layer.block, layer.kv_heads, layer.head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table = torch.full((requests, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.free = torch.arange(blocks - 1, -1, -1, dtype=torch.int32, device="cuda")
        self.free_count = torch.tensor([blocks], dtype=torch.int32, device="cuda")
        self.context = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.attention = PagedAttention(layer.q_heads, layer.kv_heads, layer.head_dim, layer.block, max_tokens=max_tokens,
                                        max_seqs=requests)
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, x, new, max_len):
        """x [tokens, hidden], new int32 [requests] tokens of each; max_len: no request has more.
        Returns the layer's output and what it was made of."""
        L, w = self.layer, self.w
        m = slot_map(new, self.context, L.block, self.table, self.free, self.free_count, x.shape[0], error=self.error)
        rows = linear_w4(x, *w["proj"])
        q, kv = L.q_heads * L.head_dim, L.kv_heads * L.head_dim
        turned = kv_append(rows[:, :q], rows[:, q:q + kv], rows[:, q + kv:q + 2 * kv], m.token_pos, m.slots, w["freq"], self.k,
                           self.v, q_norm_w=w["q_norm"], k_norm_w=w["k_norm"], error=self.error)
        core = self.attention.attend(turned, self.k, self.v, self.table, m.cu_seqlens, self.context,
                                     gate=rows[:, q + 2 * kv:], max_len=max_len)
        y = linear_w4(core, *w["out"], residual=x)
        self.context = self.context + new
        self.free_count = m.free_count
        return y, dict(map=m, rows=rows, turned=turned, core=core)

    def check(self):
        status, detail = self.attention.check()
        assert status == 0 and self.error.item() == 0, f"device error words 0x{detail:08x} 0x{self.error.item():08x}"


def main(steps=4, lens=(37, 1, 130, 64), seed=0, layer=TINY):
    R = len(lens)
    server = Server(layer, make_weights(layer, seed), blocks=64, max_blocks=16, requests=R, max_tokens=sum(lens))
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rows = lambda n: torch.randn(n, layer.hidden, generator=g, device="cuda").to(torch.bfloat16)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    outs = [server.step(rows(sum(lens)), ints(lens), max(lens))[0]]
    for _ in range(steps):
        outs.append(server.step(rows(R), ints([1] * R), 1)[0])
    server.check()
    return outs, server


if __name__ == "__main__":
    outs, server = main(int(sys.argv[1]) if len(sys.argv) > 1 else 4)
    print(f"{outs[0].shape[0]} prompt rows, {len(outs) - 1} decode steps, contexts {server.context.tolist()}, "
          f"{server.free_count.item()} blocks left")
