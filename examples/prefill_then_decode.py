"""Prompts through one Gated DeltaNet layer, then decode steps on the same states.

A ragged batch of prompts goes through the prompt-side operators:
  slot_map            each request's state slot and the rows' offsets
  linear              in_proj_qkvz and in_proj_ba over all rows
  GdnPrefill.conv     causal conv1d + SiLU, leaving each request's conv state
  GdnPrefill.delta    the gated delta rule and the gated norm, leaving its SSM state
  linear              out_proj, added to the residual stream
and GdnDecode.step continues from the slots they wrote. The input RMSNorm of the
prompt side is plain torch.

    python examples/prefill_then_decode.py [layer: tiny or shard] [decode steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_deltanet_layer_gb300 import GdnDecode, GdnPrefill, linear, linear_check, slot_map, workloads as WL  # noqa: E402


def prefill_layer(shape, prefill, x, residual, weights, out_proj, cu_seqlens, state_in, state_out, conv_state, ssm_state,
                  max_len=None):
    """One layer over the rows x [tokens, H] of a ragged batch. Returns (x', residual')
    as the decode step's caller has them: the layer's output added to the residual."""
    r = x if residual is None else x + residual
    f = r.float()
    normed = (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + shape.norm_eps)
              * (1 + weights["input_norm_w"].float())).to(torch.bfloat16)
    qkvz, ba = linear(normed, weights["qkvz"]), linear(normed, weights["ba"])
    C = shape.conv_channels
    y = prefill.conv(qkvz[:, :C], weights["conv_w"], cu_seqlens, state_in, state_out, conv_state)
    core = prefill.delta(y, ba, weights, cu_seqlens, state_in, state_out, ssm_state, z=qkvz[:, C:], max_len=max_len)
    return linear(core, out_proj, residual=r), r


def main(layer="tiny", steps=4, lens=(37, 1, 130, 64), seed=0):
    shape = WL.SHAPES[layer]
    w = {k: (v.cuda() if v is not None else None) for k, v in WL.make_weights(shape, seed, conv_std=0.4).items()}
    out_proj = WL.make_out_proj(shape, seed + 1).cuda()
    conv = torch.zeros(shape.num_slots, shape.conv_channels, 3, dtype=torch.bfloat16, device="cuda")
    ssm = torch.zeros(shape.num_slots, shape.num_v_heads, shape.head_v_dim, shape.head_k_dim, device="cuda",
                      dtype=torch.bfloat16 if shape.ssm_dtype == "bf16" else torch.float32)
    R, T = len(lens), sum(lens)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    # one state slot a request: blocks longer than any request, taken off a free list
    # that leaves out slot 0, the pad slot
    table, free = torch.zeros(R, 1, dtype=torch.int32, device="cuda"), ints(list(range(shape.num_slots - 1, 0, -1)))
    m = slot_map(ints(lens), ints([0] * R), 1 << 20, table, free, ints([free.numel()]), T)
    slots, fresh = table[:, 0].contiguous(), torch.zeros(R, dtype=torch.int32, device="cuda")

    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, shape.hidden, generator=g, device="cuda").to(torch.bfloat16)
    prefill = GdnPrefill(shape, max_tokens=T, max_seqs=R)
    y, _ = prefill_layer(shape, prefill, x, None, w, out_proj, m.cu_seqlens, fresh, slots, conv, ssm, max_len=max(lens))
    status, detail = prefill.check()
    assert status == 0 and linear_check()[0] == 0, f"device error word 0x{detail:08x}"

    decode = GdnDecode(shape)
    cores = []
    for _ in range(steps):
        x = torch.randn(R, shape.hidden, generator=g, device="cuda").to(torch.bfloat16)
        core, _ = decode.step(x, None, w, slots, conv, ssm)
        cores.append(core)
    status, detail = decode.check()
    assert status == 0, f"device error word 0x{detail:08x}"
    return y, cores, conv, ssm, slots, m


if __name__ == "__main__":
    layer = sys.argv[1] if len(sys.argv) > 1 else "tiny"
    y, cores, _, ssm, slots, m = main(layer, int(sys.argv[2]) if len(sys.argv) > 2 else 4)
    print(f"{layer}: {y.shape[0]} prompt rows of {slots.numel()} requests, slots {slots.tolist()}, "
          f"{m.free_count.item()} slots left, {len(cores)} decode steps")
