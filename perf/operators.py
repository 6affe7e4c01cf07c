"""Measured cases of the prompt-side operators of a Gated DeltaNet layer.

Four operators, each in its plain form (torch operations in 32 bits) and as the
package's call:

  slots   gated_deltanet_layer_gb300.slot_map: offsets, block tables and slots of
          a ragged batch from its request lengths
  conv    GdnPrefill.conv: causal depthwise conv1d + SiLU over ragged prompts,
          with the conv state in and out
  delta   GdnPrefill.delta: the gated delta rule over ragged prompts (L2 norms,
          gates, recurrence, optional gated RMSNorm x SiLU(z)), with the SSM state
          in and out; requests of one token are its recurrent form
  linear  linear: act(x W^T + bias) + residual

Sizes are the package's layer shapes: the tiny layer (1024 wide, 4/8 heads of 64),
one tensor-parallel rank's shard (8192 wide, 2/8 heads of 128) and the full layer
(8192 wide, 16/64 heads of 128).
"""
import random

import numpy as np
import torch

own = False

LAYERS = {
    "tiny": dict(hidden=1024, Hk=4, Hv=8, d=64),
    "shard": dict(hidden=8192, Hk=2, Hv=8, d=128),
    "full": dict(hidden=8192, Hk=16, Hv=64, d=128),
}
EPS = 1e-6


def channels(layer):
    c = LAYERS[layer]
    return 2 * c["Hk"] * c["d"] + c["Hv"] * c["d"]


def columns(layer):
    c = LAYERS[layer]
    return channels(layer) + c["Hv"] * c["d"]


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a small server: the call's latency
        dict(name="slots decode", op="slots", requests=8, tokens=8, block=64, longest=4096, seed=1),
        # a wide prefill step over long contexts, pages of 16 tokens
        dict(name="slots long prompts", op="slots", requests=2048, tokens=524289, block=16, longest=65536, seed=2),
        # one short prompt on the tiny layer: latency
        dict(name="conv short", op="conv", layer="tiny", requests=1, tokens=5, longest=5, seed=3),
        # a full prefill step of the unsharded layer, read out of the fused projection's rows
        dict(name="conv full", op="conv", layer="full", requests=9, tokens=16384, longest=4096, seed=4),
        # ragged short prompts on the tiny layer, no gate: latency
        dict(name="delta short", op="delta", layer="tiny", requests=5, tokens=259, longest=130, state="f32",
             gated=False, seed=5),
        # decode-like: every request brings one token (the recurrent form), the full layer's f32 states
        dict(name="delta single tokens", op="delta", layer="full", requests=129, tokens=129, longest=1, state="f32",
             gated=True, seed=6),
        # one long prompt beside a few short ones on one rank's shard, bf16 states
        dict(name="delta shard bf16", op="delta", layer="shard", requests=4, tokens=5003, longest=4097,
             state="bf16", gated=True, seed=7),
        # a full prefill step of the unsharded layer
        dict(name="delta full", op="delta", layer="full", requests=13, tokens=16384, longest=2500, state="f32",
             gated=True, seed=8),
        # few rows: the shard's in_proj_qkvz for five rows, bound by its weights
        dict(name="linear few rows", op="linear", rows=5, cols=2560, inner=8192, bias=False, act="none",
             residual=False, seed=9),
        # odd sizes with everything in the epilogue
        dict(name="linear odd", op="linear", rows=777, cols=1037, inner=1000, bias=True, act="gelu", residual=True,
             seed=10),
        # the shard's out_proj over a prefill step, added to the residual stream
        dict(name="linear out_proj", op="linear", rows=4100, cols=8192, inner=1024, bias=False, act="none",
             residual=True, seed=11),
        # the full layer's in_proj_qkvz over a prefill step
        dict(name="linear in_proj", op="linear", rows=8192, cols=20480, inner=8192, bias=True, act="silu",
             residual=False, seed=12),
    ]


def spread(rng, low, high):
    """A whole number between low and high, its logarithm evenly spread."""
    v = int(round(low * (high / low) ** rng.random()))
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["slots", "conv", "delta", "delta", "linear", "linear"])
    seed = rng.randrange(1 << 20)
    if op == "slots":
        requests = spread(rng, 1, 2048)
        longest = spread(rng, 64, 65536)
        tokens = min(524289, spread(rng, requests, max(requests, min(requests * longest, 524289))))
        return dict(op=op, requests=requests, tokens=tokens, block=rng.choice([1, 16, 64, 256, 1 << 20])
                    if longest <= 1024 else rng.choice([16, 64, 256, 1 << 20]), longest=longest, seed=seed)
    if op == "conv":
        requests = spread(rng, 1, 128)
        longest = spread(rng, 1, 4096)
        tokens = min(16384, spread(rng, requests, requests * longest))
        return dict(op=op, layer=rng.choice(sorted(LAYERS)), requests=requests, tokens=tokens, longest=longest, seed=seed)
    if op == "delta":
        requests = spread(rng, 1, 128)
        longest = 1 if rng.random() < 0.25 else spread(rng, 2, 2500)
        tokens = min(16384, spread(rng, requests, requests * longest))
        return dict(op=op, layer=rng.choice(sorted(LAYERS)), requests=requests, tokens=tokens, longest=longest,
                    state=rng.choice(["f32", "bf16"]), gated=rng.random() < 0.7, seed=seed)
    return dict(op=op, rows=spread(rng, 1, 8192), cols=spread(rng, 16, 20480), inner=8 * spread(rng, 8, 1024),
                bias=rng.random() < 0.5, act=rng.choice(["none", "silu", "gelu"]), residual=rng.random() < 0.5, seed=seed)


# ------------------------------------------------------------------- inputs

def lengths(case, rng):
    """New tokens of each request: at most `longest`, together `tokens`; one each, or ragged with an empty one among them."""
    n, total, top = case["requests"], case["tokens"], case["longest"]
    if n == total:
        return np.ones(n, np.int64)
    w = rng.exponential(size=n) + 0.05
    if n > 3:
        w[rng.integers(0, n)] = 0.0
    if total > top:
        w[rng.integers(0, n)] = w.max() + 1.0
    got = np.minimum(np.floor(w / w.sum() * total).astype(np.int64), top)
    left = int(total - got.sum())
    order = np.argsort(-w, kind="stable")
    for r in order:
        add = min(left, int(top - got[r]))
        got[r] += add
        left -= add
        if not left:
            break
    return got


def ints(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


def prepare_slots(case, rng):
    R, B, top = case["requests"], case["block"], case["longest"]
    new = lengths(case, rng)
    ctx = np.where(rng.random(R) < 0.3, 0, rng.integers(0, np.maximum(1, top - new + 1)))
    have, want = -(-ctx // B), -(-(ctx + new) // B)
    wide = -(-top // B)
    pool = int(want.sum()) + 37
    order = rng.permutation(pool).astype(np.int64) + 1
    table = np.full((R, wide), -1, np.int32)
    inside = np.arange(wide)[None, :] < have[:, None]
    table[inside] = order[: int(have.sum())]
    free = order[int(have.sum()):]
    return dict(case=case, new=ints(new), ctx=ints(ctx), table=ints(table), free=ints(free),
                count=ints([len(free)]), tokens=case["tokens"])


def slots_of_states(rng, requests):
    """Each request's state slots: it starts from one of the first `requests`
    slots, or from zero, and ends in one of the next `requests`; one is padding."""
    first = rng.permutation(requests) + 1
    first[rng.random(requests) < 0.25] = 0
    last = rng.permutation(requests) + 1 + requests
    if requests > 2:
        last[rng.integers(0, requests)] = 0
    return first, last


def normal(shape, std, gen, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def ragged(case, rng, state):
    new = lengths(case, rng)
    first, last = slots_of_states(rng, case["requests"])
    cu = np.zeros(case["requests"] + 1, np.int64)
    np.cumsum(new, out=cu[1:])
    state.update(cu=ints(cu), first=ints(first), last=ints(last), longest=int(new.max()))


def handle(case):
    from gated_deltanet_layer_gb300 import GdnPrefill, workloads
    c = LAYERS[case["layer"]]
    shape = workloads.LayerShape(case["layer"], hidden=c["hidden"], num_k_heads=c["Hk"], num_v_heads=c["Hv"],
                                 head_k_dim=c["d"], head_v_dim=c["d"], num_slots=2 * case["requests"] + 1,
                                 ssm_dtype=case.get("state", "f32"))
    return GdnPrefill(shape, max_tokens=case["tokens"], max_seqs=case["requests"])


def prepare(case, seed):
    mix = (int(seed) * 1000003 + case["seed"]) % (1 << 31)
    rng = np.random.default_rng(mix)
    gen = torch.Generator(device="cuda").manual_seed(mix)
    if case["op"] == "slots":
        return prepare_slots(case, rng)
    if case["op"] == "linear":
        M, N, K = case["rows"], case["cols"], case["inner"]
        return dict(case=case, x=normal((M, K), 1.0, gen), w=normal((N, K), 0.02, gen),
                    bias=normal((N,), 0.5, gen) if case["bias"] else None,
                    residual=normal((M, N), 1.0, gen) if case["residual"] else None)
    c = LAYERS[case["layer"]]
    state = dict(case=case)
    ragged(case, rng, state)
    slots, T = 2 * case["requests"] + 1, case["tokens"]
    if own:
        state["handle"] = handle(case)
    # the fused projection's rows: q | k | v | z
    state["qkvz"] = normal((T, columns(case["layer"])), 1.8, gen)
    if case["op"] == "conv":
        state["w"] = normal((channels(case["layer"]), 4), 0.3, gen)
        state["pool"] = normal((slots, channels(case["layer"]), 3), 1.8, gen)
        return state
    state["qkv"] = torch.nn.functional.silu(normal((T, channels(case["layer"])), 1.0, gen))
    state["ba"] = normal((T, 2 * c["Hv"]), 1.8, gen)
    state["weights"] = dict(
        A_log=-2.0 * torch.rand((c["Hv"],), generator=gen, device="cuda"),
        dt_bias=normal((c["Hv"],), 0.5, gen),
        gated_norm_w=(1.0 + normal((c["d"],), 0.1, gen, torch.float32)).to(torch.bfloat16))
    state["pool"] = normal((slots, c["Hv"], c["d"], c["d"]), 0.1, gen,
                           torch.bfloat16 if case["state"] == "bf16" else torch.float32)
    return state


# ------------------------------------------------------------------- the plain forms

def plain_slots(s):
    B, N = s["case"]["block"], s["tokens"]
    new, ctx, table = s["new"].long(), s["ctx"].long(), s["table"]
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    have, want = (ctx + B - 1) // B, (ctx + new + B - 1) // B
    need = want - have
    before = torch.cumsum(need, 0) - need
    column = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (column >= have[:, None]) & (column < want[:, None])
    at = s["count"].long() - 1 - (before[:, None] + column - have[:, None])
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, max(0, s["free"].numel() - 1))], table))
    t = torch.arange(N, device="cuda")
    request = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = ctx[request] + t - cu[request]
    slots = table[request, pos // B].long() * B + pos % B
    return (cu.int(), request.int(), pos.int(), slots, s["count"] - need.sum().int(), table)


def starts(s, total):
    """Request and offset of every token."""
    t = torch.arange(total, device="cuda")
    request = torch.searchsorted(s["cu"][1:].long().contiguous(), t, right=True)
    return request, t - s["cu"].long()[request]


def plain_conv(s):
    C = channels(s["case"]["layer"])
    x, w, pool = s["qkvz"][:, :C].float(), s["w"].float(), s["pool"]
    T = x.shape[0]
    request, at = starts(s, T)
    first, last, cu = s["first"].long(), s["last"].long(), s["cu"].long()
    old = torch.where((first > 0)[:, None, None], pool[first].float(), 0.0)  # [requests, C, 3]
    y = x * w[:, 3]
    for j in range(3):
        back = 3 - j
        near = x[(torch.arange(T, device="cuda") - back).clamp(min=0)]
        far = old[request, :, (at + j).clamp(max=2)]
        y = y + torch.where((at >= back)[:, None], near, far) * w[:, j]
    y = y / (1 + torch.exp(-y))
    y = torch.where((last > 0)[request][:, None], y, 0.0).to(torch.bfloat16)
    n = cu[1:] - cu[:-1]
    p = n[:, None] - 3 + torch.arange(3, device="cuda")[None, :]  # offsets of the last three inputs
    inside = x[(cu[:-1, None] + p).clamp(0, T - 1)].transpose(1, 2)
    before = torch.gather(old, 2, (p + 3).clamp(0, 2)[:, None, :].expand_as(old))
    new = torch.where((p >= 0)[:, None, :], inside, before).to(pool.dtype)
    pool[last] = torch.where((last > 0)[:, None, None], new, pool[last])
    return y, pool[1 + s["case"]["requests"]:]


def plain_delta(s):
    case = s["case"]
    c = LAYERS[case["layer"]]
    Hk, Hv, d, G = c["Hk"], c["Hv"], c["d"], c["Hv"] // c["Hk"]
    qkv, ba, w, pool = s["qkv"].float(), s["ba"].float(), s["weights"], s["pool"]
    T = qkv.shape[0]
    q, k = qkv[:, :Hk * d].view(T, Hk, d), qkv[:, Hk * d:2 * Hk * d].view(T, Hk, d)
    v = qkv[:, 2 * Hk * d:].view(T, Hv, d)
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS) * d ** -0.5
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS)
    beta = 1 / (1 + torch.exp(-ba[:, :Hv]))
    a = ba[:, Hv:] + w["dt_bias"].float()
    decay = torch.exp(-torch.exp(w["A_log"]) * torch.where(a > 20, a, torch.log1p(torch.exp(a.clamp(max=20)))))
    first, last, cu = s["first"].long(), s["last"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    S = torch.where((first > 0)[:, None, None, None], pool[first].float(), 0.0)  # [requests, Hv, dv, dk]
    step = torch.arange(s["longest"], device="cuda")[:, None]
    on, at = (step < n)[:, :, None], (cu[:-1] + step).clamp(max=T - 1)  # [steps, requests]
    head = torch.arange(Hv, device="cuda") // G
    decay, beta = torch.where(on, decay[at], 1.0)[..., None, None], torch.where(on, beta[at], 0.0)[..., None]
    k, q, v = k[at], q[at], v[at]
    line = torch.zeros(s["longest"], *v.shape[1:3], d, device="cuda")
    for t in range(s["longest"]):
        kt = k[t][:, head]
        S *= decay[t]
        u = (v[t] - (S @ kt[..., None])[..., 0]) * beta[t]
        S += u[..., None] * kt[..., None, :]
        line[t] = (S @ q[t][:, head, :, None])[..., 0]
    o = torch.zeros(T, Hv, d, device="cuda")
    o[at[on[..., 0]]] = line[on[..., 0]]
    if case["gated"]:
        z = s["qkvz"][:, channels(case["layer"]):].float().view(T, Hv, d)
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * w["gated_norm_w"].float() * z / (1 + torch.exp(-z))
    request, _ = starts(s, T)
    o = torch.where((last > 0)[request][:, None, None], o, 0.0)
    pool[last] = torch.where((last > 0)[:, None, None, None], S.to(pool.dtype), pool[last])
    return o.reshape(T, Hv * d).to(torch.bfloat16), pool[1 + case["requests"]:]


def plain_linear(s):
    y = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["case"]["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif s["case"]["act"] == "gelu":
        y = 0.5 * y * (1 + torch.tanh(0.7978845608028654 * (y + 0.044715 * y * y * y)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


PLAIN = {"slots": plain_slots, "conv": plain_conv, "delta": plain_delta, "linear": plain_linear}


# ------------------------------------------------------------------- the package's calls

def run(state):
    op, case = state["case"]["op"], state["case"]
    if not own:
        return PLAIN[op](state)
    if op == "slots":
        from gated_deltanet_layer_gb300 import slot_map
        m = slot_map(state["new"], state["ctx"], case["block"], state["table"], state["free"], state["count"],
                     state["tokens"])
        return m.cu_seqlens, m.token_seq, m.token_pos, m.slots, m.free_count, state["table"]
    if op == "linear":
        from gated_deltanet_layer_gb300 import linear
        return linear(state["x"], state["w"], bias=state["bias"], activation=case["act"], residual=state["residual"])
    C, h, pool = channels(case["layer"]), state["handle"], state["pool"]
    if op == "conv":
        y = h.conv(state["qkvz"][:, :C], state["w"], state["cu"], state["first"], state["last"], pool)
    else:
        y = h.delta(state["qkv"], state["ba"], state["weights"], state["cu"], state["first"], state["last"], pool,
                    z=state["qkvz"][:, C:] if case["gated"] else None, max_len=state["longest"])
    return y, pool[1 + case["requests"]:]


# ------------------------------------------------------------------- the least work

def work(case):
    if case["op"] == "slots":
        R, N, B = case["requests"], case["tokens"], case["block"]
        return {"bytes": 8 * R + 4 * (R + 1) + 16 * N + 8 * (N / B + R), "flops": 0}
    if case["op"] == "linear":
        M, N, K = case["rows"], case["cols"], case["inner"]
        return {"bytes": 2 * (M * K + N * K + M * N * (2 if case["residual"] else 1) + (N if case["bias"] else 0)),
                "flops": 2 * M * N * K}
    c, T, R = LAYERS[case["layer"]], case["tokens"], case["requests"]
    C = channels(case["layer"])
    if case["op"] == "conv":
        return {"bytes": 4 * T * C + 12 * R * C + 8 * C, "flops": 12 * T * C}
    row = c["Hv"] * c["d"]
    state = row * c["d"] * (4 if case["state"] == "f32" else 2)
    return {"bytes": 2 * T * (C + 2 * c["Hv"] + row * (2 if case["gated"] else 1)) + 2 * R * state,
            "flops": T * row * c["d"] * 6}


# ------------------------------------------------------------------- the definitions, in 64 bits

def exact_conv(s):
    C = channels(s["case"]["layer"])
    x, w, pool = s["qkvz"][:, :C].double(), s["w"].double(), s["pool"].double()
    cu, first, last = s["cu"].tolist(), s["first"].tolist(), s["last"].tolist()
    y, new = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), pool.clone()
    for r, (i, j) in enumerate(zip(first, last)):
        if j <= 0:
            continue
        before = pool[i].T if i > 0 else torch.zeros(3, C, dtype=torch.float64, device="cuda")
        line = torch.cat([before, x[cu[r]:cu[r + 1]]])
        if cu[r + 1] > cu[r]:
            y[cu[r]:cu[r + 1]] = (line.unfold(0, 4, 1) * w).sum(-1)
        new[j] = line[-3:].T
    return y * torch.sigmoid(y), new[1 + s["case"]["requests"]:]


def exact_delta(s):
    case, f = s["case"], torch.float64
    c = LAYERS[case["layer"]]
    Hk, Hv, d = c["Hk"], c["Hv"], c["d"]
    cu, first, last = s["cu"].tolist(), s["first"].tolist(), s["last"].tolist()
    out, pool = torch.zeros(case["tokens"], Hv, d, dtype=f, device="cuda"), s["pool"].clone()
    new = pool[1 + case["requests"]:].to(f)
    rate, shift, scale = torch.exp(s["weights"]["A_log"].to(f)), s["weights"]["dt_bias"].to(f), s["weights"]["gated_norm_w"].to(f)
    for r, (i, j) in enumerate(zip(first, last)):
        if j <= 0:
            continue
        rows = slice(cu[r], cu[r + 1])
        n = cu[r + 1] - cu[r]
        x, ba = s["qkv"][rows].to(f), s["ba"][rows].to(f)
        S = pool[i].to(f) if i > 0 else torch.zeros(Hv, d, d, dtype=f, device="cuda")
        q, k, v = x[:, :Hk * d].reshape(n, Hk, d), x[:, Hk * d:2 * Hk * d].reshape(n, Hk, d), x[:, 2 * Hk * d:].reshape(n, Hv, d)
        q = (q * (q.square().sum(-1, keepdim=True) + EPS).rsqrt() / d ** 0.5).repeat_interleave(Hv // Hk, 1)
        k = (k * (k.square().sum(-1, keepdim=True) + EPS).rsqrt()).repeat_interleave(Hv // Hk, 1)
        b = torch.sigmoid(ba[:, :Hv])
        g = torch.exp(-rate * torch.nn.functional.softplus(ba[:, Hv:] + shift))
        for t in range(n):
            S = S * g[t, :, None, None]
            e = b[t, :, None] * (v[t] - torch.einsum("hvk,hk->hv", S, k[t]))
            S = torch.addcmul(S, e[:, :, None], k[t, :, None, :])
            out[cu[r] + t] = torch.einsum("hvk,hk->hv", S, q[t])
        if case["gated"]:
            z = s["qkvz"][rows, channels(case["layer"]):].to(f).reshape(n, Hv, d)
            o = out[rows]
            out[rows] = o * (o.square().mean(-1, keepdim=True) + EPS).rsqrt() * scale * z * torch.sigmoid(z)
        new[j - 1 - case["requests"]] = S
    return out.reshape(case["tokens"], Hv * d), new


def exact_linear(s):
    x, w = s["x"].double(), s["w"].double()
    y = torch.empty(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for i in range(0, x.shape[0], 2048):
        y[i:i + 2048] = torch.mm(x[i:i + 2048], w.t())
    if s["bias"] is not None:
        y += s["bias"].double()
    if s["case"]["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif s["case"]["act"] == "gelu":
        y = torch.nn.functional.gelu(y, approximate="tanh")
    return y + s["residual"].double() if s["residual"] is not None else y


def exact(case, seed):
    if case["op"] == "slots":
        return None
    state = prepare(case, seed)
    return {"conv": exact_conv, "delta": exact_delta, "linear": exact_linear}[case["op"]](state)
