"""Measured cases of the operators of a full-attention layer that is served beside
Gated DeltaNet layers.

Three operators, each in its plain form (torch operations in 32 bits) and as the
package's call:

  append  gated_deltanet_layer_gb300.kv_append: the step's queries and keys
          normalised and rotated to their positions, keys and values into the
          slots of a paged cache
  attend  PagedAttention.attend: the step's queries over their requests' pages,
          causal; one new token each, a few (verify steps), or chunks of prompts
  w4      linear_w4: act(x W^T + bias) + residual for few rows, W in 4 bits with
          group scales

Heads are those of attention layers that fit the package's layer shapes: the tiny
layer (1024 wide, heads of 64), the full layer (8192 wide, heads of 128), one of its
tensor-parallel ranks ("shard"), and the dense layer (5120 wide), with heads of 128
or of 256 with norms, a part of each rotated, and an output gate.
"""
import numpy as np
import torch

own = False

LAYERS = {
    "tiny": dict(Hq=8, Hkv=2, d=64, rotary=64, norms=False, gate=False),
    "shard": dict(Hq=8, Hkv=1, d=128, rotary=128, norms=False, gate=False),
    "full": dict(Hq=64, Hkv=8, d=128, rotary=128, norms=False, gate=False),
    "dense": dict(Hq=40, Hkv=8, d=128, rotary=128, norms=True, gate=False),
    "dense256": dict(Hq=24, Hkv=4, d=256, rotary=64, norms=True, gate=True),
}
EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a small server: the call's latency
        dict(name="append single tokens", op="append", layer="shard", requests=8, tokens=8, context=4096, block=64,
             pairs="halves", seed=1),
        # pieces of prompts far into long contexts, norms and a part of each head rotated
        dict(name="append far", op="append", layer="dense256", requests=5, tokens=1777, context=500000, block=32,
             pairs="halves", seed=2),
        # a full prefill step of the unsharded layer, pages of 16 tokens
        dict(name="append prompts", op="append", layer="full", requests=9, tokens=16384, context=0, block=16,
             pairs="neighbours", seed=3),
        # one short request on the tiny layer: latency
        dict(name="attend one", op="attend", layer="tiny", requests=1, tokens=1, context=130, block=16, seed=4),
        # a decode step of a busy server: ragged contexts, one new token each
        dict(name="attend single tokens", op="attend", layer="full", requests=64, tokens=64, context=8192, block=64,
             seed=5),
        # a decode step over two long documents
        dict(name="attend long", op="attend", layer="dense256", requests=2, tokens=2, context=131072, block=256,
             seed=6),
        # a verify step: four tokens a request
        dict(name="attend verify", op="attend", layer="dense", requests=24, tokens=96, context=6000, block=32,
             seed=7),
        # the next chunk of two long prompts
        dict(name="attend chunk", op="attend", layer="dense256", requests=2, tokens=2048, context=30000, block=64,
             seed=8),
        # a full prefill step of fresh prompts
        dict(name="attend prompts", op="attend", layer="full", requests=5, tokens=8192, context=0, block=16, seed=9),
        # one row through the shard's in_proj_qkvz
        dict(name="w4 one row", op="w4", rows=1, cols=2560, inner=8192, format="mxfp4", group=32, zeros=False,
             bias=False, act="none", residual=False, seed=10),
        # odd sizes with everything in the epilogue
        dict(name="w4 odd", op="w4", rows=33, cols=1037, inner=1056, format="int4", group=32, zeros=True, bias=True,
             act="gelu", residual=True, seed=11),
        # a decode step's rows through the full layer's in_proj_qkvz
        dict(name="w4 rows", op="w4", rows=8, cols=20480, inner=8192, format="int4", group=128, zeros=True,
             bias=False, act="none", residual=False, seed=12),
    ]


def spread(rng, low, high):
    """A whole number between low and high, its logarithm evenly spread."""
    v = int(round(low * (high / low) ** rng.random()))
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "w4"])
    seed = rng.randrange(1 << 20)
    if op == "append":
        requests = spread(rng, 1, 64)
        return dict(op=op, layer=rng.choice(sorted(LAYERS)), requests=requests,
                    tokens=requests if rng.random() < 0.3 else spread(rng, requests, 16384),
                    context=rng.choice([0, spread(rng, 1, 500000)]), block=rng.choice([1, 16, 24, 32, 64, 256]),
                    pairs=rng.choice(["halves", "neighbours"]), seed=seed)
    if op == "w4":
        format = rng.choice(["mxfp4", "int4"])
        group = 32 if format == "mxfp4" else rng.choice([32, 64, 128])
        return dict(op=op, rows=spread(rng, 1, 64), cols=spread(rng, 16, 20480), inner=group * spread(rng, 2, 8192 // group),
                    format=format, group=group, zeros=format == "int4" and rng.random() < 0.5, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "silu", "gelu"]), residual=rng.random() < 0.5, seed=seed)
    kind = rng.choice(["single", "verify", "chunk"])
    works = [work(c) for c in listed() if c["op"] == "attend"]
    most = {key: max(w[key] for w in works) for key in ("bytes", "flops")}
    while True:
        requests = spread(rng, 1, 96 if kind != "chunk" else 8)
        tokens = requests * {"single": 1, "verify": rng.randint(2, 8)}.get(kind, 1)
        if kind == "chunk":
            tokens = spread(rng, 16 * requests, 8192)
        context = spread(rng, 1, 131072)
        if kind == "chunk" and rng.random() < 0.4:
            context = 0
        case = dict(op=op, layer=rng.choice(sorted(LAYERS)), requests=requests, tokens=tokens, context=context,
                    block=rng.choice([1, 16, 24, 32, 64, 256]), seed=seed)
        if all(work(case)[key] <= most[key] for key in most):
            return case


# ------------------------------------------------------------------- inputs

def lengths(case):
    """New tokens and context of each request: one token each, as many each, or
    ragged; contexts from an eighth of the longest up."""
    rng = np.random.default_rng(case["seed"])
    n, total = case["requests"], case["tokens"]
    if total % n == 0 and total // n <= 8:
        new = np.full(n, total // n, np.int64)
    else:
        w = rng.exponential(size=n) + 0.05
        new = np.floor(w / w.sum() * total).astype(np.int64)
        new[rng.integers(0, n)] += total - new.sum()
    ctx = np.floor(case["context"] * 8.0 ** (rng.random(n) - 1)).astype(np.int64)
    ctx[rng.integers(0, n)] = case["context"]
    return new, ctx


def ints(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


def normal(shape, std, gen, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def pool(slots, heads, d, gen):
    """A cache that is in use throughout."""
    t = torch.empty(slots, heads, d, dtype=torch.bfloat16, device="cuda")
    for i in range(0, slots, 1 << 17):
        t[i:i + (1 << 17)].normal_(generator=gen)
    return t


def starts(new):
    cu = np.zeros(len(new) + 1, np.int64)
    np.cumsum(new, out=cu[1:])
    return cu


def prepare_append(case, rng, gen):
    c, B, T = LAYERS[case["layer"]], case["block"], case["tokens"]
    new, ctx = lengths(case)
    owner = np.repeat(np.arange(len(new)), new)
    pos = ctx[owner] + np.arange(T) - starts(new)[owner]
    # the pages that the new tokens fall into, anywhere in a pool of them and some more
    page, where = np.unique(owner * (1 << 32) + pos // B, return_inverse=True)
    pages = len(page) + 3
    slots = rng.permutation(pages)[where.reshape(-1)] * B + pos % B
    state = dict(case=case, pos=ints(pos), slots=ints(slots, torch.int64))
    # the fused projection's rows: q | k | v
    state["qkv"] = normal((T, (c["Hq"] + 2 * c["Hkv"]) * c["d"]), 1.5, gen)
    r = c["rotary"]
    state["freq"] = (THETA ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()
    state["qw"] = normal((c["d"],), 0.1, gen) if c["norms"] else None
    state["kw"] = normal((c["d"],), 0.1, gen) if c["norms"] else None
    state["k"], state["v"] = (pool(pages * B, c["Hkv"], c["d"], gen) for _ in range(2))
    return state


def prepare_attend(case, rng, gen):
    c, B, T = LAYERS[case["layer"]], case["block"], case["tokens"]
    new, ctx = lengths(case)
    need = -(-(new + ctx) // B)
    pages = int(need.sum()) + 3
    table = np.full((len(new), int(need.max())), -1, np.int32)
    table[np.arange(table.shape[1])[None, :] < need[:, None]] = rng.permutation(pages)[:int(need.sum())]
    state = dict(case=case, table=ints(table), cu=ints(starts(new)), ctx=ints(ctx), longest=int(new.max()))
    # queries, and beside them the gate, as the projection leaves them
    rows = normal((T, (2 if c["gate"] else 1) * c["Hq"] * c["d"]), 2.0, gen)
    state["q"] = rows[:, :c["Hq"] * c["d"]]
    state["gate"] = rows[:, c["Hq"] * c["d"]:] if c["gate"] else None
    state["k"], state["v"] = (pool(pages * B, c["Hkv"], c["d"], gen) for _ in range(2))
    if own:
        from gated_deltanet_layer_gb300 import PagedAttention
        state["handle"] = PagedAttention(c["Hq"], c["Hkv"], c["d"], B, max_tokens=T, max_seqs=len(new))
    return state


def prepare_w4(case, rng, gen):
    M, N, K, G = case["rows"], case["cols"], case["inner"], case["group"]
    state = dict(case=case, x=normal((M, K), 1.0, gen))
    state["codes"] = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    if case["format"] == "mxfp4":
        state["scales"] = torch.randint(119, 124, (N, K // G), generator=gen, device="cuda", dtype=torch.uint8)
    else:
        state["scales"] = (0.001 + 0.004 * torch.rand((N, K // G), generator=gen, device="cuda")).to(torch.bfloat16)
    state["zeros"] = (torch.randint(0, 16, (N, K // G), generator=gen, device="cuda", dtype=torch.uint8)
                      if case["zeros"] else None)
    state["bias"] = normal((N,), 0.5, gen) if case["bias"] else None
    state["residual"] = normal((M, N), 1.0, gen) if case["residual"] else None
    return state


def prepare(case, seed):
    mix = (int(seed) * 1000003 + case["seed"]) % (1 << 31)
    rng = np.random.default_rng(mix)
    gen = torch.Generator(device="cuda").manual_seed(mix)
    return {"append": prepare_append, "attend": prepare_attend, "w4": prepare_w4}[case["op"]](case, rng, gen)


# ------------------------------------------------------------------- the plain forms

def plain_append(s):
    c = LAYERS[s["case"]["layer"]]
    d, r, T = c["d"], c["rotary"], s["pos"].shape[0]
    cut = [c["Hq"] * d, c["Hkv"] * d, c["Hkv"] * d]
    q, k, v = s["qkv"].split(cut, 1)
    angle = s["pos"].double()[:, None] * s["freq"].double()[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]

    def turned(x, w):
        x = x.float().view(T, -1, d)
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * (1 + w.float())
        if s["case"]["pairs"] == "halves":
            a, b = x[..., :r // 2], x[..., r // 2:r]
        else:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
        y, z = a * cos - b * sin, b * cos + a * sin
        head = torch.cat([y, z], -1) if s["case"]["pairs"] == "halves" else torch.stack([y, z], -1).flatten(-2)
        return torch.cat([head, x[..., r:]], -1).to(torch.bfloat16)

    s["k"][s["slots"]] = turned(k, s["kw"])
    s["v"][s["slots"]] = v.reshape(T, -1, d)
    return turned(q, s["qw"]).view(T, -1), s["k"], s["v"]


def plain_attend(s):
    case = s["case"]
    c, B = LAYERS[case["layer"]], case["block"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    new, ctx = lengths(case)
    cu = starts(new)
    out = torch.zeros(case["tokens"], Hq * d, device="cuda")
    for r in range(len(new)):
        n, L = int(new[r]), int(new[r] + ctx[r])
        if n == 0:
            continue
        at = torch.arange(L, device="cuda")
        slots = s["table"][r][at // B].long() * B + at % B
        k = s["k"][slots].float().permute(1, 2, 0)  # [Hkv, d, L]
        v = s["v"][slots].float().permute(1, 0, 2)  # [Hkv, L, d]
        q = s["q"][cu[r]:cu[r + 1]].float().view(n, Hkv, G, d).permute(1, 0, 2, 3)
        step = max(1, (1 << 28) // (Hq * L))
        for i in range(0, n, step):
            j = min(n, i + step)
            p = q[:, i:j].reshape(Hkv, -1, d) @ k * d ** -0.5  # [Hkv, rows, L]
            last = int(ctx[r]) + torch.arange(i, j, device="cuda").repeat_interleave(G)
            p = torch.where(at[None, :] <= last[:, None], p, float("-inf"))
            p = torch.exp(p - p.amax(-1, keepdim=True))
            o = (p @ v) / p.sum(-1, keepdim=True)
            out[cu[r] + i:cu[r] + j] = o.view(Hkv, j - i, G, d).permute(1, 0, 2, 3).reshape(j - i, -1)
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].float()))
    return out.to(torch.bfloat16)


def plain_w4(s):
    case, codes = s["case"], s["codes"]
    N, G = case["cols"], case["group"]
    code = torch.stack([codes & 15, codes >> 4], -1).view(N, -1, G)
    if case["format"] == "mxfp4":
        values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
        w = torch.cat([values, -values])[code.int()] * torch.exp2(s["scales"].float() - 127)[..., None]
    else:
        zero = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
        w = (code.float() - zero) * s["scales"].float()[..., None]
    y = s["x"].float() @ w.view(N, -1).T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = 0.5 * y * (1 + torch.tanh(0.7978845608028654 * (y + 0.044715 * y * y * y)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


PLAIN = {"append": plain_append, "attend": plain_attend, "w4": plain_w4}


# ------------------------------------------------------------------- the package's calls

def run(state):
    op, case = state["case"]["op"], state["case"]
    if not own:
        return PLAIN[op](state)
    if op == "append":
        from gated_deltanet_layer_gb300 import kv_append
        c = LAYERS[case["layer"]]
        a, b = c["Hq"] * c["d"], c["Hkv"] * c["d"]
        rows = state["qkv"]
        q = kv_append(rows[:, :a], rows[:, a:a + b], rows[:, a + b:], state["pos"], state["slots"], state["freq"],
                      state["k"], state["v"], q_norm_w=state["qw"], k_norm_w=state["kw"], norm_eps=EPS,
                      interleaved=case["pairs"] == "neighbours")
        return q, state["k"], state["v"]
    if op == "w4":
        from gated_deltanet_layer_gb300 import linear_w4
        return linear_w4(state["x"], state["codes"], state["scales"], zeros=state["zeros"], bias=state["bias"],
                         activation=case["act"], residual=state["residual"])
    return state["handle"].attend(state["q"], state["k"], state["v"], state["table"], state["cu"], state["ctx"],
                                  gate=state["gate"], max_len=state["longest"])


# ------------------------------------------------------------------- the least work

def work(case):
    if case["op"] == "w4":
        M, N, K = case["rows"], case["cols"], case["inner"]
        groups = N * K // case["group"]
        weights = N * K // 2 + groups * (1 if case["format"] == "mxfp4" else 2) + (groups if case["zeros"] else 0)
        return {"bytes": weights + 2 * (M * K + M * N * (2 if case["residual"] else 1) + (N if case["bias"] else 0)),
                "flops": 2 * M * N * K}
    c, T = LAYERS[case["layer"]], case["tokens"]
    if case["op"] == "append":
        row = (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        return {"bytes": T * (4 * row + 12), "flops": T * (c["Hq"] + c["Hkv"]) * (3 * c["rotary"] + 4 * c["d"] * c["norms"])}
    new, ctx = lengths(case)
    scores = int((new * ctx + new * (new + 1) // 2).sum())
    keys = int((new + ctx)[new > 0].sum())
    return {"bytes": 4 * keys * c["Hkv"] * c["d"] + 2 * T * c["Hq"] * c["d"] * (3 if c["gate"] else 2) + 4 * keys // case["block"],
            "flops": 4 * scores * c["Hq"] * c["d"]}


# ------------------------------------------------------------------- the definitions, in 64 bits

def exact_append(s):
    c, f = LAYERS[s["case"]["layer"]], torch.float64
    d, h, T = c["d"], c["rotary"] // 2, s["pos"].shape[0]
    x = s["qkv"].to(f).view(T, -1, d)
    n = c["Hq"] + c["Hkv"]
    y = x[:, :n].clone()
    if c["norms"]:
        w = torch.cat([s["qw"].to(f).expand(c["Hq"], d), s["kw"].to(f).expand(c["Hkv"], d)])
        y *= (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * (1 + w)
    turn = torch.polar(torch.ones(T, h, dtype=f, device="cuda"), s["pos"].to(f)[:, None] * s["freq"].to(f))
    first, second = ((slice(0, h), slice(h, 2 * h)) if s["case"]["pairs"] == "halves"
                     else (slice(0, 2 * h, 2), slice(1, 2 * h, 2)))
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    k, v = s["k"].to(f), s["v"].to(f)
    k[s["slots"]], v[s["slots"]] = y[:, c["Hq"]:], x[:, n:]
    return y[:, :c["Hq"]].reshape(T, -1), k, v


def exact_attend(s):
    case, f = s["case"], torch.float64
    c = LAYERS[case["layer"]]
    d, G = c["d"], c["Hq"] // c["Hkv"]
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    out = torch.zeros(case["tokens"], c["Hq"], d, dtype=f, device="cuda")
    for r in range(case["requests"]):
        n = cu[r + 1] - cu[r]
        if n == 0:
            continue
        L = ctx[r] + n
        pages = s["table"][r, :-(-L // case["block"])].long()
        rows = (pages[:, None] * case["block"] + torch.arange(case["block"], device="cuda")).flatten()[:L]
        q = s["q"][cu[r]:cu[r + 1]].to(f).view(n, c["Hq"], d) / d ** 0.5
        for h in range(c["Hkv"]):
            k, v = s["k"][rows, h].to(f), s["v"][rows, h].to(f)
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                a = torch.einsum("thd,ld->htl", q[i:i + m, h * G:(h + 1) * G], k)
                hidden = torch.ones(m, L, dtype=torch.bool, device="cuda").triu(ctx[r] + i + 1)
                a = torch.softmax(a.masked_fill_(hidden, float("-inf")), -1)
                out[cu[r] + i:cu[r] + i + m, h * G:(h + 1) * G] = torch.einsum("htl,ld->thd", a, v)
    out = out.view(case["tokens"], -1)
    return out * torch.sigmoid(s["gate"].to(f)) if s["gate"] is not None else out


def exact_w4(s):
    case, f = s["case"], torch.float64
    N, K, G = case["cols"], case["inner"], case["group"]
    w = torch.empty(N, K, dtype=f, device="cuda")
    for at, code in ((0, s["codes"] % 16), (1, s["codes"] // 16)):
        code = code.to(f)
        if case["format"] == "mxfp4":
            size = code % 8
            # 0, 1/2, 1, 3/2, 2, 3, 4, 6
            value = torch.where(size < 4, size / 2, torch.where(size < 6, size - 2, 2 * size - 8))
            w[:, at::2] = torch.where(code >= 8, -value, value)
        else:
            w[:, at::2] = code
    grouped = w.view(N, K // G, G)
    if case["format"] == "mxfp4":
        grouped *= torch.pow(2.0, s["scales"].to(f) - 127)[:, :, None]
    else:
        grouped -= 8 if s["zeros"] is None else s["zeros"].to(f)[:, :, None]
        grouped *= s["scales"].to(f)[:, :, None]
    y = torch.mm(s["x"].to(f), w.t())
    if s["bias"] is not None:
        y += s["bias"].to(f)
    if case["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif case["act"] == "gelu":
        y = torch.nn.functional.gelu(y, approximate="tanh")
    return y + s["residual"].to(f) if s["residual"] is not None else y


def exact(case, seed):
    state = prepare(case, seed)
    return {"append": exact_append, "attend": exact_attend, "w4": exact_w4}[case["op"]](state)
