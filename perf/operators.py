"""Operators around the rotated int8 layer, as cases that can be timed and compared.

Three operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and, where ``own`` is true, through the calls
of this package:

* block:   the step between two blocks of a transformer: norm of a block's
           output (or of the weighted sum of the rows its experts made), gate,
           residual scale and residual sum, then the next block's norm with
           its scale and shift -- as 16-bit values, or as the int8 codes the
           next layer's product reads;
* lora:    the int8 layer with the low-rank adapters of many requests beside
           it, each token with its own request's adapter;
* experts: the int8 layer grouped by expert, with as many rows for each
           expert as the router sent there.
"""
import math

import torch

own = False

_IO = {"bf16": torch.bfloat16, "fp16": torch.float16}
_EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a chat: the norms around one block, where latency counts
        _block("block_one_token", m=1, k=4096, io="bf16", post="rms", pre="rms", mods=0, routes=0, group=0, n=0),
        # an image model's step at 1024^2: four requests with their own modulation
        _block("block_image", m=4608, k=4096, io="bf16", post="none", pre="layer", mods=4, routes=0, group=0, n=0),
        # after the experts: eight rows summed per token, the norm coded as the next projection reads it
        _block("block_routes_coded", m=1000, k=2048, io="fp16", post="rms", pre="rms", mods=0, routes=8, group=128,
               n=1152),
        # an image model's step at 2048^2, norms on both sides of the block
        _block("block_large", m=16896, k=6144, io="bf16", post="rms", pre="rms", mods=2, routes=0, group=0, n=0),
        # sixteen chats in one decoding step, each with an adapter of its own
        _lora("lora_decode", m=16, k=4096, n=4096, io="bf16", adapters=16, rank=16, spread=False, rows=False, group=128),
        # a mixed batch of short prompts, ranks of all sizes, some tokens without an adapter
        _lora("lora_mixed", m=777, k=2048, n=6144, io="fp16", adapters=12, rank=64, spread=True, rows=True, group=256),
        # the up projection at 1024^2 for four requests with an adapter each
        _lora("lora_up", m=4608, k=4096, n=12288, io="bf16", adapters=4, rank=64, spread=False, rows=False, group=128),
        # the down projection of a batch with many adapters
        _lora("lora_down", m=2000, k=12288, n=4096, io="bf16", adapters=48, rank=32, spread=True, rows=False, group=128),
        # one token of a chat through its four experts
        _experts("experts_one_token", m=1, k=2048, n=1408, experts=16, top=4, io="bf16", rows=False, bias=False, group=128),
        # a decoding step of 64 chats: a few rows for each of 64 experts
        _experts("experts_decode", m=64, k=2048, n=1536, experts=64, top=8, io="bf16", rows=False, bias=False, group=256),
        # a prompt through 64 experts
        _experts("experts_prompt", m=4096, k=2048, n=1536, experts=64, top=8, io="bf16", rows=False, bias=False, group=128),
        # a prompt of odd length through eight wide experts, with bias and a scale for each channel
        _experts("experts_wide", m=1537, k=4096, n=14336, experts=8, top=2, io="fp16", rows=True, bias=True, group=256),
    ]


def _block(name, m, k, io, post, pre, mods, routes, group, n):
    return {"name": name, "op": "block", "m": m, "k": k, "io": io, "post": post, "pre": pre, "mods": mods,
            "routes": routes, "group": group, "n": n}


def _lora(name, m, k, n, io, adapters, rank, spread, rows, group):
    return {"name": name, "op": "lora", "m": m, "k": k, "n": n, "io": io, "adapters": adapters, "rank": rank,
            "spread": spread, "rows": rows, "group": group}


def _experts(name, m, k, n, experts, top, io, rows, bias, group):
    return {"name": name, "op": "experts", "m": m, "k": k, "n": n, "experts": experts, "top": top, "io": io,
            "rows": rows, "bias": bias, "group": group}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("block", "lora", "experts"))
    io, group = rng.choice(("bf16", "fp16")), rng.choice((128, 256))
    if op == "block":
        k = group * _log(rng, 4, 8192 // group)
        coded = rng.random() < 0.4
        case = _block("", m=min(_log(rng, 1, 16896), (16896 * 6144) // k), k=k, io=io,
                      post=rng.choice(("none", "rms", "layer")), pre=rng.choice(("rms", "layer")),
                      mods=rng.choice((0, 1, 5)), routes=rng.choice((0, 0, 2, 6)), group=group if coded else 0,
                      n=_log(rng, 64, 2048) if coded else 0)
        case["m"] = case["m"] if not case["routes"] else max(1, case["m"] // (1 + case["routes"]))
    elif op == "lora":
        k, n = group * _log(rng, 4, 12288 // group), 8 * _log(rng, 64, 1536)
        case = _lora("", m=min(_log(rng, 1, 4608), max(1, 2 ** 37 // (k * n))), k=k, n=n, io=io,
                     adapters=_log(rng, 1, 48), rank=_log(rng, 4, 128), spread=rng.random() < 0.5,
                     rows=rng.random() < 0.5, group=group)
    else:
        k, n = group * _log(rng, 4, 4096 // group), 8 * _log(rng, 64, 512)
        experts = _log(rng, 4, 64)
        case = _experts("", m=_log(rng, 1, 4096), k=k, n=n, experts=experts, top=rng.randint(1, min(8, experts)), io=io,
                        rows=rng.random() < 0.5, bias=rng.random() < 0.5, group=group)
        case["m"] = max(1, min(case["m"], 2 ** 36 // (k * n * case["top"])))
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _stream(g, m, k, io):
    """Activations with a few channels far above the others, as these layers meet them."""
    x = _normal(g, m, k)
    x[:, torch.randint(0, k, (max(1, k // 100),), generator=g, device="cuda")] *= 20.0
    return x.to(_IO[io])


def _codes(g, *shape):
    return (_normal(g, *shape) * 28.0).round_().clamp_(-127, 127).to(torch.int8)


def _weight_scales(g, *shape):
    return (0.8 + 0.4 * torch.rand(shape, generator=g, device="cuda")) * (0.02 / 28.0)


def prepare(case, seed):
    g = _generator(seed)
    return {"block": _prepare_block, "lora": _prepare_lora, "experts": _prepare_experts}[case["op"]](case, g)


def _prepare_block(case, g):
    m, k, io = case["m"], case["k"], _IO[case["io"]]
    s = {"case": case, "h": _stream(g, m, k, case["io"])}
    if case["routes"]:
        # the experts' rows lie sorted by expert, so a token's rows are anywhere among them
        t = case["routes"]
        s["u"] = _normal(g, m * t, k).to(io)
        s["row"] = torch.randperm(m * t, generator=g, device="cuda").view(m, t).to(torch.int32)
        s["weight"] = torch.softmax(_normal(g, m, t), dim=1)
    else:
        s["u"] = _normal(g, m, k).to(io)
    s["post_weight"] = (1 + 0.1 * _normal(g, k)).to(io) if case["post"] != "none" else None
    s["pre_weight"] = (1 + 0.1 * _normal(g, k)).to(io) if case["pre"] == "rms" else None
    if case["mods"]:
        # one row of gate, shift and scale for each request, as one projection gives them
        b = case["mods"]
        s["mod"] = (0.3 * _normal(g, b, 3 * k)).to(io)
        cuts = torch.sort(torch.randint(0, m + 1, (b - 1,), generator=g, device="cuda")).values
        s["index"] = torch.bucketize(torch.arange(m, device="cuda"), cuts, right=True).to(torch.int32)
    if case["group"]:
        s["wq"], s["w_scale"] = _codes(g, case["n"], k), _weight_scales(g, 1)
    return s


def _prepare_lora(case, g):
    m, k, n, io, a = case["m"], case["k"], case["n"], _IO[case["io"]], case["adapters"]
    ranks = torch.full((a,), case["rank"], dtype=torch.int64, device="cuda")
    if case["spread"]:
        ranks = torch.randint(1, case["rank"] + 1, (a,), generator=g, device="cuda")
        ranks[0] = case["rank"]
    offsets = torch.zeros(a + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(ranks, 0)
    total = int(offsets[-1])
    # a batch is its requests one after another, each with its adapter; some have none
    cuts = torch.sort(torch.randint(0, m + 1, (a - 1,), generator=g, device="cuda")).values
    index = torch.bucketize(torch.arange(m, device="cuda"), cuts, right=True)
    if m <= a:
        index = torch.randperm(a, generator=g, device="cuda")[:m]
    elif case["spread"]:
        index = torch.where(index % 5 == 3, -1, index)
    return {"case": case, "x": _stream(g, m, k, case["io"]), "wq": _codes(g, n, k),
            "w_scale": _weight_scales(g, n if case["rows"] else 1), "bias": (0.1 * _normal(g, n)).to(io),
            "a": (_normal(g, total, k) / math.sqrt(k)).to(io), "b": (0.2 * _normal(g, total, n)).to(io),
            "scale": 0.5 + torch.rand(a, generator=g, device="cuda"), "offsets": offsets,
            "index": index.to(torch.int32)}


def _prepare_experts(case, g):
    m, k, n, e, top = case["m"], case["k"], case["n"], case["experts"], case["top"]
    # some experts are liked more than others
    score = _normal(g, m, e) + 0.5 * _normal(g, e)
    chosen = torch.topk(score, top, dim=1).indices.reshape(-1)
    expert, order = torch.sort(chosen, stable=True)
    counts = torch.bincount(expert, minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return {"case": case, "x": _stream(g, m, k, case["io"]), "wq": _codes(g, e, n, k),
            "w_scale": _weight_scales(g, e, n) if case["rows"] else _weight_scales(g, e),
            "bias": (0.1 * _normal(g, e, n)).to(_IO[case["io"]]) if case["bias"] else None,
            "rows": (order // top).to(torch.int32), "offsets": offsets, "most": int(counts.max())}


# ---------------------------------------------------------------- one pass

def run(state):
    return {"block": _run_block, "lora": _run_lora, "experts": _run_experts}[state["case"]["op"]](state)


def _run_block(s):
    c = s["case"]
    k = c["k"]
    gate, shift, scale = (s["mod"][:, :k], s["mod"][:, k:2 * k], s["mod"][:, 2 * k:]) if c["mods"] else (None,) * 3
    if own:
        from w8a8_rotated_int8_convrot_amd import binding as B
        got = B.convrot_block_norm(
            s["h"], s["u"], routes=(s["row"], s["weight"]) if c["routes"] else None, post_norm=c["post"],
            post_weight=s["post_weight"], gate=gate, pre_norm=c["pre"], pre_weight=s["pre_weight"], scale=scale,
            shift=shift, mod_index=s["index"] if c["mods"] else None, eps=_EPS, group=c["group"])
        if not c["group"]:
            return got
        h, q, q_scale = got
        return h, B.convrot_gemm_dequant_ex(q, q_scale, s["wq"], s["w_scale"], out_dtype=_IO[c["io"]])
    io = _IO[c["io"]]
    u = s["u"].float()
    if c["routes"]:
        u = (u[s["row"].long()] * s["weight"][:, :, None]).sum(1)
    u = _norm(u, c["post"], s["post_weight"])
    at = s["index"].long() if c["mods"] else None
    if c["mods"]:
        u = u * gate.float()[at]
    h = (s["h"].float() + u).to(io)
    y = _norm(h.float(), c["pre"], s["pre_weight"])
    if c["mods"]:
        y = y * (1 + scale.float()[at]) + shift.float()[at]
    if not c["group"]:
        return h, y.to(io)
    return h, _project(*_coded(y, c["group"]), s["wq"], s["w_scale"]).to(io)


def _norm(x, kind, weight):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + _EPS)
    return x if weight is None else x * weight.float()


def _hadamard(g):
    """H_g / sqrt(g): the sign is the parity of the bits that row and column share."""
    i = torch.arange(g, device="cuda")
    b = i[:, None] & i[None, :]
    b = b ^ (b >> 4)
    b = b ^ (b >> 2)
    b = b ^ (b >> 1)
    return (1.0 - 2.0 * (b & 1)) / math.sqrt(g)


def _coded(x, g):
    """int8 codes (as fp32 values) and scales of the rotated rows."""
    v = (x.reshape(-1, g) @ _hadamard(g)).reshape(x.shape)
    s = v.abs().amax(1) / 127.0
    q = torch.where(s[:, None] > 0, v / s[:, None], 0.0).round().clamp(-127, 127)
    return q, s


def _project(q, s, wq, w_scale):
    return (q @ wq.float().t()) * (s[:, None] * w_scale[None, :])


def _run_lora(s):
    c = s["case"]
    if own:
        from w8a8_rotated_int8_convrot_amd import binding as B
        return B.convrot_linear_lora(s["x"], s["wq"], s["w_scale"], c["group"], s["a"], s["b"], s["scale"], s["offsets"],
                                     s["index"], c["rank"], bias=s["bias"])
    x = s["x"].float()
    y = _project(*_coded(x, c["group"]), s["wq"], s["w_scale"]) + s["bias"].float()
    # every rank row of every adapter, then only those of the token's own
    at = torch.arange(s["a"].shape[0], device="cuda", dtype=torch.int32)
    owner = torch.searchsorted(s["offsets"][1:], at, right=True)
    t = x @ s["a"].float().t()
    t = torch.where(s["index"][:, None] == owner[None, :], t * s["scale"][owner], 0.0)
    return (y + t @ s["b"].float()).to(_IO[c["io"]])


def _run_experts(s):
    c = s["case"]
    if own:
        from w8a8_rotated_int8_convrot_amd import binding as B
        return B.convrot_grouped_linear(s["x"], s["wq"], s["w_scale"], c["group"], s["offsets"], rows=s["rows"],
                                        bias=s["bias"])
    q, qs = _coded(s["x"].float(), c["group"])
    # each expert's rows in a block as long as the longest, one batched product
    p, e = s["rows"].shape[0], c["experts"]
    rows, start = s["rows"].long(), s["offsets"][:-1].long()
    at = torch.arange(p, device="cuda")
    owner = torch.searchsorted(s["offsets"][1:], at.to(torch.int32), right=True)
    padded = q.new_zeros(e, s["most"], c["k"])
    padded[owner, at - start[owner]] = q[rows]
    y = torch.bmm(padded, s["wq"].float().transpose(1, 2))[owner, at - start[owner]]
    ws = s["w_scale"] if c["rows"] else s["w_scale"][:, None]
    y = y * (qs[rows][:, None] * ws[owner])
    if s["bias"] is not None:
        y = y + s["bias"].float()[owner]
    return y.to(_IO[c["io"]])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    m, k = case["m"], case["k"]
    if case["op"] == "block":
        # stream and block output in, stream and norm out; coded, the codes' product too
        rows = m * max(1, case["routes"])
        out = 2 * m * case["n"] + case["n"] * k if case["group"] else 2 * m * k
        return {"bytes": 4 * m * k + 2 * rows * k + 8 * m * case["routes"] + 6 * case["mods"] * k + out,
                "flops": 20 * m * k + 2 * rows * k + 2 * m * k * case["n"]}
    n = case["n"]
    if case["op"] == "lora":
        ranks = case["rank"] if not case["spread"] else (case["rank"] + 1) / 2
        used = min(m, case["adapters"]) * ranks
        return {"bytes": 2 * m * k + n * k + 2 * used * (k + n) + 2 * m * n + 2 * n,
                "flops": 2 * m * n * k + 2 * m * ranks * (k + n)}
    p, e = m * case["top"], case["experts"]
    met = e * (1 - (1 - case["top"] / e) ** m)
    return {"bytes": 2 * m * k + met * n * k + 2 * p * n + 4 * p, "flops": 2 * p * n * k}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"block": _exact_block, "lora": _exact_lora, "experts": _exact_experts}[case["op"]](s)


def _exact_codes(x, g):
    """Butterflies of half-span 1, 2, ..., g / 2, one by one, then absmax / 127 and the nearest code."""
    m, k = x.shape
    v, half = x.double(), 1
    while half < g:
        v = v.view(m, k // (2 * half), 2, half)
        v = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), 2)
        half *= 2
    v = v.reshape(m, k) * g ** -0.5
    s = v.abs().max(1).values / 127
    safe = torch.where(s > 0, s, torch.ones_like(s))
    return torch.round(v / safe[:, None]).clamp(-127, 127), s


def _exact_norm(x, kind, weight):
    if kind == "none":
        return x
    mean = x.sum(1, keepdim=True) / x.shape[1] if kind == "layer" else 0.0
    var = ((x - mean) ** 2).sum(1, keepdim=True) / x.shape[1]
    y = (x - mean) / torch.sqrt(var + _EPS)
    return y if weight is None else y * weight.double()


def _exact_block(s):
    c = s["case"]
    k, u = c["k"], s["u"].double()
    if c["routes"]:
        total = torch.zeros(c["m"], k, dtype=torch.float64, device="cuda")
        for j in range(c["routes"]):
            total += s["weight"][:, j, None].double() * u[s["row"][:, j].long()]
        u = total
    u = _exact_norm(u, c["post"], s["post_weight"])
    mod = s["mod"].double()[s["index"].long()] if c["mods"] else None
    h = s["h"].double() + (u if mod is None else mod[:, :k] * u)
    # the norm is that of the stream as it is stored
    y = _exact_norm(h.to(_IO[c["io"]]).double(), c["pre"], s["pre_weight"])
    if mod is not None:
        y = y * (1 + mod[:, 2 * k:]) + mod[:, k:2 * k]
    if not c["group"]:
        return h, y
    q, qs = _exact_codes(y, c["group"])
    return h, (q @ s["wq"].double().t()) * qs[:, None] * s["w_scale"].double()


def _exact_lora(s):
    x = s["x"].double()
    q, qs = _exact_codes(x, s["case"]["group"])
    y = (q @ s["wq"].double().t()) * qs[:, None] * s["w_scale"].double() + s["bias"].double()
    ends = s["offsets"].tolist()
    for a in range(s["case"]["adapters"]):
        mine = torch.nonzero(s["index"] == a).flatten()
        lo, hi = ends[a], ends[a + 1]
        y[mine] += s["scale"][a].double() * ((x[mine] @ s["a"][lo:hi].double().t()) @ s["b"][lo:hi].double())
    return y


def _exact_experts(s):
    c = s["case"]
    q, qs = _exact_codes(s["x"], c["group"])
    y = torch.empty(s["rows"].shape[0], c["n"], dtype=torch.float64, device="cuda")
    ends = s["offsets"].tolist()
    for e in range(c["experts"]):
        at = s["rows"][ends[e]:ends[e + 1]].long()
        part = (q[at] @ s["wq"][e].double().t()) * qs[at][:, None] * s["w_scale"][e].double()
        y[ends[e]:ends[e + 1]] = part if s["bias"] is None else part + s["bias"][e].double()
    return y
