"""Operators between two layers, as cases that can be timed and compared.

What a transformer block does between its QKV layer and its output layer, in
its plain form (elementary torch operations in 32 bits, 64 where a border
between two codes or the angle of a far position asks for them, rounded once at
the end) and, where ``own`` is true, through the calls of this package:

* rope:      rotary positions on the query and key heads of a batch of tokens;
* append:    new tokens into a paged cache that holds keys and values as 4-bit
             codes of the rotated head, and the same tokens read back from it;
* attention: new tokens' queries over that cache, from one token of one
             sequence to whole prompts;
* copy:      pages of the cache moved, for a forked sequence or to close gaps.

The cache is bytes, [pages, page_bytes]; a page is [heads][units] of 32 tokens,
and a unit of head size D is, one after another,
    key codes     [32][D / 2] bytes: dim 2 i in the low half of byte i, 2 i + 1 above it
    value codes   [4][D] 32-bit words: token 8 o + i of dim d in bits 4 i .. 4 i + 3 of word [o][d]
    key scales    [32] bf16
    value scales  [32] bf16
with codes -7 .. 7 held as code + 8.
"""
import math

import torch

own = False

_IO = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a chat: all its heads, where latency counts
        _rope("rope_one_token", m=1, hq=32, hk=8, d=128, rot=128, io="bf16", layout="half", kind="none", far=2000),
        # a batch of long prompts, half of each head turned, positions stretched past the trained length
        _rope("rope_prompt", m=4608, hq=40, hk=8, d=128, rot=64, io="fp16", layout="interleaved", kind="yarn", far=120000),
        # a decoding step of 64 chats, one new token each
        _append("append_decode", seqs=64, new=1, old=4000, hk=8, d=128, page=64, io="bf16"),
        # three prompts of odd lengths, one of them the continuation of a cached beginning
        _append("append_prompt", seqs=3, new=4099, old=333, hk=16, d=64, page=32, io="fp16"),
        # one token of one chat
        _attention("attention_one_token", seqs=1, new=1, old=1000, hq=32, hk=8, d=128, page=64, io="bf16", window=0),
        # a decoding step of 64 chats of all lengths up to 8192
        _attention("attention_decode", seqs=64, new=1, old=8191, hq=32, hk=8, d=128, page=64, io="bf16", window=0),
        # four very long documents, one new token each
        _attention("attention_long", seqs=4, new=1, old=131000, hq=64, hk=8, d=128, page=256, io="bf16", window=0),
        # five drafted tokens of each of 16 chats checked at once, wide heads, a sliding window
        _attention("attention_drafts", seqs=16, new=5, old=4000, hq=16, hk=8, d=256, page=32, io="fp16", window=1024),
        # one whole prompt as long as an image's token sequence at 1024^2
        _attention("attention_prompt", seqs=1, new=4608, old=0, hq=32, hk=8, d=128, page=128, io="bf16", window=0),
        # pieces of three prompts of odd lengths behind what is cached of them, a key head for each query head
        _attention("attention_pieces", seqs=3, new=1001, old=16000, hq=24, hk=24, d=64, page=64, io="fp16", window=0),
        # a sequence forked: its last, partly filled page copied in one layer
        _copy("copy_fork", pairs=1, layers=1, hk=8, d=128, page=64),
        # gaps closed in all layers of a cache
        _copy("copy_compact", pairs=200, layers=32, hk=8, d=128, page=64),
    ]


def _rope(name, m, hq, hk, d, rot, io, layout, kind, far):
    return {"name": name, "op": "rope", "m": m, "hq": hq, "hk": hk, "d": d, "rot": rot, "io": io, "layout": layout,
            "kind": kind, "far": far}


def _append(name, seqs, new, old, hk, d, page, io):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "old": old, "hk": hk, "d": d, "page": page, "io": io}


def _attention(name, seqs, new, old, hq, hk, d, page, io, window):
    return {"name": name, "op": "attention", "seqs": seqs, "new": new, "old": old, "hq": hq, "hk": hk, "d": d,
            "page": page, "io": io, "window": window}


def _copy(name, pairs, layers, hk, d, page):
    return {"name": name, "op": "copy", "pairs": pairs, "layers": layers, "hk": hk, "d": d, "page": page}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "attention", "attention", "copy"))
    io, page = rng.choice(("bf16", "fp16")), rng.choice((32, 64, 128, 256))
    hk, d = rng.choice((1, 2, 3, 4, 8, 8, 16)), rng.choice((64, 128, 128, 256))
    if op == "rope":
        d = rng.choice((64, 80, 96, 128, 256))
        hq = hk * rng.choice((1, 2, 4, 5, 7))
        case = _rope("", m=min(_log(rng, 1, 8192), max(1, 2 ** 24 // ((hq + hk) * d))), hq=hq, hk=hk, d=d,
                     rot=rng.choice((d, d, d // 2, d // 4)), io=io, layout=rng.choice(("half", "interleaved")),
                     kind=rng.choice(("none", "linear", "ntk", "yarn", "bands")), far=_log(rng, 1000, 1000000))
    elif op == "append":
        seqs = _log(rng, 1, 64)
        new = rng.choice((1, _log(rng, 1, 4096)))
        case = _append("", seqs=seqs, new=max(1, min(new, 2 ** 24 // (seqs * hk * d))), old=_log(rng, 1, 5000) - 1, hk=hk,
                       d=d, page=page, io=io)
    elif op == "attention":
        g = rng.choice((1, 2, 4, 5, 7, 8))
        if rng.random() < 0.6:
            seqs, new = _log(rng, 1, 64), rng.choice((1, 1, 2, 7))
            old = _log(rng, 1, max(2, min(60000, 2 ** 28 // (seqs * hk * d)))) - 1
        else:
            seqs, new = _log(rng, 1, 6), _log(rng, 16, 3000)
            new = max(1, new // seqs)
            old = rng.choice((0, _log(rng, 1, 8000)))
            old = max(0, min(old, 2 ** 35 // (seqs * new * hk * g * d) - new))
        case = _attention("", seqs=seqs, new=new, old=old, hq=hk * g, hk=hk, d=d, page=page, io=io,
                          window=rng.choice((0, 0, 0, _log(rng, 1, 4096))))
    else:
        layers = _log(rng, 1, 32)
        case = _copy("", pairs=max(1, min(_log(rng, 1, 300), 2 ** 28 // (layers * hk * d * page))), layers=layers, hk=hk,
                     d=d, page=page)
    del case["name"]
    return case


def _lens(case):
    """(tokens cached before, new tokens) of each sequence: spread up to the case's own, the first the longest."""
    b = case["seqs"]
    return [(case["old"] * (b - i) // b if i else case["old"], max(1, case["new"] * (2 * b - i) // (2 * b)) if i else case["new"])
            for i in range(b)]


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _heads(g, m, h, d, io):
    """Head vectors with a few dims above the others, as keys and values have them."""
    x = _normal(g, m, h, d)
    x[:, :, torch.randint(0, d, (max(1, d // 40),), generator=g, device="cuda")] *= 8.0
    return x.to(_IO[io])


def _unit_bytes(d):
    return 32 * d + 128


def _page_bytes(case):
    return case["hk"] * (case["page"] // 32) * _unit_bytes(case["d"])


def _random_pages(g, n, case):
    """n pages of codes and scales as rotated heads give them."""
    d, step = case["d"], _unit_bytes(case["d"])
    pages = torch.empty(n, _page_bytes(case), dtype=torch.uint8, device="cuda")
    units = pages.view(-1, step)
    for lo in range(0, units.shape[0], 8192):
        u = units[lo:lo + 8192]
        codes = (2.6 * _normal(g, u.shape[0], 64 * d)).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        u[:, :32 * d] = codes[:, 0::2] | (codes[:, 1::2] << 4)
        u[:, 32 * d:] = (0.25 + 0.3 * torch.rand(u.shape[0], 64, generator=g, device="cuda")).to(torch.bfloat16).view(torch.uint8)
    return pages


def _sequences(g, case):
    """Page table, tokens before and row offsets of the case's sequences, their pages anywhere in the cache."""
    lens, page = _lens(case), case["page"]
    need = [(old + new + page - 1) // page for old, new in lens]
    n = sum(need) + 3
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at, offsets = 0, [0]
    for b, (k, (_, new)) in enumerate(zip(need, lens)):
        table[b, :k] = order[at:at + k]
        at += k
        offsets.append(offsets[-1] + new)
    return {"lens": lens, "n_pages": n, "table": table, "rows": offsets[-1],
            "starts": torch.tensor([old for old, _ in lens], dtype=torch.int32, device="cuda"),
            "offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    g = _generator(seed)
    return {"rope": _prepare_rope, "append": _prepare_append, "attention": _prepare_attention,
            "copy": _prepare_copy}[case["op"]](case, g)


def _scaling(case):
    kind = case["kind"]
    return dict(kind=kind, factor=1.0 if kind == "none" else 8.0, original_length=8192,
                low=1.0, high=32.0 if kind == "yarn" else 4.0)


def _prepare_rope(case, g):
    m, d = case["m"], case["d"]
    # queries, keys and values of a token are one row of the QKV layer's output
    qkv = _normal(g, m, case["hq"] + 2 * case["hk"], d).to(_IO[case["io"]])
    first = torch.randint(0, case["far"], (1,), generator=g, device="cuda")
    positions = ((first + torch.arange(m, device="cuda")) % case["far"]).to(torch.int32)
    if own:
        from w8a8_rotated_int8_convrot_amd import binding as B
        freqs, scale = B.convrot_rope_frequencies(case["rot"], base=500000.0, device="cuda", **_scaling(case))
    else:
        freqs, scale = _frequencies(case["rot"], 500000.0, **_scaling(case))
    return {"case": case, "q": qkv[:, :case["hq"]], "k": qkv[:, case["hq"]:case["hq"] + case["hk"]],
            "positions": positions, "freqs": freqs, "scale": scale}


def _prepare_append(case, g):
    s = _sequences(g, case)
    if own:
        s["pages"] = torch.empty(s["n_pages"], _page_bytes(case), dtype=torch.uint8, device="cuda")
        s["pages"].random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(1))
    else:
        # the plain cache: a token's packed codes and its scale, [pages, page, heads]
        shape = (s["n_pages"], case["page"], case["hk"])
        s["plain"] = [(torch.zeros(*shape, case["d"] // 2, dtype=torch.uint8, device="cuda"),
                       torch.zeros(shape, dtype=torch.bfloat16, device="cuda")) for _ in range(2)]
    return {"case": case, "k": _heads(g, s["rows"], case["hk"], case["d"], case["io"]),
            "v": _heads(g, s["rows"], case["hk"], case["d"], case["io"]), **s}


def _prepare_attention(case, g):
    s = _sequences(g, case)
    q = (2.0 * _normal(g, s["rows"], case["hq"], case["d"])).to(_IO[case["io"]])
    return {"case": case, "pages": _random_pages(g, s["n_pages"], case), "q": q, **s}


def _prepare_copy(case, g):
    n = 2 * case["pairs"] + 2
    pages = torch.empty(case["layers"], n, _page_bytes(case), dtype=torch.uint8, device="cuda")
    pages.random_(0, 256, generator=g)
    # the host keeps the lists of free and live pages
    order = torch.randperm(n, generator=g, device="cuda").tolist()
    return {"case": case, "pages": pages, "pairs": list(zip(order[:case["pairs"]], order[case["pairs"]:2 * case["pairs"]]))}


# ---------------------------------------------------------------- one pass

def run(state):
    return {"rope": _run_rope, "append": _run_append, "attention": _run_attention, "copy": _run_copy}[state["case"]["op"]](state)


def _frequencies(rot, base, kind, factor, original_length, low, high):
    """Radians per position of each turned pair, and the factor of sine and cosine."""
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    scale = 1.0
    if kind == "linear":
        f = f / factor
    elif kind == "yarn":
        # pairs that turn more than `high` times over the trained length stay, less than `low` are interpolated
        at = [rot * math.log(original_length / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (high, low)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    elif kind == "bands":
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f.cuda(), scale


def _run_rope(s):
    c = s["case"]
    if own:
        from w8a8_rotated_int8_convrot_amd import binding as B
        return B.convrot_rope(s["q"], s["k"], s["positions"], s["freqs"], scale=s["scale"], layout=c["layout"])
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = ((f(angle) * s["scale"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    return tuple(_turned(x, cos, sin, c["rot"], c["layout"]).to(_IO[c["io"]]) for x in (s["q"], s["k"]))


def _turned(x, cos, sin, rot, layout):
    x = x.float()
    part, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((part, rest), -1)


def _hadamard(d, dtype):
    """H_d: the sign is the parity of the bits that row and column share."""
    i = torch.arange(d, device="cuda")
    b = i[:, None] & i[None, :]
    b = b ^ (b >> 4)
    b = b ^ (b >> 2)
    b = b ^ (b >> 1)
    return (1 - 2 * (b & 1)).to(dtype)


def _run_append(s):
    c = s["case"]
    if own:
        from w8a8_rotated_int8_convrot_amd import binding as B
        B.convrot_cache_append(s["pages"], s["table"], s["starts"], s["offsets"], s["k"], s["v"], c["page"])
        return B.convrot_cache_read(s["pages"], s["table"], s["starts"], s["offsets"], s["rows"], c["hk"], c["d"], c["page"],
                                    _IO[c["io"]])
    d = c["d"]
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"][1:], row, right=True)
    at = (s["starts"][seq] + row - s["offsets"][seq]).long()
    page, slot = s["table"][seq, at // c["page"]].long(), at % c["page"]
    out = []
    for x, (codes, scales) in zip((s["k"], s["v"]), s["plain"]):
        # whether a value lies below or above the border between two codes takes 64 bits
        r = (x.double() @ _hadamard(d, torch.float64)) * (1 / math.sqrt(d))
        sc = (r.abs().amax(-1) / 7).float().to(torch.bfloat16)
        q = torch.where(sc[..., None] > 0, r / sc[..., None].double(), 0.0).round().clamp(-7, 7).add(8).to(torch.uint8)
        codes[page, slot] = q[..., 0::2] | (q[..., 1::2] << 4)
        scales[page, slot] = sc
        got = codes[page, slot]
        q = torch.stack((got & 15, got >> 4), -1).flatten(-2).float() - 8
        r = (q * scales[page, slot].float()[..., None]) @ _hadamard(d, torch.float32)
        out.append((r * (1 / math.sqrt(d))).to(_IO[c["io"]]))
    return tuple(out)


def _unpack(pages, d, hk, page):
    """Key and value codes [heads, tokens, D] and their scales [heads, tokens] of one sequence's pages."""
    n, units = pages.shape[0], page // 32
    u = pages.view(n, hk, units, _unit_bytes(d)).transpose(0, 1).reshape(hk, n * units, _unit_bytes(d))
    k = u[..., :16 * d].reshape(hk, -1, d // 2)
    k = torch.stack((k & 15, k >> 4), -1).flatten(-2).float() - 8
    v = u[..., 16 * d:32 * d].reshape(hk, -1, 4, d, 4)
    v = torch.stack((v & 15, v >> 4), -1).reshape(hk, -1, 4, d, 8).transpose(3, 4).reshape(hk, -1, d).float() - 8
    scales = u[..., 32 * d:].reshape(hk, n * units, 2, 32, 2).view(torch.bfloat16).float()
    return k, v, scales[:, :, 0].reshape(hk, -1), scales[:, :, 1].reshape(hk, -1)


def _run_attention(s):
    c = s["case"]
    d, hk, g = c["d"], c["hk"], c["hq"] // c["hk"]
    if own:
        from w8a8_rotated_int8_convrot_amd import binding as B
        return B.convrot_cache_attention(s["q"], s["pages"], s["table"], s["starts"], s["offsets"], hk, c["page"],
                                         window=c["window"])
    turn = _hadamard(d, torch.float32) * (1 / math.sqrt(d))
    out, at = torch.empty_like(s["q"]), 0
    for b, (old, n) in enumerate(s["lens"]):
        end = old + n
        used = (end + c["page"] - 1) // c["page"]
        k, v, ks, vs = _unpack(s["pages"][s["table"][b, :used].long()], d, hk, c["page"])
        k, v = k[:, :end] * ks[:, :end, None], v[:, :end] * vs[:, :end, None]
        q = (s["q"][at:at + n].float() @ turn).view(n, hk, g, d).permute(1, 2, 0, 3).reshape(hk, g * n, d)
        t = (torch.bmm(q, k.transpose(1, 2).contiguous()) * (1 / math.sqrt(d))).view(hk, g, n, end)
        pos = torch.arange(old, end, device="cuda")[:, None]
        key = torch.arange(end, device="cuda")[None, :]
        hidden = key > pos
        if c["window"]:
            hidden = hidden | (key <= pos - c["window"])
        t = t.masked_fill_(hidden, -math.inf)
        t = t.sub_(t.amax(-1, keepdim=True)).exp_()
        t = t.div_(t.sum(-1, keepdim=True)).view(hk, g * n, end)
        o = torch.bmm(t, v) @ turn
        out[at:at + n] = o.view(hk, g, n, d).permute(2, 0, 1, 3).reshape(n, hk * g, d).to(_IO[c["io"]])
        at += n
    return out


def _run_copy(s):
    if own:
        from w8a8_rotated_int8_convrot_amd import binding as B
        B.convrot_cache_copy(s["pages"], s["pairs"])
        return s["pages"]
    src, dst = torch.tensor(s["pairs"], device="cuda").t()
    s["pages"][:, dst] = s["pages"][:, src]
    return s["pages"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "rope":
        n = case["m"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 4 * n + 4 * case["m"], "flops": 3 * n * case["rot"] // case["d"]}
    if op == "copy":
        return {"bytes": 2 * case["pairs"] * case["layers"] * _page_bytes(case), "flops": 0}
    d, hk, lens = case["d"], case["hk"], _lens(case)
    rows = sum(n for _, n in lens)
    if op == "append":
        # 16-bit rows in, codes and scales out, and the way back
        n = 2 * rows * hk
        return {"bytes": 2 * n * (2 * d + d // 2 + 2), "flops": 4 * n * d * int(math.log2(d))}
    keys = pairs = 0
    for old, n in lens:
        w = case["window"] or old + n
        keys += min(old + n, w + n - 1)
        pairs += sum(min(p + 1, w) for p in range(old, old + n))
    return {"bytes": keys * hk * (d + 4) + 4 * rows * case["hq"] * d, "flops": 4 * pairs * case["hq"] * d}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attention": _exact_attention, "copy": _exact_copy}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    rot, pairs = c["rot"], c["rot"] // 2
    f, scale = _frequencies(rot, 500000.0, **_scaling(c))
    out = []
    for x in (s["q"], s["k"]):
        y = x.double()
        for i in range(pairs):
            a, b = (i, i + pairs) if c["layout"] == "half" else (2 * i, 2 * i + 1)
            turn = torch.polar(torch.full((c["m"],), float(scale), dtype=torch.float64, device="cuda"),
                               s["positions"].double() * f[i])
            z = torch.complex(y[:, :, a], y[:, :, b]) * turn[:, None]
            y[:, :, a], y[:, :, b] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _butterfly(x):
    """H_d times the rows, by stages of half-span 1, 2, ..., d / 2."""
    shape, half = x.shape, 1
    while half < shape[-1]:
        x = x.reshape(-1, shape[-1] // (2 * half), 2, half)
        x = torch.stack((x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]), 2)
        half *= 2
    return x.reshape(shape)


def _exact_append(s):
    d, out = s["case"]["d"], []
    for x in (s["k"], s["v"]):
        r = _butterfly(x.double()) * d ** -0.5
        scale = (r.abs().max(-1, keepdim=True).values / 7).float().bfloat16().double()
        safe = torch.where(scale > 0, scale, torch.ones_like(scale))
        out.append(_butterfly(torch.round(r / safe).clamp(-7, 7) * scale) * d ** -0.5)
    return tuple(out)


def _exact_attention(s):
    c = s["case"]
    d, hk, g, page, step = c["d"], c["hk"], c["hq"] // c["hk"], c["page"], _unit_bytes(c["d"])
    out = torch.zeros(s["rows"], c["hq"], d, dtype=torch.float64, device="cuda")
    nib = 4 * torch.arange(8, device="cuda", dtype=torch.int32)
    at = 0
    for b, (old, n) in enumerate(s["lens"]):
        end = old + n
        used = s["table"][b, :(end + page - 1) // page].long()
        for h in range(hk):
            u = s["pages"].view(-1, hk, page // 32, step)[used, h].reshape(-1, step)
            words = u[:, :32 * d].contiguous().view(torch.int32)
            codes = ((words[:, :, None] >> nib) & 15).double() - 8
            k = codes[:, :4 * d].reshape(-1, 32, d)
            v = codes[:, 4 * d:].reshape(-1, 4, d, 8).permute(0, 1, 3, 2).reshape(-1, 32, d)
            sc = u[:, 32 * d:].contiguous().view(torch.bfloat16).double()
            # the head itself: the rotation taken back
            k = (_butterfly(k * sc[:, :32, None]) * d ** -0.5).reshape(-1, d)[:end]
            v = (_butterfly(v * sc[:, 32:, None]) * d ** -0.5).reshape(-1, d)[:end]
            for lo in range(0, n, 1024):
                hi = min(n, lo + 1024)
                pos = torch.arange(old + lo, old + hi, device="cuda")[:, None]
                key = torch.arange(end, device="cuda")[None, :]
                seen = key <= pos
                if c["window"]:
                    seen &= key > pos - c["window"]
                for j in range(h * g, h * g + g):
                    t = (s["q"][at + lo:at + hi, j].double() @ k.t()) / math.sqrt(d)
                    w = torch.softmax(torch.where(seen, t, -math.inf), 1)
                    out[at + lo:at + hi, j] = w @ v
        at += n
    return out


def _exact_copy(s):
    pages = s["pages"].clone()
    for src, dst in s["pairs"]:
        pages[:, dst] = s["pages"][:, src]
    return pages
