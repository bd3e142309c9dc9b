"""The paged 4-bit cache, its rotary positions and its attention in 64 bits, from the formulas
(include/convrot.h), for the tests that compare the kernels with them."""
import math

import torch


def unit_bytes(D):
    return 32 * D + 128


def page_bytes(page, H, D):
    return H * (page // 32) * unit_bytes(D)


def butterfly(x):
    """x H_D over the last dim, by stages."""
    shape, h = x.shape, 1
    while h < shape[-1]:
        x = x.reshape(-1, shape[-1] // (2 * h), 2, h)
        x = torch.stack((x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]), 2)
        h *= 2
    return x.reshape(shape)


def encode(x):
    """Codes (as held, 1 .. 15) and bf16 scales of rows [..., D] of 16-bit values."""
    v = butterfly(x.double()) * (1 / math.sqrt(x.shape[-1]))
    s = (v.abs().amax(-1) / 7).float().to(torch.bfloat16)
    finite = torch.isfinite(x.double()).all(-1) & torch.isfinite(s.double())
    s = torch.where(finite, s, torch.full_like(s, math.nan))
    sd = s.double()[..., None]
    c = torch.where(finite[..., None] & (sd > 0), v / sd, torch.zeros_like(v)).round().clamp(-7, 7)
    return c.to(torch.int64) + 8, s


def write(pages, page, H, D, table, starts, offsets, k, v):
    """convrot_cache_append on a CPU copy of the pages, token by token."""
    M, n = k.shape[0], pages.shape[0]
    units = pages.view(n, H, page // 32, unit_bytes(D))
    (kc, ks), (vc, vs) = encode(k), encode(v)
    for b in range(table.shape[0]):
        lo = min(max(int(offsets[b]), 0), M)
        for r in range(lo, max(lo, min(int(offsets[b + 1]), M))):
            t = int(starts[b]) + r - lo
            if t < 0 or t >= table.shape[1] * page:
                continue
            p = int(table[b, t // page])
            if p < 0 or p >= n:
                continue
            i = t % 32
            for h in range(H):
                u = units[p, h, t % page // 32]
                u[i * D // 2:(i + 1) * D // 2] = (kc[r, h, 0::2] | kc[r, h, 1::2] << 4).to(torch.uint8)
                words = u[16 * D:32 * D].view(4, D, 4)[i // 8, :, i % 8 // 2]
                shift = 4 * (i % 2)
                words.copy_((words & (0xf0 >> shift)) | (vc[r, h] << shift).to(torch.uint8))
                u[32 * D:32 * D + 64].view(torch.bfloat16)[i] = ks[r, h]
                u[32 * D + 64:].view(torch.bfloat16)[i] = vs[r, h]


def tokens(pages, page, H, D, row, length):
    """Rotated keys and values [H, length, D] of one sequence (its row of the table, on the pages'
    device) and which tokens a page holds."""
    n = pages.shape[0]
    cols = (length + page - 1) // page
    p = row[:cols].long()
    held = (p >= 0) & (p < n)
    u = pages.view(n, H, page // 32, unit_bytes(D))[p.clamp(0, n - 1)].transpose(0, 1).reshape(H, -1, unit_bytes(D))
    k = u[..., :16 * D].reshape(H, -1, D // 2)
    k = torch.stack((k & 15, k >> 4), -1).reshape(H, -1, D).double() - 8
    v = u[..., 16 * D:32 * D].reshape(H, -1, D, 4)
    v = torch.stack((v & 15, v >> 4), -1).reshape(H, -1, D, 8).transpose(2, 3).reshape(H, -1, D).double() - 8
    s = u[..., 32 * D:].contiguous().view(torch.bfloat16).double()
    ks, vs = s[..., :32].reshape(H, -1), s[..., 32:].reshape(H, -1)
    return ((k * ks[..., None])[:, :length], (v * vs[..., None])[:, :length],
            held.repeat_interleave(page)[:length] if cols else torch.zeros(0, dtype=torch.bool, device=pages.device))


def attention(q, pages, page, H, table, starts, offsets, scale, causal=True, window=0):
    """(the attention, its tolerance) in 64 bits; rows of no sequence are NaN in the first.

    Tolerance of a row: half a step of the output's type, and before it
    - the rotated query rounded to fp16, 2^-12 of each value (2^-25 of its largest for one that fp16
      holds as a subnormal, below 2^-24 2^4), and D fp32 sums: a score off by
      eta = (2^-12 + D 2^-23) sum |q_d k_d| scale + 2^-20 max|q| sum |k_d| scale, so a weight by exp(2 eta);
    - weights and their exponents, 2^-12 and a few fp32 steps of the exponent's own size; n fp32 sums.
    Errors of the rotated output are then mixed by H / sqrt(D)."""
    M, Hq, D = q.shape
    G = Hq // H
    out = torch.full((M, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    half = torch.finfo(q.dtype).eps / 2
    for b in range(table.shape[0]):
        lo = min(max(int(offsets[b]), 0), M)
        n = max(lo, min(int(offsets[b + 1]), M)) - lo
        end = min(max(int(starts[b]) + n, 0), table.shape[1] * page)
        out[lo:lo + n] = 0
        if n == 0 or end == 0:
            continue
        k, v, held = tokens(pages, page, H, D, table[b], end)
        qr = butterfly(q[lo:lo + n].double()) / math.sqrt(D)
        pos = int(starts[b]) + torch.arange(n, device=q.device)[:, None]
        key = torch.arange(end, device=q.device)[None, :]
        seen = held[None, :] & (key <= pos if causal else key >= 0)
        if window:
            seen = seen & (key > pos - window)
        for h in range(Hq):
            kk, vv = k[h // G], v[h // G]
            kk = torch.where(seen.any(0)[:, None], kk, 0.0)
            vv = torch.where(seen.any(0)[:, None], vv, 0.0)
            x = qr[:, h]
            t = (x @ kk.t()) * scale
            eta = ((2 ** -12 + D * 2.0 ** -23) * (x.abs() @ kk.abs().t())
                   + 2.0 ** -20 * x.abs().amax(1, keepdim=True) * kk.abs().sum(1)[None]) * abs(scale)
            t = torch.where(seen, t, -math.inf)
            top = torch.where(seen.any(1, keepdim=True), t.amax(1, keepdim=True), 0.0)
            w = torch.exp(t - top)
            l = w.sum(1, keepdim=True)
            w = torch.where(l > 0, w / l, 0.0)
            rot = w @ torch.where(seen.any(0)[:, None], vv, 0.0)
            out[lo:lo + n, h] = butterfly(rot) / math.sqrt(D)
            spread = torch.where(seen, eta + 8 * 2.0 ** -24 * (t - top).abs().nan_to_num(0.0, 0.0, 0.0).clamp(max=200.0), 0.0)
            rho = 2 * spread.amax(1, keepdim=True) + 2 ** -11 + end * 2.0 ** -23
            rough = (torch.exp(rho) - 1) * (w @ vv.abs())
            tol[lo:lo + n, h] = rough.sum(1, keepdim=True) / math.sqrt(D)
    return out, tol * (1 + half) + half * out.abs().nan_to_num() + 2.0 ** -25


def rope(x, positions, freqs, scale, layout, inverse=False):
    """(the turned heads, the magnitudes that were added up) in 64 bits."""
    rot = 2 * freqs.shape[0]
    phi = positions.double()[:, None] * freqs.double() * (-1 if inverse else 1)
    c, s = torch.cos(phi)[:, None] * scale, torch.sin(phi)[:, None] * scale
    y, mag = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    ia = torch.arange(rot // 2, device=x.device) * (1 if layout == "half" else 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    a, b = x[..., ia].double(), x[..., ib].double()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * abs(scale)
    return y, mag
