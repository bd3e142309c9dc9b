"""convrot_cache_attention over tokens whose key and value scales are far apart, within a unit of 32
tokens and between units: every row's result is that of the keys with weight in it, whatever
others hold, against the formula in 64 bits."""
import math

import pytest
import torch

from tests import _cache as ref
from tests.test_cache_attention import DEV, B, filled, wide_table  # noqa: F401
from tests.test_cache_attention_scores import shifted, units

pytestmark = pytest.mark.gpu


def attention(q, pages, page, H, table, starts, offsets, window=0, least=2.0 ** -25):
    """(the attention, its tolerance) in 64 bits.  Key j's weight is off by the factor exp(rho_j), with
    rho_j = 2 eta_j + 8 2^-24 |t_j - top| + 2^-11 + n 2^-23 and its score off by
      eta_j = ((2^-12 + D 2^-23) sum |q_d k_d| + 2^-16 max |q| sum |k_d|) / sqrt(D)
    (the rotated query in fp16, or in 15 bits of its row's largest value; D sums; twice, for the sum of
    the weights is off as they are; weights, exponents and n sums in the rest).  A result is then off by
    sum_j w_j (exp(rho_j) - 1) (|v_j| + |result|), mixed by H / sqrt(D), half a step of its type, and
    `least`, half a step of its smallest values (fp16 2^-25, bf16 2^-134)."""
    M, Hq, D = q.shape
    out = torch.zeros(M, Hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for b in range(table.shape[0]):
        lo, n = int(offsets[b]), int(offsets[b + 1]) - int(offsets[b])
        if n == 0:
            continue
        end = int(starts[b]) + n
        k, v, held = ref.tokens(pages, page, H, D, table[b], end)
        qr = ref.butterfly(q[lo:lo + n].double()) / math.sqrt(D)
        pos = int(starts[b]) + torch.arange(n, device=q.device)[:, None]
        key = torch.arange(end, device=q.device)[None, :]
        seen = held[None, :] & (key <= pos) & ((key > pos - window) if window else (key >= 0))
        for h in range(Hq):
            kk, vv, x = k[h * H // Hq], v[h * H // Hq], qr[:, h]
            t = torch.where(seen, x @ kk.t() / math.sqrt(D), -math.inf)
            top = t.amax(1, keepdim=True)
            w = torch.softmax(t, 1)
            none = torch.isnan(vv).any(-1)
            vv = vv.nan_to_num(0.0)
            rot = torch.where((seen & none).any(1, keepdim=True), math.nan, w @ vv)
            eta = ((2 ** -12 + D * 2.0 ** -23) * (x.abs() @ kk.abs().t())
                   + 2.0 ** -16 * x.abs().amax(1, keepdim=True) * kk.abs().sum(1)[None]) / math.sqrt(D)
            rho = 2 * eta + 8 * 2.0 ** -24 * (top - t).clamp(max=200.0) + 2 ** -11 + end * 2.0 ** -23
            off = torch.where(w > 0, w * torch.expm1(rho), 0.0)
            rough = off @ vv.abs() + off.sum(1, keepdim=True) * rot.abs()
            out[lo:lo + n, h] = ref.butterfly(rot) / math.sqrt(D)
            tol[lo:lo + n, h] = rough.sum(1, keepdim=True) / math.sqrt(D)
    half = torch.finfo(q.dtype).eps / 2
    return out, tol * (1 + half) + half * out.abs() + least


# sequences (tokens before, new), query heads a key head, key heads, D, page
BY_OPERANDS = [([(200, 600)], 4, 2, 128, 32), ([(70, 950)], 1, 1, 64, 64), ([(30, 260)], 4, 1, 128, 128)]

KINDS = ["a loud unit", "a loud token", "loud tokens at the end", "values of all sizes", "values of 0 seen first", "keys of all sizes",
         "a far key", "tiny values", "a value that is none"]
# two of them have results past fp16's largest value
KINDS = [(k, io) for k in KINDS for io in ("bf16", "fp16") if io == "bf16" or k not in ("values of all sizes", "values of 0 seen first")]


def prepared(kind, lens, G, H, D, page, dt):
    """A cache and queries: `loud` tokens have values 2^30 times the others' and scores 40 below them."""
    shift = 20.0
    base = (0.4, 0.4)
    g, pages, table, starts, offsets = filled(len(lens) + D, lens, H, D, page, W=wide_table(lens, G, page), scales=base)
    q = shifted(g, pages, offsets, H, G * H, D, page, dt, shift)
    for b, (s, n) in enumerate(lens):
        end = s + n
        for t in range(end):
            p = int(table[b, t // page])
            u, i = units(pages, H, D, page)[p, :, t % page // 32], t % 32
            ks, vs = u[:, 32 * D:32 * D + 64].view(torch.bfloat16)[:, i], u[:, 32 * D + 64:].view(torch.bfloat16)[:, i]

            def far(code):                                  # dim 0 of the key: 7 at the others'
                u[:, i * D // 2] = (u[:, i * D // 2] & 0xf0) | (code + 8)
            if kind == "a loud unit" and t // 32 == 1:
                vs.mul_(2.0 ** 30), far(-7)
            elif kind == "a loud token" and t % 96 == 5:
                vs.mul_(2.0 ** 30), far(-7)
            elif kind == "loud tokens at the end" and t >= end - 3:
                vs.mul_(2.0 ** 30), far(-7)
            elif kind == "values of all sizes":
                vs.mul_(2.0 ** (t * 37 % 81 - 40))
            elif kind == "values of 0 seen first":
                vs.mul_(0.0 if t % 8 == 3 and t < 64 else 2.0 ** 50)
                if not (t % 8 == 3 and t < 64):
                    far(-7)                                 # all others 40 below
            elif kind == "keys of all sizes":
                ks.mul_(2.0 ** -(t * 37 % 31))
            elif kind == "a far key" and t % 64 == 9:
                ks.mul_(2.0 ** 20), far(-7)
            elif kind == "tiny values":
                vs.mul_(2.0 ** (-85 if dt == torch.bfloat16 else -3))
            elif kind == "a value that is none" and t == end - 2:
                vs.fill_(math.nan), far(-7)
    return q, pages, table, starts, offsets


def check(B, kind, lens, G, H, D, page, dt):  # noqa: F811
    q, pages, table, starts, offsets = prepared(kind, lens, G, H, D, page, dt)
    lo, hi = int(offsets[0]), int(offsets[-1])
    for window in (0, 70):
        got = B.convrot_cache_attention(q, pages, table, starts, offsets, H, page, window=window)[lo:hi]
        want, tol = (x[lo:hi] for x in attention(q, pages, page, H, table, starts, offsets, window,
                                                 2.0 ** (-134 if dt == torch.bfloat16 else -25)))
        none = torch.isnan(want)
        assert torch.equal(torch.isnan(got), none)
        bad = ~((got.double() - want).abs() <= tol) & ~none
        assert not bad.any().item(), (window, int(bad.sum()), (got.double() - want)[~none].abs().max().item(), bad.nonzero()[:3].tolist())
        assert kind == "a value that is none" or not none.any()


@pytest.mark.parametrize("kind,io", KINDS)
@pytest.mark.parametrize("lens,G,H,D,page", BY_OPERANDS)
def test_long_prompts(B, lens, G, H, D, page, kind, io):  # noqa: F811
    check(B, kind, lens, G, H, D, page, torch.bfloat16 if io == "bf16" else torch.float16)


FEW = [([(200, 3), (400, 1)], 4, 2, 128, 32), ([(150, 20), (1, 33)], 1, 3, 64, 64), ([(300, 1)], 8, 1, 256, 32),
       ([(100, 40), (64, 1)], 1, 2, 256, 64), ([(260, 24), (90, 40)], 4, 1, 128, 128),
       ([(40, 33), (50, 1), (500, 1100)], 2, 2, 64, 32)]          # both kernels


@pytest.mark.parametrize("kind,io", KINDS)
@pytest.mark.parametrize("lens,G,H,D,page", FEW)
def test_few_rows(B, lens, G, H, D, page, kind, io):  # noqa: F811
    check(B, kind, lens, G, H, D, page, torch.bfloat16 if io == "bf16" else torch.float16)
