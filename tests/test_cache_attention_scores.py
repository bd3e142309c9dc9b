"""convrot_cache_attention where scores are far from 0 or scales differ from token to token: softmax
does not change under a shift that all scores share, and what holds no key moves nothing.

Against the formula in 64 bits (tests/_cache.py, with the tolerance and where it comes from)."""
import math

import pytest
import torch

from tests import _cache as ref
from tests.test_cache_attention import DEV, B, filled, wide_table  # noqa: F401

pytestmark = pytest.mark.gpu


def check(B, q, pages, table, starts, offsets, H, page, causal=True, window=0):  # noqa: F811
    """Each value within the tolerance of tests/_cache.py.  (No bound on the error's norm: a query whose
    rotated values are X in dim 0 and about 1 elsewhere has 15 bits of X, steps of X / 32512, so scores
    off by D^-1/2 0.4 2.6 D^1/2 X / (32512 12^1/2) = X / 108000 in the mean, for codes of 2.6: at a shift
    of 60 and D = 256, X = 343, weights and results by 3.2e-3.)"""
    D = q.shape[2]
    got = B.convrot_cache_attention(q, pages, table, starts, offsets, H, page, causal=causal, window=window)
    want, tol = ref.attention(q, pages, page, H, table, starts, offsets, D ** -0.5, causal, window)
    lo, hi = int(offsets[0]), int(offsets[-1])
    bad = ~((got[lo:hi].double() - want[lo:hi]).abs() <= tol[lo:hi])
    assert not bad.any().item(), (int(bad.sum()), (got[lo:hi].double() - want[lo:hi]).abs().max().item(), bad.nonzero()[:3].tolist())


def units(pages, H, D, page):
    return pages.view(pages.shape[0], H, page // 32, ref.unit_bytes(D))


def shifted(g, pages, offsets, H, Hq, D, page, dt, shift, scale=0.4):
    """Queries whose scores all lie around ``shift``, for keys of one scale: dim 0 of every rotated key
    becomes the code 7, and dim 0 of the rotated queries what gives the shift with it."""
    first = units(pages, H, D, page)[..., :16 * D].unflatten(-1, (32, D // 2))[..., 0]
    first.copy_((first & 0xf0) | 15)
    M = int(offsets[-1]) + 2
    x = torch.randn(M, Hq, D, generator=g, device=DEV, dtype=torch.float64)
    x[..., 0] = shift * math.sqrt(D) / (7 * scale)
    return (ref.butterfly(x) / math.sqrt(D)).to(dt)


# sequences (tokens before, new), query heads a key head, key heads, D, page: by the kernel for few
# rows, by operands, and both in a call
SHIFTED = [([(200, 3), (500, 1)], 4, 2, 128, 32), ([(200, 600)], 4, 2, 128, 32), ([(70, 950)], 1, 1, 64, 64),
           ([(100, 300), (50, 1), (0, 200), (90, 250)], 4, 2, 128, 32), ([(40, 33), (50, 1), (500, 1100)], 2, 2, 64, 32),
           ([(30, 300)], 2, 1, 256, 64)]


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("shift", [-60.0, -25.0, 60.0])
@pytest.mark.parametrize("lens,G,H,D,page", SHIFTED)
def test_pages_without_a_place_and_keys_of_nothing(B, lens, G, H, D, page, shift, io):  # noqa: F811
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    g, pages, table, starts, offsets = filled(len(lens) + D, lens, H, D, page, W=wide_table(lens, G, page), scales=(0.4, 0.4))
    q = shifted(g, pages, offsets, H, G * H, D, page, dt, shift)
    check(B, q, pages, table, starts, offsets, H, page)
    # the first page, one between and the last of none
    holes = table.clone()
    holes[0, 0], holes[0, 2], holes[-1, 0] = -1, pages.shape[0], -5
    for kw in (dict(), dict(window=40), dict(causal=False)):
        check(B, q, pages, holes, starts, offsets, H, page, **kw)
    # units whose keys are all 0, which rows leave behind with their window
    zero = pages.clone()
    for b, column in ((0, 0), (0, 2), (-1, 0)):
        units(zero, H, D, page)[int(table[b, column]), :, 0, 32 * D:32 * D + 64] = 0
    for kw in (dict(), dict(window=40)):
        check(B, q, zero, table, starts, offsets, H, page, **kw)
