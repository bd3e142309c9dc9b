"""How accurate convrot_cache_attention is, as the norm of its error over the norm of what rounding the
exact result to the output's type costs by itself.

Of normal queries of size 2 and keys of codes of 2.6 and scales of 0.4 (scores of 2.1), the kernels' own
errors, relative and in the mean (a value rounded to p bits is off by 2^-p / 12^1/2 to twice that):
- few rows: the query in 15 bits of its row's largest value, 3 of its mean size: steps of 6 / 32512, scores
  and so weights off by 6 / 32512 / 12^1/2 1.05 = 5.6e-5; for bf16 rows the weight in one fp16, 2.8e-4 at most;
- long prompts, bf16: the query in one fp16, 2.8e-4 of scores of 2.1, at most 5.9e-4 (2.1e-4 where its
  mantissas are spread as a normal value's are: 4.4e-4), and the weight, 2.1e-4: 4.9e-4 together;
- long prompts, fp16, 64 wide: two terms of each, below 1e-6 (128 and 256 wide fp16 heads, and 256 wide
  ones of bf16, have the kernel for few rows only).
Rounding the result costs at least 2^-11 / 12^1/2 = 1.4e-4 in fp16, 2^-8 / 12^1/2 = 1.13e-3 in bf16.
So the ratios are at most (1 + (5.6 / 14)^2)^1/2 = 1.08, (1 + (2.9 / 11.3)^2)^1/2 = 1.04,
(1 + (4.9 / 11.3)^2)^1/2 = 1.09 and 1.001.  A weight in one fp16 where two are due gives 1.4."""
import math

import pytest
import torch

from tests import _cache as ref
from tests.test_cache_attention import DEV, B, filled, queries, wide_table  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,io,many,most", [
    (64, "fp16", False, 1.08), (128, "fp16", False, 1.08), (256, "fp16", False, 1.08), (64, "bf16", False, 1.04),
    (128, "bf16", False, 1.04), (256, "bf16", False, 1.04), (64, "bf16", True, 1.09), (128, "bf16", True, 1.09),
    (256, "bf16", True, 1.04), (64, "fp16", True, 1.002), (128, "fp16", True, 1.08), (256, "fp16", True, 1.08)])
def test_error_beside_the_roundings(B, D, io, many, most):  # noqa: F811
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    H, G, page = 2, 4, 64
    lens = [(700, 300)] if many else [(900 + i, 1 + i % 3) for i in range(16)]
    g, pages, table, starts, offsets = filled(D + many, lens, H, D, page, W=wide_table(lens, G, page), scales=(0.3, 0.5))
    q = queries(g, offsets, G * H, D, dt)
    lo, hi = int(offsets[0]), int(offsets[-1])
    got = B.convrot_cache_attention(q, pages, table, starts, offsets, H, page)[lo:hi].double()
    want = ref.attention(q, pages, page, H, table, starts, offsets, 1 / math.sqrt(D))[0][lo:hi]
    ratio = ((got - want).norm() / (want.to(dt).double() - want).norm()).item()
    print("%s %d %s: %.4f" % (io, D, "many" if many else "few", ratio))
    assert ratio <= most
