"""convrot_cache_append and convrot_cache_read of rows near the type's largest values: what is read
back is finite wherever the formula's result is.  Tolerance: half a step of the type and, for
D = 128, of the fp32 product before it."""
import math

import pytest
import torch

from tests import _cache as ref
from tests.test_kv_cache import DEV, B  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_rows_come_back(B, D, io):  # noqa: F811
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    top = 3e37 if io == "bf16" else 6e4
    g = torch.Generator().manual_seed(D)
    x = torch.zeros(12, 1, D, dtype=torch.float64)
    x[0] = top                                              # one rotated value of sqrt(D) times that
    x[1] = top * (1 - 2 * (torch.arange(D) % 2))
    x[2, 0, 5] = top                                        # D equal ones
    x[3, 0, 0], x[3, 0, 1] = top, -top
    for i, size in enumerate((2.0 ** -3, 2.0 ** -6, 2.0 ** -20, 2.0 ** -60 if io == "bf16" else 2.0 ** -14)):
        x[4 + 2 * i:6 + 2 * i] = top * size * torch.randn(2, 1, D, generator=g, dtype=torch.float64).clamp(-4, 4) / 4
    x = x.to(dt)
    pages = torch.zeros(1, ref.page_bytes(32, 1, D), dtype=torch.uint8)
    table, starts = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    offsets = torch.tensor([0, 12], dtype=torch.int32)
    dev = [t.to(DEV) for t in (pages, table, starts, offsets, x)]
    B.convrot_cache_append(*dev[:4], dev[4], dev[4], 32)
    ref.write(pages, 32, 1, D, table, starts, offsets, x, x)
    assert torch.equal(dev[0].cpu(), pages)
    c, s = ref.encode(x)
    assert torch.isfinite(s.double()).all()
    want = ref.butterfly((c.double() - 8) * s.double()[..., None]) / math.sqrt(D)
    for got in B.convrot_cache_read(*dev[:4], 12, 1, D, 32, dtype=dt):
        got = got.cpu().double()
        fits = want.abs() <= torch.finfo(dt).max            # a little more may come back than went in
        assert fits[:2].all() and torch.isfinite(got[fits]).all()
        tol = torch.finfo(dt).eps / 2 * (1 + 2 ** -10) * want.abs() + (2.0 ** -25 if io == "fp16" else 2.0 ** -134)
        assert ((got - want).abs() <= tol)[fits].all()
