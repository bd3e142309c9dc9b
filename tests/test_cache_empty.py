"""Calls on the 4-bit cache with nothing to do: no rows, no sequences, no columns, no pages."""
import ctypes

import pytest
import torch

from tests.test_kv_cache import A, DEV, EINVAL, OK, B, cache  # noqa: F401


def calls(B, c, M):  # noqa: F811
    r, lib = ctypes.byref(c), B.lib()
    return (lib.convrot_cache_append(r, A, 256, A, 256, 1, M, None), lib.convrot_cache_read(r, A, 256, A, 256, 1, M, None),
            lib.convrot_cache_attention(r, A, 8, 1024, 1, M, 0.1, 1, 0, A + 65536, A, 1 << 30, None))


NONE = [dict(n_seqs=0), dict(max_pages=0, table_stride=0), dict(max_pages=0), dict(n_pages=0),
        dict(n_seqs=0, max_pages=0, table_stride=0, n_pages=0, pages=None, table=None, starts=None, offsets=None)]


@pytest.mark.parametrize("kw", NONE)
def test_no_rows_and_nothing_else(B, kw):  # noqa: F811
    assert calls(B, cache(B, **kw), 0) == (OK,) * 3 and B.lib().convrot_last_error() == b""
    assert calls(B, cache(B, **kw), 3) == (EINVAL,) * 3


@pytest.mark.parametrize("kw", [dict(n_seqs=-1), dict(max_pages=-1), dict(n_pages=-1), dict(n_seqs=(1 << 20) + 1), dict(table_stride=-1)])
def test_bad_sizes_are_refused_without_rows_too(B, kw):  # noqa: F811
    assert calls(B, cache(B, **kw), 0) == (EINVAL,) * 3


@pytest.mark.gpu
def test_an_empty_batch(B):  # noqa: F811
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    for n, W in ((0, 0), (4, 0), (4, 3)):
        pages = torch.full((n, B.convrot_cache_page_bytes(32, 2, 64)), 7, dtype=torch.uint8, device=DEV)
        args = (pages, i32(0, W), i32(0), i32(1))
        x = torch.zeros(0, 2, 64, dtype=torch.float16, device=DEV)
        B.convrot_cache_append(*args, x, x, 32)
        k, v = B.convrot_cache_read(*args, 0, 2, 64, 32)
        q = torch.zeros(0, 8, 64, dtype=torch.float16, device=DEV)
        assert k.shape == v.shape == (0, 2, 64) and B.convrot_cache_attention(q, *args, 2, 32).shape == (0, 8, 64)
        torch.cuda.synchronize()
        assert (pages == 7).all()
