"""convrot_cache_attention: attention over the paged 4-bit cache, against its formula in 64 bits
(tests/_cache.py, with the tolerance and where it comes from)."""
import ctypes
import math

import pytest
import torch

from tests import _cache as ref
from tests.test_kv_cache import CACHE_REFUSALS, cache

OK, EINVAL, EUNSUPPORTED, EALIGN, EWORKSPACE = 0, -1, -2, -3, -4
A = 0x10000          # a fake, 16-byte aligned device address (never dereferenced)
DEV = "cuda:0"


@pytest.fixture(scope="module")
def B():
    import os
    from w8a8_rotated_int8_convrot_amd import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    binding.lib()
    return binding


# ---------------------------------------------------------------- refusals (no GPU, no launch)

def test_refusals(B):
    def go(c, q=A, heads=8, stride=1024, io=1, M=3, scale=0.1, causal=1, window=0, out=A + 65536, ws=A, ws_bytes=1 << 30):
        return B.lib().convrot_cache_attention(ctypes.byref(c) if c is not None else None, q, heads, stride, io, M, scale,
                                               causal, window, out, ws, ws_bytes, None)
    for kw, status in CACHE_REFUSALS:
        assert go(cache(B, **kw)) == status, kw
        assert b"convrot_cache_attention" in B.lib().convrot_last_error()
    for kw, status in [
            (dict(io=0), EUNSUPPORTED), (dict(M=-1), EINVAL), (dict(M=1 << 28), EINVAL), (dict(heads=0), EINVAL),
            (dict(heads=7), EINVAL), (dict(heads=-8), EINVAL), (dict(stride=1016), EINVAL), (dict(stride=1028), EINVAL),
            (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL), (dict(window=-1), EINVAL),
            (dict(window=1 << 31), EINVAL), (dict(window=5, causal=0), EINVAL), (dict(q=None), EINVAL), (dict(out=None), EINVAL),
            (dict(q=A + 8), EALIGN), (dict(out=A + 4), EALIGN), (dict(ws=A + 8), EALIGN)]:
        assert go(cache(B), **kw) == status, kw
    assert go(None) == EINVAL
    long = cache(B, max_pages=1000, table_stride=1000)
    need = B.convrot_cache_attention_workspace(3, 8, 2, 128, 2, 64000)
    assert need > 0
    assert go(long, ws=None, ws_bytes=0) == EWORKSPACE and go(long, ws_bytes=need - 1) == EWORKSPACE
    assert go(cache(B, pages=None, table=None, starts=None, offsets=None), M=0, q=None, out=None, ws=None) == OK


def test_workspace_sizes(B):
    f = B.convrot_cache_attention_workspace
    assert f(1, 1, 1, 64, 1, 32) == 0
    for bad in ((0, 8, 2, 128, 1, 64), (1, 7, 2, 128, 1, 64), (1, 8, 0, 128, 1, 64), (1, 8, 2, 100, 1, 64), (1, 8, 2, 128, 0, 64),
                (1, 8, 2, 128, 1, 0), (1, 8, 2, 128, 1, (1 << 30) + 1), (1 << 29, 8, 2, 128, 1, 64), (1, -8, 2, 128, 1, 64)):
        assert f(*bad) == 0
    # parts cost their sums and no more than 64 of them
    for args in ((1, 32, 8, 128, 1, 1 << 20), (64, 32, 8, 128, 64, 8192), (100, 8, 8, 64, 3, 1 << 16)):
        assert f(*args) <= 64 * args[0] * args[1] * (args[3] + 2) * 4
    # a long prompt's keys and values as 16-bit operands, 8 GiB of them at most
    assert 4096 * 8 * 128 * 4 <= f(4096, 32, 8, 128, 1, 4096) <= 1.02 * 4096 * 8 * 128 * 4 + (1 << 20)
    assert f(4096, 32, 8, 128, 1, 1 << 24) <= 64 * 4096 * 32 * 130 * 4


# ---------------------------------------------------------------- inputs

def filled(seed, lens, H, D, page, spare=2, W=None, scales=(0.25, 0.55)):
    """A cache whose tokens hold codes and scales of ordinary rows, and 0xff everywhere else: unread
    places hold NaN scales."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ends = [max(0, s + n) for s, n in lens]
    W = W or max(1, max((e + page - 1) // page for e in ends))
    n = sum((e + page - 1) // page for e in ends) + spare
    order = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), W), -1, dtype=torch.int32, device=DEV)
    pages = torch.full((n, ref.page_bytes(page, H, D)), 255, dtype=torch.uint8, device=DEV)
    units = pages.view(n, H, page // 32, ref.unit_bytes(D))
    at = 0
    for b, e in enumerate(ends):
        cols = (e + page - 1) // page
        ids = order[at:at + cols]
        at += cols
        table[b, :cols] = ids
        u = torch.full((cols, H, page // 32, ref.unit_bytes(D)), 255, dtype=torch.uint8, device=DEV)
        c = (2.6 * torch.randn(cols, H, page // 32, 64 * D, generator=g, device=DEV)).round().clamp(-7, 7).add(8).to(torch.uint8)
        u[..., :32 * D] = c[..., 0::2] | (c[..., 1::2] << 4)
        s = scales[0] + (scales[1] - scales[0]) * torch.rand(cols, H, page // 32, 2, 32, generator=g, device=DEV)
        token = (torch.arange(cols, device=DEV)[:, None, None] * page + torch.arange(page, device=DEV).view(1, -1, 32))
        s = torch.where((token < e)[:, None, :, None, :], s, math.nan).to(torch.bfloat16)
        u[..., 32 * D:] = s.reshape(cols, H, page // 32, 64).view(torch.uint8)
        units[ids.long()] = u
    first = 1
    offsets = torch.tensor([first] + [first + sum(m for _, m in lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device=DEV)
    starts = torch.tensor([s for s, _ in lens], dtype=torch.int32, device=DEV)
    return g, pages, table, starts, offsets


def wide_table(lens, G, page):
    """Columns with which a sequence alone is long enough for operands of its own."""
    rows = lens[0][1] * G
    return 2 ** 23 // rows // page + 2 if len(lens) == 1 and rows > 896 else None


def queries(g, offsets, Hq, D, dt, size=2.0):
    """A part of a wider row, as the projection gives it; two rows behind the last sequence."""
    M = int(offsets[-1]) + 2
    return (size * torch.randn(M, Hq + 3, D, generator=g, device=DEV)).to(dt)[:, :Hq]


def check(B, q, pages, table, starts, offsets, H, page, scale=None, causal=True, window=0):
    D = q.shape[2]
    out = torch.full(q.shape, 55.0, dtype=q.dtype, device=DEV)
    got = B.convrot_cache_attention(q, pages, table, starts, offsets, H, page, scale=scale, causal=causal, window=window, out=out)
    want, tol = ref.attention(q, pages, page, H, table, starts, offsets, D ** -0.5 if scale is None else scale, causal, window)
    lo, hi = int(offsets[0].clamp(min=0)), int(offsets[-1])
    assert (got[:lo] == 55).all() and (got[hi:] == 55).all(), "rows of no sequence"
    bad = ~((got[lo:hi].double() - want[lo:hi]).abs() <= tol[lo:hi])
    assert not bad.any(), (int(bad.sum()), (got[lo:hi].double() - want[lo:hi]).abs().max(), bad.nonzero()[:3].tolist())
    # the bound adds all errors up; in the mean they are far below it
    err = (got[lo:hi].double() - want[lo:hi]).norm()
    assert err <= (torch.finfo(q.dtype).eps / 2 + 2 ** -9) * want[lo:hi].norm() + 1e-7, err / want[lo:hi].norm()
    return got


# ---------------------------------------------------------------- against the formula

FEW = [
    # sequences (tokens before, new), query heads a key head, key heads, D, page
    ([(0, 1)], 1, 1, 64, 32), ([(0, 1)], 4, 2, 128, 32), ([(31, 1), (32, 1), (30, 1), (63, 1), (64, 1)], 4, 2, 128, 32),
    ([(100, 1), (0, 1), (777, 1), (1, 0), (500, 1)], 7, 3, 128, 64), ([(1000, 1)], 8, 1, 256, 256),
    ([(200, 5), (0, 5), (33, 2)], 2, 2, 256, 32), ([(127, 3), (128, 2), (95, 1)], 5, 1, 64, 128),
    ([(50, 1)], 40, 1, 128, 64), ([(300, 4), (10, 4)], 8, 2, 64, 64), ([(i * 13 % 200, 1) for i in range(130)], 4, 1, 128, 32),
]


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,G,H,D,page", FEW)
def test_few_tokens(B, lens, G, H, D, page, io):
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    g, *c = filled(len(lens) + D, lens, H, D, page)
    q = queries(g, c[3], G * H, D, dt)
    check(B, q, *c, H, page)
    check(B, q, *c, H, page, window=33)
    check(B, q, *c, H, page, causal=False, scale=-0.2)


MANY = [
    ([(0, 40)], 4, 1, 128, 64), ([(0, 300)], 1, 2, 64, 32), ([(5, 130), (70, 1), (0, 65), (9, 0), (300, 90)], 4, 2, 128, 32),
    ([(0, 257)], 2, 1, 256, 256), ([(1000, 77), (31, 64)], 3, 2, 128, 128), ([(0, 70), (400, 100)], 8, 1, 64, 64),
    ([(17, 150), (3, 33)], 1, 3, 256, 64),
    # around 512 rows a key head
    ([(0, 700)], 1, 2, 64, 32), ([(100, 300), (50, 1), (0, 200), (7, 2)], 4, 1, 128, 64), ([(1000, 600), (31, 64), (3, 530)], 1, 2, 128, 128),
    ([(17, 650)], 1, 1, 256, 64), ([(2000, 90)], 8, 1, 64, 64), ([(3, 140), (300, 257), (0, 0), (64, 129)], 4, 2, 256, 256),
    ([(0, 513)], 1, 1, 128, 32), ([(1, 33), (5, 1025)], 2, 1, 64, 128),
    # of several more than 2048, and more than 896 alone in a wide table: their keys and values made operands first
    ([(0, 897)], 1, 1, 128, 32), ([(0, 910)], 1, 2, 64, 32), ([(17, 1000)], 1, 1, 256, 64), ([(3, 240), (300, 300), (0, 0), (64, 225)], 4, 2, 256, 256),
    ([(1000, 950), (31, 64), (3, 930)], 1, 2, 128, 128), ([(2000, 130)], 8, 1, 64, 64), ([(100, 1), (9, 2100), (0, 1), (50, 3)], 1, 1, 128, 64),
    ([(100, 300), (50, 1), (0, 200), (7, 250)], 4, 1, 128, 64), ([(100, 300), (50, 1), (0, 3), (7, 25)], 8, 1, 128, 64),
    ([(40, 33), (50, 1), (500, 1100), (0, 0), (31, 2)], 2, 2, 64, 128), ([(0, 300), (20, 350)], 3, 30, 64, 32),
]


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,G,H,D,page", MANY)
def test_many_tokens(B, lens, G, H, D, page, io):
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    g, *c = filled(len(lens) + D + 1, lens, H, D, page, W=wide_table(lens, G, page))
    q = queries(g, c[3], G * H, D, dt)
    check(B, q, *c, H, page)
    check(B, q, *c, H, page, window=1)
    check(B, q, *c, H, page, window=50)
    check(B, q, *c, H, page, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,G,H,D,page,window", [
    ([(20000, 1)], 8, 2, 128, 64, 0), ([(9000, 1), (12, 1), (4000, 1)], 4, 2, 64, 256, 0), ([(7000, 3), (6000, 2)], 4, 1, 256, 32, 3000),
    ([(8000, 60), (100, 70)], 4, 1, 128, 128, 0), ([(8000, 160)], 4, 1, 128, 128, 0), ([(6000, 600)], 1, 1, 64, 128, 700), ([(9000, 1000)], 1, 1, 128, 64, 700), ([(5000, 500)], 2, 1, 256, 128, 0), ([(5000, 130)], 2, 1, 64, 64, 2000), ([(30000, 1), (200, 90), (3, 2)], 4, 1, 128, 64, 0)])
def test_long_sequences_in_parts(B, lens, G, H, D, page, window):
    g, *c = filled(sum(s for s, _ in lens), lens, H, D, page)
    q = queries(g, c[3], G * H, D, torch.float16)
    M = q.shape[0]
    assert B.convrot_cache_attention_workspace(M, G * H, H, D, len(lens), c[1].shape[1] * page) > 0
    first = check(B, q, *c, H, page, window=window)
    # the same bytes again, and from a workspace that holds what it happens to
    assert torch.equal(check(B, q, *c, H, page, window=window), first)
    ws = torch.full((B.convrot_cache_attention_workspace(M, G * H, H, D, len(lens), c[1].shape[1] * page),), 255,
                    dtype=torch.uint8, device=DEV)
    again = B.convrot_cache_attention(q, *c, H, page, window=window, workspace=ws, out=torch.full_like(first, 55.0))
    assert torch.equal(again, first)


@pytest.mark.gpu
def test_rows_without_a_token_are_zero(B):
    H, D, page = 2, 128, 32
    lens = [(-5, 8), (-40, 30), (0, 1), (-33, 40)]
    g, *c = filled(1, lens, H, D, page)
    q = queries(g, c[3], 8, D, torch.bfloat16)
    got = check(B, q, *c, H, page)
    lo = int(c[3][0])
    assert (got[lo:lo + 5] == 0).all() and (got[lo + 5:lo + 8] != 0).any()
    assert (got[lo + 8:lo + 38] == 0).all()
    check(B, q, *c, H, page, causal=False)
    check(B, q, *c, H, page, window=2)


@pytest.mark.gpu
def test_tokens_without_a_page_are_left_out(B):
    H, D, page = 2, 64, 32
    lens = [(200, 3), (100, 40), (60, 1), (95, 1)]
    g, pages, table, starts, offsets = filled(2, lens, H, D, page)
    table[0, 2], table[0, 5], table[1, 0] = -1, pages.shape[0], -2 ** 31
    table[2, :] = 2 ** 31 - 1
    # a table wider than the columns given, and sequences that reach past them
    wide = torch.full((4, 40), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    q = queries(g, offsets, 6, D, torch.float16)
    got = check(B, q, pages, wide[:, :table.shape[1]], starts, offsets, H, page)
    lo = int(offsets[2])
    assert (got[lo] == 0).all()
    check(B, q, pages, wide[:, :3], starts, offsets, H, page)
    check(B, q, pages, wide, starts, offsets, H, page)


@pytest.mark.gpu
@pytest.mark.parametrize("many", [False, True])
def test_what_is_not_finite_stays_with_who_reads_it(B, many):
    H, D, page = 2, 128, 32
    lens = [(64, 260 if many else 5)]
    g, pages, table, starts, offsets = filled(3, lens, H, D, page, W=wide_table(lens, 4, page))
    q = queries(g, offsets, 8, D, torch.bfloat16).clone()
    lo, n = int(offsets[0]), lens[0][1]
    clean = B.convrot_cache_attention(q, pages, table, starts, offsets, H, page)
    # a query row with NaN, one with infinity: their own results only
    bad = q.clone()
    bad[lo + 1, 2, 5], bad[lo + 3, 7, 0] = math.nan, math.inf
    got = B.convrot_cache_attention(bad, pages, table, starts, offsets, H, page)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[lo + 1, 2], hit[lo + 3, 7] = True, True
    assert torch.isnan(got[hit]).all() and torch.equal(got[lo:lo + n][~hit[lo:lo + n]], clean[lo:lo + n][~hit[lo:lo + n]])
    # a key of NaN scale, and a value of one: those who see it, and no others
    for off in (0, 64):
        spoiled = pages.clone()
        t = 64 + 2                                            # the third new token, key head 1
        u = spoiled.view(-1, H, 1, ref.unit_bytes(D))[int(table[0, t // 32]), 1, 0]
        u[32 * D + off:32 * D + off + 64].view(torch.bfloat16)[t % 32] = math.nan
        got = B.convrot_cache_attention(q, spoiled, table, starts, offsets, H, page)
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[lo + 2:lo + n, 4:] = True
        assert torch.isnan(got[lo:lo + n][hit[lo:lo + n]]).all()
        assert torch.equal(got[lo:lo + n][~hit[lo:lo + n]], clean[lo:lo + n][~hit[lo:lo + n]])


@pytest.mark.gpu
@pytest.mark.parametrize("size,scales,scale", [
    (0.0, (0.3, 0.5), None), (1e-30, (0.3, 0.5), 1e28), (3e4, (0.3, 0.5), 3e-6), (1e30, (1e-6, 1e-5), 1e-26),
    (60.0, (0.3, 0.5), None), (2.0, (1e-15, 1e-12), 1e12), (2.0, (1e4, 1e9), 1e-9), (1.0, (0.0, 0.4), None), (2.0, (0.0, 0.0), None)])
def test_sizes_of_values(B, size, scales, scale):
    """Queries, keys and values from very small to very large, scores that pick one token of all."""
    for lens, G in (([(300, 1), (40, 1)], 4), ([(100, 80)], 2), ([(64, 300)], 2), ([(64, 460)], 2)):
        g, *c = filled(7, lens, 1, 128, 64, scales=scales, W=wide_table(lens, G, 64))
        check(B, queries(g, c[3], G, 128, torch.bfloat16, size), *c, 1, 64, scale=scale)


@pytest.mark.gpu
def test_a_row_does_not_see_its_neighbours(B):
    """The same token alone, in a batch of others of its size, and beside rows far larger: the same bytes."""
    H, G, D, page = 2, 4, 128, 64
    lens = [(500, 1), (100, 1), (900, 1), (3, 1)]
    g, pages, table, starts, offsets = filled(5, lens, H, D, page)
    q = queries(g, offsets, H * G, D, torch.float16).clone()
    got = B.convrot_cache_attention(q, pages, table, starts, offsets, H, page)
    lo = int(offsets[0])
    q[lo + 1], q[lo + 2] = 30000.0, 1e-7
    again = B.convrot_cache_attention(q, pages, table, starts, offsets, H, page)
    assert torch.equal(got[lo], again[lo]) and torch.equal(got[lo + 3], again[lo + 3])
    q2 = q.clone()
    q2[lo, 1:] = -20000.0                                     # its own other heads, in the same columns' tile
    other = B.convrot_cache_attention(q2, pages, table, starts, offsets, H, page)
    assert torch.equal(other[lo, 0], again[lo, 0])


@pytest.mark.gpu
def test_the_same_pages_twice(B):
    """Two sequences that share the pages of a beginning, as forks do."""
    H, D, page = 2, 64, 32
    g, pages, table, starts, offsets = filled(6, [(128, 1), (128, 1)], H, D, page)
    table[1, :4] = table[0, :4]
    q = queries(g, offsets, 8, D, torch.float16)
    check(B, q, pages, table, starts, offsets, H, page)


@pytest.mark.gpu
@pytest.mark.parametrize("D,io", [(64, "bf16"), (128, "bf16"), (128, "fp16"), (256, "fp16")])
def test_long_prompts_with_gaps(B, D, io):
    """Prompts long enough for operands of their own: tokens before the first, pages that no cache
    has, sequences past their table, one of them alone and beside others."""
    H, G, page = 2, 4, 64
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    for lens in ([(-40, 300)], [(200, 600), (10, 1), (-500, 300), (3, 1), (0, 2), (105, 1)]):
        g, pages, table, starts, offsets = filled(len(lens) + D, lens, H, D, page, W=wide_table(lens, G, page))
        table[0, 1], table[-1, 1] = -1, pages.shape[0]
        q = queries(g, offsets, H * G, D, dt)
        for kw in (dict(), dict(window=70), dict(causal=False)):
            check(B, q, pages, table, starts, offsets, H, page, **kw)
        check(B, q, pages, table[:, :3], starts, offsets, H, page)


@pytest.mark.gpu
def test_many_sequences(B):
    """More sequences than a wave has lanes, of none to thousands of rows, with and without a window."""
    lens = [(7 * i, i % 4) for i in range(150)]
    lens[3], lens[66], lens[140] = (5, 2100), (0, 2300), (300, 2049)
    g, *c = filled(21, lens, 1, 64, 32)
    q = queries(g, c[3], 1, 64, torch.bfloat16)
    check(B, q, *c, 1, 32)
    check(B, q, *c, 1, 32, window=45)


@pytest.mark.gpu
def test_offsets_outside_the_rows_of_long_prompts_reach_nothing(B):
    D, page, M = 64, 32, 1000
    for seqs, offs in ((1, ([-5, 2 ** 31 - 1], [3, 3], [900, 2], [-2 ** 31, 990])),
                       (6, ([0, M, 0, M, 0, M, M], [0, 2 ** 31 - 1, -1, M, 7, 8, M - 1], [M, 0, M, 0, M, 0, M], [300, 200, 999, 1000, 2000, 0, 0]))):
        g, pages, table, _, _ = filled(4, [(64, 1000)] * seqs, 1, D, page, W=wide_table([(64, 1000)] * seqs, 4, page))
        q = torch.randn(M, 4, D, device=DEV).half()
        for off in offs:
            for st in (0, 2 ** 31 - 1, -2 ** 31, -70, 1000):
                B.convrot_cache_attention(q, pages, table, torch.full((seqs,), st, dtype=torch.int32, device=DEV),
                                          torch.tensor(off, dtype=torch.int32, device=DEV), 1, page)
                torch.cuda.synchronize()


@pytest.mark.gpu
def test_long_prompts_captured_with_others(B):
    """A long prompt and single tokens in one captured call: starts move between the replays."""
    H, G, D, page = 1, 2, 128, 64
    lens = [(2000, 1), (300, 1200), (64, 1), (0, 3)]
    g, pages, table, starts, offsets = filled(13, lens, H, D, page)
    q = queries(g, offsets, H * G, D, torch.bfloat16).clone()
    out = torch.empty_like(q)
    need = B.convrot_cache_attention_workspace(q.shape[0], H * G, H, D, 4, table.shape[1] * page)
    guarded = torch.full((need + 4096,), 165, dtype=torch.uint8, device=DEV)
    ws = guarded[:need]
    run = lambda: B.convrot_cache_attention(q, pages, table, starts, offsets, H, page, out=out, workspace=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    lo, hi = int(offsets[0]), int(offsets[-1])
    for i in range(3):
        q.normal_()
        starts.copy_(torch.tensor([2000 - i, 300 - 70 * i, 64, 0], dtype=torch.int32))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        want, tol = ref.attention(q, pages, page, H, table, starts, offsets, D ** -0.5, True, 0)
        assert ((out[lo:hi].double() - want[lo:hi]).abs() <= tol[lo:hi]).all()
        assert torch.equal(B.convrot_cache_attention(q, pages, table, starts, offsets, H, page)[lo:hi], out[lo:hi])
    assert (guarded[need:] == 165).all()


@pytest.mark.gpu
def test_pages_past_four_gigabytes(B):
    H, D, page = 16, 256, 256
    g, pages, table, starts, offsets = filled(8, [(300, 1), (20, 40)], H, D, page)
    n = (5 << 30) // pages.shape[1]
    far = torch.full((n, pages.shape[1]), 255, dtype=torch.uint8, device=DEV)
    far[n - pages.shape[0]:] = pages
    table = torch.where(table >= 0, table + (n - pages.shape[0]), table)
    q = queries(g, offsets, H, D, torch.bfloat16)
    check(B, q, far, table, starts, offsets, H, page)


@pytest.mark.gpu
def test_offsets_outside_the_rows_reach_nothing(B):
    H, D, page = 1, 64, 32
    g, pages, table, _, _ = filled(4, [(64, 32)] * 4, H, D, page)
    q = torch.randn(8, 4, D, device=DEV).half()
    for off in ([0, 100, 2 ** 31 - 1, 50, 60], [-5, 3, 3, 8, 8], [8, 6, 4, 2, 0], [-2 ** 31, 2 ** 31 - 1, -1, 9, 8]):
        for st in ([0] * 4, [2 ** 31 - 1, -2 ** 31, 31, -1]):
            B.convrot_cache_attention(q, pages, table, torch.tensor(st, dtype=torch.int32, device=DEV),
                                      torch.tensor(off, dtype=torch.int32, device=DEV), H, page)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_captured_two_graphs_and_two_streams(B):
    H, G, D, page = 2, 4, 128, 64
    lens = [(3000, 1), (900, 1), (64, 1)]
    g, pages, table, starts, offsets = filled(11, lens, H, D, page)
    q = queries(g, offsets, H * G, D, torch.bfloat16).clone()
    q2 = torch.randn_like(q)
    need = B.convrot_cache_attention_workspace(q.shape[0], H * G, H, D, 3, table.shape[1] * page)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    args = (pages, table, starts, offsets, H, page)
    run = lambda x, o: B.convrot_cache_attention(x, *args, out=o, workspace=ws)  # noqa: E731
    o1, o2 = torch.empty_like(q), torch.empty_like(q)
    run(q, o1), run(q2, o2)
    torch.cuda.synchronize()
    graphs = []
    for x, o in ((q, o1), (q2, o2)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(x, o)
        graphs.append(graph)
    lo, hi = int(offsets[0]), int(offsets[-1])
    for i in range(3):
        q.normal_(), q2.normal_()
        starts.copy_(torch.tensor([3000 - 1000 * i, 900, 64 - i], dtype=torch.int32))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for x, o in ((q, o1), (q2, o2)):
            assert torch.equal(B.convrot_cache_attention(x, *args)[lo:hi], o[lo:hi])
    # two streams at once, each with a workspace of its own
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s, x in zip(sides, (q, q2)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([B.convrot_cache_attention(x, *args) for _ in range(5)])
    torch.cuda.synchronize()
    for o, runs in zip((o1, o2), outs):
        assert all(torch.equal(r[lo:hi], o[lo:hi]) for r in runs)


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit(B):
    g, pages, table, starts, offsets = filled(4, [(64, 2)], 2, 64, 32)
    q = queries(g, offsets, 4, 64, torch.float16)
    good = dict(q=q, pages=pages, table=table, starts=starts, offsets=offsets, kv_heads=2, page=32)
    B.convrot_cache_attention(**good)
    for bad in (dict(q=q.cpu()), dict(q=q.float()), dict(q=q[:, :, ::2]), dict(q=q.transpose(0, 1)), dict(kv_heads=4),
                dict(page=64), dict(table=table.long()), dict(starts=starts.long()), dict(offsets=offsets[:1]),
                dict(out=torch.empty_like(q)[:1]), dict(pages=pages.cpu())):
        with pytest.raises(ValueError):
            B.convrot_cache_attention(**{**good, **bad})
    for bad in (dict(q=q[:, :3]), dict(scale=math.inf), dict(window=-1), dict(window=3, causal=False)):
        with pytest.raises(B.ConvrotError):
            B.convrot_cache_attention(**{**good, **bad})
