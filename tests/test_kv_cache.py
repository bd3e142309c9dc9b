"""convrot_cache_append, convrot_cache_read and convrot_cache_copy: the paged 4-bit cache.

Codes and scales are taken in 64 bits, so every byte of the pages is compared with what the
formulas give in 64 bits, the bytes no token writes among them.  What is read back is within half
a step of its type (and of the fp32 product before it, D = 128)."""
import ctypes
import math

import pytest
import torch

from tests import _cache as ref

OK, EINVAL, EUNSUPPORTED, EALIGN = 0, -1, -2, -3
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

def cache(B, **kw):
    a = dict(pages=A, n_pages=5, page=64, head_dim=128, kv_heads=2, table=A, table_stride=3, n_seqs=2, max_pages=3, starts=A,
             offsets=A)
    a.update(kw)
    return B.Cache(**a)


CACHE_REFUSALS = [
    (dict(page=16), EUNSUPPORTED), (dict(page=512), EUNSUPPORTED), (dict(page=96), EUNSUPPORTED), (dict(page=0), EUNSUPPORTED),
    (dict(head_dim=96), EUNSUPPORTED), (dict(head_dim=512), EUNSUPPORTED), (dict(kv_heads=0), EINVAL),
    (dict(kv_heads=1025), EINVAL), (dict(n_pages=0), EINVAL), (dict(n_pages=1 << 31), EINVAL), (dict(n_seqs=0), EINVAL),
    (dict(n_seqs=(1 << 20) + 1), EINVAL), (dict(max_pages=0), EINVAL), (dict(max_pages=(1 << 24) + 1, table_stride=1 << 25), EINVAL),
    (dict(table_stride=2), EINVAL), (dict(pages=None), EINVAL), (dict(table=None), EINVAL), (dict(starts=None), EINVAL),
    (dict(offsets=None), EINVAL), (dict(pages=A + 8), EALIGN)]
ROW_REFUSALS = [
    (dict(io=0), EUNSUPPORTED), (dict(io=5), EUNSUPPORTED), (dict(M=-1), EINVAL), (dict(M=(1 << 30) + 1), EINVAL),
    (dict(ks=248), EINVAL), (dict(vs=260), EINVAL), (dict(k=A + 8), EALIGN), (dict(v=A + 2), EALIGN)]


@pytest.mark.parametrize("call", ["append", "read"])
def test_refusals(B, call):
    fn = getattr(B.lib(), f"convrot_cache_{call}")

    def go(c, k=A, ks=256, v=A + 4096, vs=512, io=1, M=3):
        return fn(ctypes.byref(c) if c is not None else None, k, ks, v, vs, io, M, None)
    for kw, status in CACHE_REFUSALS:
        assert go(cache(B, **kw)) == status, kw
        assert f"convrot_cache_{call}".encode() in B.lib().convrot_last_error()
    for kw, status in ROW_REFUSALS:
        assert go(cache(B), **kw) == status, kw
    assert go(None) == EINVAL
    assert go(cache(B), k=None, v=None) == EINVAL
    if call == "append":
        assert go(cache(B), v=None) == EINVAL
    assert go(cache(B, pages=None, table=None, starts=None, offsets=None), k=None, v=None, M=0) == OK
    assert B.lib().convrot_last_error() == b""


def test_page_bytes(B):
    assert ctypes.sizeof(B.Cache) == 80
    assert B.convrot_cache_page_bytes(64, 8, 128) == 8 * 2 * 4224
    for bad in ((48, 8, 128), (64, 0, 128), (64, 8, 100), (64, 1025, 64)):
        assert B.convrot_cache_page_bytes(*bad) == 0


def test_copy_refusals(B):
    def go(pairs, pages=A, layers=2, layer_bytes=16 * 48, n_pages=16, page_bytes=48, n=None):
        src = (ctypes.c_int32 * max(1, len(pairs)))(*[a for a, _ in pairs])
        dst = (ctypes.c_int32 * max(1, len(pairs)))(*[b for _, b in pairs])
        return B.lib().convrot_cache_copy(pages, layers, layer_bytes, n_pages, page_bytes, src, dst,
                                          len(pairs) if n is None else n, None)
    one = [(1, 2)]
    for kw in (dict(layers=0), dict(layers=65536), dict(layer_bytes=16 * 47), dict(layer_bytes=16 * 48 + 8), dict(n_pages=0),
               dict(n_pages=1 << 31), dict(page_bytes=0), dict(page_bytes=40), dict(page_bytes=(1 << 31) + 16), dict(n=-1),
               dict(n=(1 << 20) + 1), dict(pages=None)):
        assert go(one, **kw) == EINVAL, kw
    for pairs in ([(1, 16)], [(-1, 2)], [(16, 2)], [(1, -1)], [(3, 3)], [(1, 2), (3, 2)], [(1, 2), (2, 4)], [(1, 2), (4, 1)]):
        assert go(pairs) == EINVAL, pairs
        assert b"convrot_cache_copy" in B.lib().convrot_last_error()
    assert go(one, pages=A + 8) == EALIGN
    assert go([], pages=None) == OK
    with pytest.raises(ValueError):
        B.convrot_cache_copy(torch.zeros(4, 64, dtype=torch.uint8), [(0, 1)])


# ---------------------------------------------------------------- against the formulas

def batch(seed, lens, H, D, page, dt, spare=3):
    """A cache of random bytes, a table over scattered pages, and rows for it, strided and with
    rows of no sequence on both sides."""
    g = torch.Generator()
    g.manual_seed(seed)
    ends = [max(0, s + n) for s, n in lens]
    W = max(1, max((e + page - 1) // page for e in ends))
    need = len(lens) * W + spare
    table = torch.randperm(need, generator=g)[:len(lens) * W].view(len(lens), W).to(torch.int32)
    pages = torch.randint(0, 256, (need, ref.page_bytes(page, H, D)), generator=g, dtype=torch.uint8)
    first = 2
    offsets = torch.tensor([first] + [first + sum(n for _, n in lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
    M = int(offsets[-1]) + 3
    kv = torch.randn(M, 2, H, D, generator=g)
    kv[:, :, :, :: max(1, D // 3)] *= 9
    kv = kv.to(dt)
    starts = torch.tensor([s for s, _ in lens], dtype=torch.int32)
    return pages, table, starts, offsets, kv


CASES = [
    ([(0, 1)], 1, 128, 32), ([(5, 1), (31, 1), (32, 1), (63, 1), (0, 1)], 2, 64, 32),
    ([(0, 40), (7, 3), (100, 0), (33, 65)], 2, 128, 64), ([(3, 300)], 3, 64, 128), ([(250, 20), (0, 9)], 1, 256, 256),
    ([(-3, 10), (-20, 8), (-8, 9), (1, 2)], 2, 128, 32), ([(13, 2), (14, 2), (15, 2)], 5, 256, 64),
    ([(i * 7, 1 + i % 3) for i in range(70)], 1, 64, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,H,D,page", CASES)
def test_every_byte_and_back(B, lens, H, D, page, io):
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    pages, table, starts, offsets, kv = batch(len(lens) + D + page, lens, H, D, page, dt)
    dev = [t.to(DEV) for t in (pages, table, starts, offsets, kv)]
    k, v = dev[4][:, 0], dev[4][:, 1]
    B.convrot_cache_append(dev[0], dev[1], dev[2], dev[3], k, v, page)
    ref.write(pages, page, H, D, table, starts, offsets, kv[:, 0], kv[:, 1])
    assert torch.equal(dev[0].cpu(), pages)
    # the rows back, between rows of no sequence, in parts of a wider row
    M = kv.shape[0]
    out = torch.full((M, 2, H, D), 77.0, dtype=dt, device=DEV)
    B.convrot_cache_read(dev[0], dev[1], dev[2], dev[3], M, H, D, page, k=out[:, 0], v=out[:, 1])
    alone_k, _ = B.convrot_cache_read(dev[0], dev[1], dev[2], dev[3], M, H, D, page, dtype=dt)
    out = out.cpu()
    want = torch.full((M, 2, H, D), 77.0, dtype=torch.float64)
    for b, (s, n) in enumerate(lens):
        lo = int(offsets[b])
        got_k, got_v, _ = ref.tokens(pages, page, H, D, table[b], max(0, s + n))
        for j, x in ((0, got_k), (1, got_v)):
            x = ref.butterfly(x) / math.sqrt(D)
            for r in range(n):
                want[lo + r, j] = x[:, s + r] if s + r >= 0 else 0.0
    tol = torch.finfo(dt).eps / 2 * (1 + 2 ** -10) * want.abs() + 2.0 ** -25
    assert ((out.double() - want).abs() <= tol).all()
    inside = slice(int(offsets[0]), int(offsets[-1]))
    assert torch.equal(alone_k.cpu()[inside], out[inside, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_at_the_borders(B, D):
    """Rows of zeros, one value, equal values, ties between two codes, the smallest and the
    largest values, and rows with infinities and NaN."""
    for dt in (torch.bfloat16, torch.float16):
        x = torch.zeros(16, 1, D)
        x[1, 0, 3] = 1.0
        x[2, 0, :] = -0.375
        x[3, 0, 0], x[3, 0, 1] = 1.0, 1.0                      # half of the codes 0
        x[4, 0, 0], x[4, 0, 1] = 9.0, 5.0                      # 14 and 4: |c| 7 and 2
        x[5, 0, 0], x[5, 0, 1] = 3.0, 1.0                      # 4 and 2: 7 and 3.5, a tie where s is exact
        x[6] = torch.finfo(dt).tiny
        x[7, 0, 0] = torch.finfo(dt).tiny / 4
        x[8] = torch.finfo(dt).max
        x[9, 0, ::2] = torch.finfo(dt).max
        x[10] = torch.randn(1, D, generator=torch.Generator().manual_seed(1))
        x[10, 0, 7] = math.inf
        x[11, 0, 7] = math.nan
        x[12, 0, 7], x[12, 0, 8] = math.inf, -math.inf
        x[13] = (torch.arange(D) % 8).float()
        x[14, 0, 0], x[14, 0, 1] = 3.5 * 7 + 7, 7 - 3.5 * 7     # (14, 49): c 2 and 7, and a tie beside it
        x[15] = 2.0 ** -9 * (torch.arange(D) % 3).float()
        x = x.to(dt)
        pages = torch.randint(0, 256, (2, ref.page_bytes(32, 1, D)), dtype=torch.uint8)
        table, starts = torch.tensor([[1]], dtype=torch.int32), torch.tensor([4], dtype=torch.int32)
        offsets = torch.tensor([0, 16], dtype=torch.int32)
        dev = [t.to(DEV) for t in (pages, table, starts, offsets, x)]
        B.convrot_cache_append(dev[0], dev[1], dev[2], dev[3], dev[4], dev[4], 32)
        ref.write(pages, 32, 1, D, table, starts, offsets, x, x)
        got = dev[0].cpu()
        # a NaN scale is NaN whatever its bits
        for t in (pages, got):
            s = t.view(torch.bfloat16)
            s[torch.isnan(s)] = math.nan
        codes = 32 * D
        assert torch.equal(got[1, :codes], pages[1, :codes]) and torch.equal(got[0], pages[0])
        assert torch.equal(got[1, codes:].view(torch.bfloat16).nan_to_num(1e30), pages[1, codes:].view(torch.bfloat16).nan_to_num(1e30))
        k, v = B.convrot_cache_read(dev[0], dev[1], dev[2], dev[3], 16, 1, D, 32, dtype=dt)
        assert torch.equal(k.nan_to_num(5.0), v.nan_to_num(5.0))
        bad = torch.isnan(k).all(-1).flatten().cpu()
        assert bad[10] and bad[11] and bad[12] and not bad[:8].any() and not bad[13:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("io,sizes", [("fp16", [2.0 ** e for e in (-22, -18, -14, -7, 0, 7, 13)]),
                                      ("bf16", [2.0 ** e for e in (-130, -126, -122, -118, -60, 60, 100, 120)])])
def test_rows_of_every_size(B, io, sizes):
    """Ordinary rows from subnormal values to the type's largest: bytes as in 64 bits."""
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    for D in (64, 128, 256):
        g = torch.Generator().manual_seed(D)
        x = torch.randn(8 * len(sizes), 2, D, generator=g, dtype=torch.float64)
        x *= torch.tensor(sizes, dtype=torch.float64).repeat(8)[:, None, None]
        x = x.to(dt)
        n = (x.shape[0] + 31) // 32
        pages = torch.zeros(n, ref.page_bytes(32, 2, D), dtype=torch.uint8)
        table, starts = torch.arange(n, dtype=torch.int32)[None], torch.zeros(1, dtype=torch.int32)
        offsets = torch.tensor([0, x.shape[0]], dtype=torch.int32)
        dev = [t.to(DEV) for t in (pages, table, starts, offsets, x)]
        B.convrot_cache_append(dev[0], dev[1], dev[2], dev[3], dev[4], dev[4], 32)
        ref.write(pages, 32, 2, D, table, starts, offsets, x, x)
        assert torch.equal(dev[0].cpu(), pages)


@pytest.mark.gpu
def test_what_no_page_holds_is_not_stored(B):
    H, D, page = 2, 64, 32
    pages, _, starts, offsets, kv = batch(4, [(0, 70), (20, 70), (90, 10)], H, D, page, torch.float16)
    table = torch.tensor([[0, -1, 2], [3, pages.shape[0], 4], [5, 6, 1]], dtype=torch.int32)
    wide = torch.full((3, 8), 2 ** 31 - 1, dtype=torch.int32)
    wide[:, :3] = table
    dev = [t.to(DEV) for t in (pages, wide, starts, offsets, kv)]
    before = pages.clone()
    # tokens 96 and on of the last sequence lie past the three columns given
    B.convrot_cache_append(dev[0], dev[1][:, :3], dev[2], dev[3], dev[4][:, 0], dev[4][:, 1], page)
    ref.write(pages, page, H, D, table, starts, offsets, kv[:, 0], kv[:, 1])
    assert torch.equal(dev[0].cpu(), pages) and not torch.equal(pages, before)
    k, v = B.convrot_cache_read(dev[0], dev[1][:, :3], dev[2], dev[3], kv.shape[0], H, D, page, dtype=torch.float16)
    lo = int(offsets[0])
    assert (k[lo + 32:lo + 64] == 0).all() and (v[lo + 32:lo + 64] == 0).all()
    assert (k[lo + 140 + 6:lo + 150] == 0).all() and (k[lo:lo + 32] != 0).any()


@pytest.mark.gpu
def test_offsets_outside_the_rows_reach_nothing(B):
    H, D, page = 1, 64, 32
    pages = torch.zeros(4, ref.page_bytes(page, H, D), dtype=torch.uint8, device=DEV)
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(4, 1)
    x = torch.randn(8, H, D, device=DEV).half()
    for off in ([0, 100, 2 ** 31 - 1, 50, 60], [-5, 3, 3, 8, 8], [8, 6, 4, 2, 0], [-2 ** 31, 2 ** 31 - 1, -1, 9, 8]):
        for st in ([0] * 4, [2 ** 31 - 1, -2 ** 31, 31, -1]):
            args = (pages, table, torch.tensor(st, dtype=torch.int32, device=DEV), torch.tensor(off, dtype=torch.int32, device=DEV))
            B.convrot_cache_append(*args, x, x, page)
            B.convrot_cache_read(*args, 8, H, D, page, dtype=torch.float16)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_pages_past_four_gigabytes(B):
    H, D, page = 16, 256, 256
    pb = ref.page_bytes(page, H, D)
    n = (5 << 30) // pb
    pages = torch.zeros(n, pb, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[n - 1, 1], [2, n - 2]], dtype=torch.int32, device=DEV)
    starts, offsets = torch.tensor([250, 255], dtype=torch.int32), torch.tensor([0, 12, 15], dtype=torch.int32)
    kv = torch.randn(15, 2, H, D).to(torch.bfloat16)
    B.convrot_cache_append(pages, table, starts.to(DEV), offsets.to(DEV), kv[:, 0].to(DEV), kv[:, 1].to(DEV), page)
    used = [n - 1, 1, 2, n - 2]
    small = torch.zeros(4, pb, dtype=torch.uint8)
    ref.write(small, page, H, D, torch.tensor([[0, 1], [2, 3]]), starts, offsets, kv[:, 0], kv[:, 1])
    assert torch.equal(pages[used].cpu(), small)
    pages[used] = 0
    assert not pages.any()


@pytest.mark.gpu
def test_captured_and_on_another_stream(B):
    H, D, page = 2, 128, 64
    pages, table, starts, offsets, kv = [t.to(DEV) for t in batch(9, [(3, 30), (60, 9)], H, D, page, torch.bfloat16)]
    out = torch.empty_like(kv)
    M = kv.shape[0]
    run = lambda: (B.convrot_cache_append(pages, table, starts, offsets, kv[:, 0], kv[:, 1], page),  # noqa: E731
                   B.convrot_cache_read(pages, table, starts, offsets, M, H, D, page, k=out[:, 0], v=out[:, 1]))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        kv.normal_()
        starts.copy_(torch.tensor([i, 61 + i], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        held, bytes_ = out.clone(), pages.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        side.synchronize()
        assert torch.equal(held[2:-3], out[2:-3]) and torch.equal(bytes_, pages)


@pytest.mark.gpu
@pytest.mark.parametrize("n,layers,pb,pairs", [(9, 1, 16, 3), (40, 3, 4224 * 2, 11), (700, 1, 16416, 300), (6, 2, 67584, 1),
                                               (1100, 2, 48, 520)])
def test_copy(B, n, layers, pb, pairs):
    g = torch.Generator()
    g.manual_seed(n)
    pages = torch.randint(0, 256, (layers, n, pb), generator=g, dtype=torch.uint8)
    order = torch.randperm(n, generator=g).tolist()
    moves = [(order[i % (pairs // 2 + 1)], order[n - 1 - i]) for i in range(pairs)]      # some sources often
    got = pages.to(DEV)
    B.convrot_cache_copy(got if layers > 1 else got[0], moves)
    want = pages.clone()
    for a, b in moves:
        want[:, b] = pages[:, a]
    assert torch.equal(got.cpu(), want)
    B.convrot_cache_copy(got, [])
    with pytest.raises(B.ConvrotError):
        B.convrot_cache_copy(got, [(0, 1), (1, 2)])
    with pytest.raises(ValueError):
        B.convrot_cache_copy(got, [(0, 2 ** 40)])
    assert torch.equal(got.cpu(), want)


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit(B):
    pages, table, starts, offsets, kv = [t.to(DEV) for t in batch(9, [(3, 30)], 2, 64, 32, torch.float16)]
    k, v = kv[:, 0], kv[:, 1]
    good = dict(pages=pages, table=table, starts=starts, offsets=offsets, k=k, v=v, page=32)
    B.convrot_cache_append(**good)
    for bad in (dict(pages=pages[:, :-16].contiguous()), dict(pages=pages[0]), dict(page=64), dict(table=table.long()),
                dict(table=table.t().expand(-1, 2)), dict(starts=starts.repeat(2)), dict(offsets=offsets[:1]), dict(v=v.bfloat16()),
                dict(v=v[:-1]), dict(k=k.cpu(), v=v.cpu()), dict(k=k.float(), v=v.float()), dict(pages=pages.cpu())):
        with pytest.raises(ValueError):
            B.convrot_cache_append(**{**good, **bad})
    with pytest.raises(B.ConvrotError):
        B.convrot_cache_append(**{**good, "page": 48})
    with pytest.raises(ValueError):
        B.convrot_cache_read(pages, table, starts, offsets, 5, 2, 64, 32, k=k[:5], v=v[:4])
