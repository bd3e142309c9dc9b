"""convrot_grouped_linear: the layer grouped by expert.

Codes, int32 products and the one fp32 multiply-add per output are the
layer's, so every row has to equal, byte for byte, convrot_linear_ex on that
token with that expert's weight (itself compared with the CPU oracle
elsewhere).  The same rows are also compared with a plain product in 64 bits.
"""
import pytest
import torch

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


def call(B, x=A, io=1, M=64, K=512, wq=A, ws=A, mode=0, E=4, N=64, g=128, bias=None, off=A, rows=A, P=128, y=A, w=A,
         wb=1 << 20):
    return B.lib().convrot_grouped_linear(x, io, M, K, wq, ws, mode, E, N, g, bias, off, rows, P, y, w, wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=64), EUNSUPPORTED), (dict(K=384, g=256), EINVAL), (dict(K=131072 + 128), EINVAL), (dict(io=0), EUNSUPPORTED),
    (dict(mode=2), EUNSUPPORTED), (dict(N=0), EINVAL), (dict(M=-1), EINVAL), (dict(E=0), EINVAL), (dict(E=65537), EINVAL),
    (dict(P=-1), EINVAL), (dict(P=(1 << 30) + 1), EINVAL), (dict(rows=None), EINVAL), (dict(M=0), EINVAL),
    (dict(P=1 << 30, N=1 << 20), EINVAL), (dict(E=65536, N=1 << 30), EINVAL),
    (dict(x=None), EINVAL), (dict(wq=None), EINVAL), (dict(ws=None), EINVAL), (dict(off=None), EINVAL),
    (dict(y=None), EINVAL), (dict(x=A + 8), EALIGN), (dict(wq=A + 4), EALIGN), (dict(y=A + 2), EALIGN),
    (dict(w=A + 8), EALIGN), (dict(w=None), EWORKSPACE), (dict(wb=64 * 512 + 255), EWORKSPACE),
])
def test_refusals(B, kw, status):
    assert call(B, **kw) == status
    assert b"convrot_grouped_linear" in B.lib().convrot_last_error()


def test_empty_and_workspace(B):
    assert call(B, P=0, x=None, wq=None, y=None, w=None, wb=0) == OK
    assert call(B, P=0, M=0, rows=None, x=None) == OK
    assert B.lib().convrot_last_error() == b""
    assert B.convrot_grouped_workspace(3, 128) == 512 + 12
    assert B.convrot_grouped_workspace(-1, 128) == 0 and B.convrot_grouped_workspace(4, 0) == 0


def test_no_rows_routed(B):
    """An empty tensor of rows has no address."""
    assert call(B, P=0, rows=None) == OK and call(B, P=0, rows=None, x=None, off=None, y=None, w=None, wb=0) == OK


gpu = pytest.mark.gpu


@gpu
def test_no_rows_routed_from_python(B):
    g, dt, wq, s, b = layer(256, 40, 3, "bf16", False, False, 1)
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    y = B.convrot_grouped_linear(stream(g, 5, 256, dt), wq, s, 128, torch.zeros(4, dtype=torch.int32, device=DEV), rows=empty)
    assert y.shape == (0, 40)


def layer(K, N, E, io, row, bias, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    wq = torch.randint(-127, 128, (E, N, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
    s = (0.5 + torch.rand((E, N) if row else (E,), generator=g, device=DEV)) * 2e-4
    b = torch.randn(E, N, generator=g, device=DEV).to(dt) if bias else None
    return g, dt, wq, s, b


def stream(g, M, K, dt):
    x = torch.randn(M, K, generator=g, device=DEV)
    x[:, :: max(1, K // 3)] *= 20.0
    return x.to(dt)


def by_expert(B, x, wq, s, group, offsets, rows, bias):
    """Each expert's rows through convrot_linear_ex."""
    out = torch.zeros(rows.numel(), wq.shape[1], dtype=x.dtype, device=DEV)
    for e in range(wq.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            se = s[e].reshape(-1) if s.dim() == 2 else s[e:e + 1]
            out[a:b] = B.convrot_linear_ex(x[rows[a:b].long()].contiguous(), wq[e], se, group,
                                           bias=None if bias is None else bias[e])
    return out


def route(g, M, P, E, counts=None):
    if counts is None:
        cuts = torch.sort(torch.randint(0, P + 1, (E - 1,), generator=g, device=DEV)).values
        off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), P)])
    else:
        off = torch.cumsum(torch.tensor([0] + list(counts), device=DEV), 0)
    rows = torch.randint(0, M, (P,), generator=g, device=DEV)
    return off.to(torch.int32), rows.to(torch.int32)


# mean rows per expert from under one to some hundred: every tile the call chooses from
@gpu
@pytest.mark.parametrize("io,row,bias", [("bf16", False, True), ("fp16", True, False)])
@pytest.mark.parametrize("M,K,N,E,P,group", [
    (1, 128, 1, 1, 1, 128), (1, 256, 40, 7, 3, 256), (5, 384, 17, 70, 9, 128), (13, 512, 100, 3, 40, 256),
    (16, 2048, 264, 130, 500, 128), (40, 640, 129, 5, 150, 128), (64, 1024, 72, 9, 333, 256), (100, 512, 193, 4, 700, 128),
    (300, 768, 250, 3, 1100, 256), (411, 384, 400, 2, 1201, 128), (37, 256, 96, 1, 37, 128), (1000, 1152, 577, 6, 4001, 128)])
def test_equals_the_layer_expert_by_expert(B, M, K, N, E, P, group, io, row, bias):
    g, dt, wq, s, b = layer(K, N, E, io, row, bias, M + K + N)
    x = stream(g, M, K, dt)
    offsets, rows = route(g, M, P, E)
    got = B.convrot_grouped_linear(x, wq, s, group, offsets, rows=rows, bias=b)
    assert torch.equal(got, by_expert(B, x, wq, s, group, offsets, rows, b))


# 256 x 128 and 256 x 192 tiles: experts with many channels
@gpu
@pytest.mark.parametrize("io,row,bias", [("bf16", True, False), ("fp16", False, True)])
@pytest.mark.parametrize("M,K,N,E,P,group", [
    (70, 128, 4095, 16, 500, 128), (300, 256, 8200, 5, 777, 256), (129, 640, 1024, 33, 4100, 128), (64, 384, 33000, 1, 64, 128),
    (500, 128, 7100, 8, 1024, 128), (411, 384, 2050, 20, 5003, 128), (90, 256, 1030, 32, 9000, 256)])
def test_wide_experts(B, M, K, N, E, P, group, io, row, bias):
    g, dt, wq, s, b = layer(K, N, E, io, row, bias, M + K + N)
    x = stream(g, M, K, dt)
    offsets, rows = route(g, M, P, E)
    got = B.convrot_grouped_linear(x, wq, s, group, offsets, rows=rows, bias=b)
    assert torch.equal(got, by_expert(B, x, wq, s, group, offsets, rows, b))


# 192 x 288 and 384 x 192 tiles: experts of some hundred rows
@gpu
@pytest.mark.parametrize("io,row,bias", [("bf16", True, True), ("fp16", False, False)])
@pytest.mark.parametrize("M,K,N,E,P,group", [
    (300, 256, 380, 64, 21000, 128), (700, 512, 4100, 6, 5000, 256), (800, 128, 1400, 16, 8000, 128),
    (4100, 384, 7601, 9, 4100, 128)])
def test_large_tiles(B, M, K, N, E, P, group, io, row, bias):
    g, dt, wq, s, b = layer(K, N, E, io, row, bias, M + K + N)
    x = stream(g, M, K, dt)
    offsets, rows = route(g, M, P, E)
    rows[:7] = torch.tensor([-1, M, 0, M - 1, 2 ** 31 - 1, -2 ** 31, 5], device=DEV)
    offsets[0], offsets[-1] = 2, P - 3
    offsets = torch.cummax(offsets, 0).values.clamp(max=P - 3).to(torch.int32)
    out = torch.full((P, N), 3.0, dtype=dt, device=DEV)
    B.convrot_grouped_linear(x, wq, s, group, offsets, rows=rows, bias=b, out=out)
    good = (rows >= 0) & (rows < M) & (torch.arange(P, device=DEV) >= 2) & (torch.arange(P, device=DEV) < P - 3)
    want = by_expert(B, x, wq, s, group, offsets, rows.clamp(0, M - 1), b)
    assert (out[~good] == 3).all() and torch.equal(out[good], want[good])


# one to four tokens go through a kernel of their own up to K = 8192
@gpu
@pytest.mark.parametrize("io,row,bias", [("bf16", True, True), ("fp16", False, False)])
@pytest.mark.parametrize("M,K,N,E,P,group", [
    (1, 128, 16, 4, 1, 128), (1, 2048, 1408, 16, 4, 128), (2, 2176, 100, 5, 13, 128), (3, 4096, 264, 130, 40, 256),
    (4, 4352, 37, 3, 77, 256), (4, 8192, 48, 6, 20, 128), (4, 8448, 48, 6, 20, 256), (2, 256, 9, 70, 300, 256)])
def test_few_tokens(B, M, K, N, E, P, group, io, row, bias):
    g, dt, wq, s, b = layer(K, N, E, io, row, bias, M + K + N)
    x = stream(g, M, K, dt)
    offsets, rows = route(g, M, P, E)
    assert torch.equal(B.convrot_grouped_linear(x, wq, s, group, offsets, rows=rows, bias=b),
                       by_expert(B, x, wq, s, group, offsets, rows, b))
    # rows of no expert, of no token, and a token of zeros
    x[M - 1] = 0
    offsets = offsets.clamp(max=max(1, P - 2))
    rows[::3] = torch.where(torch.arange(len(rows[::3]), device=DEV) % 2 == 0, -1, M).to(torch.int32)
    out = torch.full((P, N), 5.0, dtype=dt, device=DEV)
    B.convrot_grouped_linear(x, wq, s, group, offsets, rows=rows, bias=b, out=out)
    good = (rows >= 0) & (rows < M) & (torch.arange(P, device=DEV) < offsets[-1])
    want = by_expert(B, x, wq, s, group, offsets, rows.clamp(0, M - 1), b)
    assert (out[~good] == 5).all() and torch.equal(out[good], want[good])


@gpu
def test_few_tokens_without_rows_captured(B):
    g, dt, wq, s, b = layer(1024, 80, 3, "bf16", True, True, 12)
    x = stream(g, 4, 1024, dt)
    x[2, 5] = float("nan")
    offsets = torch.tensor([0, 1, 3, 4], dtype=torch.int32, device=DEV)
    rows = torch.arange(4, device=DEV, dtype=torch.int32)
    out, ws = torch.empty(4, 80, dtype=dt, device=DEV), torch.empty(1 << 14, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.convrot_grouped_linear(x, wq, s, 128, offsets, bias=b, out=out, workspace=ws)
    for k in range(3):
        x[:2].mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        fine = [0, 1, 3]                      # the NaN token's codes are unspecified
        assert torch.equal(out[fine], by_expert(B, x, wq, s, 128, offsets, rows, b)[fine])


@gpu
@pytest.mark.parametrize("io", ["bf16", "fp16"])
def test_against_64_bits(B, io):
    """From the codes on: fp32 holds the int32 sum to half a step, then one
    product of scales, one fused multiply-add and the output's rounding."""
    M, K, N, E, P, group = 70, 1024, 200, 5, 260, 128
    g, dt, wq, s, b = layer(K, N, E, io, True, True, 7)
    x = stream(g, M, K, dt)
    offsets, rows = route(g, M, P, E)
    got = B.convrot_grouped_linear(x, wq, s, group, offsets, rows=rows, bias=b).double()
    q, qs = B.convrot_rotate_quant_ex(x, group)
    owner = torch.searchsorted(offsets[1:], torch.arange(P, device=DEV, dtype=torch.int32), right=True)
    prod = torch.stack([(q[rows[p].long()].double() * wq[owner[p]].double()).sum(1) for p in range(P)])
    prod = prod * qs.double()[rows.long()][:, None] * s.double()[owner]
    want = prod + b.double()[owner]
    tol = torch.finfo(dt).eps / 2 * want.abs() + 4 * 2.0 ** -24 * (prod.abs() + b.double()[owner].abs()) + 1e-7
    assert ((got - want).abs() <= tol * 1.01).all()


@gpu
@pytest.mark.parametrize("counts", [[0, 0, 0, 50], [50, 0, 0, 0], [0, 17, 0, 33], [1, 1, 1, 1], [16, 32, 0, 2], [0, 0, 0, 0]])
def test_experts_without_rows(B, counts):
    g, dt, wq, s, b = layer(256, 48, 4, "bf16", False, True, 3)
    P = sum(counts)
    x = stream(g, 20, 256, dt)
    offsets, rows = route(g, 20, P + 6, 4, counts)
    out = torch.full((P + 6, 48), 5.0, dtype=dt, device=DEV)
    B.convrot_grouped_linear(x, wq, s, 128, offsets, rows=rows, bias=b, out=out)
    assert (out[P:] == 5).all()                    # rows behind the last expert stay
    assert torch.equal(out[:P], by_expert(B, x, wq, s, 128, offsets, rows[:P], b))


@gpu
def test_rows_before_the_first_expert_and_odd_tokens(B):
    g, dt, wq, s, b = layer(512, 100, 3, "fp16", True, True, 4)
    x = stream(g, 30, 512, dt)
    offsets = torch.tensor([4, 30, 30, 71], dtype=torch.int32, device=DEV)
    rows = torch.randint(0, 30, (80,), generator=g, device=DEV).to(torch.int32)
    rows[10], rows[40], rows[70], rows[50] = -1, 30, 1 << 30, -(1 << 31)
    out = torch.full((80, 100), 5.0, dtype=dt, device=DEV)
    B.convrot_grouped_linear(x, wq, s, 256, offsets, rows=rows, bias=b, out=out)
    good = torch.zeros(80, dtype=torch.bool, device=DEV)
    good[4:71] = True
    good[[10, 40, 70, 50]] = False
    want = by_expert(B, x, wq, s, 256, offsets, rows.clamp(0, 29), b)
    assert (out[~good] == 5).all() and torch.equal(out[good], want[good])


@gpu
def test_offsets_outside_the_rows_are_clamped(B):
    g, dt, wq, s, b = layer(256, 64, 5, "bf16", False, False, 5)
    x = stream(g, 33, 256, dt)
    bad = torch.tensor([-7, 10, 6, 20, 33, 1 << 30], dtype=torch.int32, device=DEV)
    # clamped: [0, 10), none (6 is before 10), [6, 20), [20, 33), none
    out = B.convrot_grouped_linear(x, wq, s, 128, bad)
    rows = torch.arange(33, device=DEV, dtype=torch.int32)
    want = by_expert(B, x, wq, s, 128, torch.tensor([0, 10, 10, 20, 33, 33]), rows, b)
    assert torch.equal(out[10:], want[10:])
    assert torch.equal(out[:6], want[:6])         # rows 6 to 9 belong to two experts: either's
    buf = torch.full((40, 64), 5.0, dtype=dt, device=DEV)
    B.convrot_grouped_linear(x, wq, s, 128, torch.full((6,), 1 << 30, dtype=torch.int32, device=DEV), out=buf[:33])
    assert (buf == 5).all()


@gpu
@pytest.mark.parametrize("M", [3, 40, 500])
def test_offsets_that_jump_back_and_forth(B, M):
    """Every other expert claims all rows: more tiles than the call can launch.  Each piece of a
    row is some expert's or untouched, and nothing outside the rows is written."""
    E = 300
    g, dt, wq, s, b = layer(128, 48, E, "bf16", False, False, 13)
    x = stream(g, M, 128, dt)
    bad = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    bad[1::2] = 1 << 30
    buf = torch.full((M + 2, 48), 5.0, dtype=dt, device=DEV)
    B.convrot_grouped_linear(x, wq, s, 128, bad, out=buf[1:M + 1])
    torch.cuda.synchronize()
    assert (buf[[0, M + 1]] == 5).all()
    rows = torch.arange(M, device=DEV, dtype=torch.int32)
    # experts write a row's tiles in any order, 16 bytes at a time: each piece is some expert's
    pieces = lambda t: t.reshape(M, 6, 8)  # noqa: E731
    ok = (pieces(buf[1:M + 1]) == 5).all(2)
    for e in range(0, E, 2):
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[e + 1:] = M
        ok |= (pieces(by_expert(B, x, wq, s, 128, off, rows, None)) == pieces(buf[1:M + 1])).all(2)
    assert ok.all()


@gpu
def test_without_rows_row_p_is_token_p(B):
    g, dt, wq, s, b = layer(384, 130, 3, "bf16", True, True, 6)
    x = stream(g, 90, 384, dt)
    offsets = torch.tensor([0, 33, 33, 90], dtype=torch.int32, device=DEV)
    rows = torch.arange(90, device=DEV, dtype=torch.int32)
    assert torch.equal(B.convrot_grouped_linear(x, wq, s, 128, offsets, bias=b),
                       by_expert(B, x, wq, s, 128, offsets, rows, b))


@gpu
def test_non_finite_tokens_stay_alone(B):
    g, dt, wq, s, b = layer(512, 80, 2, "bf16", False, True, 8)
    x = stream(g, 24, 512, dt)
    offsets, rows = route(g, 24, 48, 2, [20, 28])
    clean = B.convrot_grouped_linear(x, wq, s, 128, offsets, rows=rows, bias=b)
    x[3, 7], x[9, 100] = float("inf"), float("nan")
    got = B.convrot_grouped_linear(x, wq, s, 128, offsets, rows=rows, bias=b)
    fine = (rows != 3) & (rows != 9)
    assert torch.equal(got[fine], clean[fine])


@gpu
def test_captured_with_other_offsets_and_on_two_streams(B):
    g, dt, wq, s, b = layer(512, 96, 6, "bf16", True, False, 9)
    M, P = 50, 150
    x = stream(g, M, 512, dt)
    offsets, rows = route(g, M, P, 6)
    out, ws = torch.empty(P, 96, dtype=dt, device=DEV), torch.empty(B.convrot_grouped_workspace(M, 512), dtype=torch.uint8,
                                                                    device=DEV)
    B.convrot_grouped_linear(x, wq, s, 256, offsets, rows=rows, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.convrot_grouped_linear(x, wq, s, 256, offsets, rows=rows, out=out, workspace=ws)
    for k in range(4):
        o, r = route(g, M, P, 6)
        offsets.copy_(o)
        rows.copy_(r)
        x.copy_(stream(g, M, 512, dt))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, by_expert(B, x, wq, s, 256, offsets, rows, None))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for st in streams:
        with torch.cuda.stream(st):
            outs.append(B.convrot_grouped_linear(x, wq, s, 256, offsets, rows=rows))
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


@gpu
def test_codes_past_four_gigabytes(B):
    """Tokens whose codes lie past 32 bits: 2^32 bytes is row 32768 of K = 131072."""
    K, M = 131072, 32768 + 40
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    g, dt, wq, s, b = layer(K, 16, 2, "bf16", False, False, 10)
    x = torch.zeros(M, K, dtype=dt, device=DEV)
    few = torch.tensor([0, 1, 32767, 32768, 32769, M - 1], device=DEV)
    x[few] = stream(g, 6, K, dt)
    rows = few.to(torch.int32)
    offsets = torch.tensor([0, 2, 6], dtype=torch.int32, device=DEV)
    got = B.convrot_grouped_linear(x, wq, s, 128, offsets, rows=rows)
    want = by_expert(B, x[few], wq, s, 128, offsets, torch.arange(6, device=DEV), None)
    assert torch.equal(got, want)


@gpu
def test_binding_refuses(B):
    g, dt, wq, s, b = layer(256, 32, 2, "bf16", False, True, 11)
    x = stream(g, 8, 256, dt)
    off, rows = route(g, 8, 20, 2)
    good = dict(x=x, wq=wq, w_scale=s, group=128, offsets=off, rows=rows, bias=b)
    for kw in (dict(x=x.float()), dict(x=x.cpu()), dict(wq=wq[0]), dict(wq=wq[:, :, :128]), dict(w_scale=s[:1]),
               dict(offsets=off[:2]), dict(offsets=off.long()), dict(rows=rows.long()), dict(bias=b[0]),
               dict(bias=b.float()), dict(out=x), dict(workspace=torch.empty(9, device=DEV))):
        with pytest.raises(ValueError):
            B.convrot_grouped_linear(**dict(good, **kw))
    with pytest.raises(B.ConvrotError):
        B.convrot_grouped_linear(**dict(good, workspace=torch.empty(64, dtype=torch.uint8, device=DEV)))
