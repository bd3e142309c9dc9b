"""convrot_linear_lora: the layer with the low-rank adapters of many requests beside it.

Tokens without an adapter have to equal convrot_linear_ex byte for byte; the
others are compared with the formula in 64 bits: the layer from its codes (exact
int32 sums), plus scale * (A x) B from the unrounded inputs.
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


def call(B, x=A, io=1, M=64, K=512, wq=A, ws=A, mode=0, N=64, g=128, bias=None, a=A, b=A, R=64, sc=A, off=A, n=4, mr=16,
         idx=A, y=A, w=A, wb=1 << 20):
    return B.lib().convrot_linear_lora(x, io, M, K, wq, ws, mode, N, g, bias, a, b, R, sc, off, n, mr, idx, y, w, wb,
                                       None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=64), EUNSUPPORTED), (dict(K=384, g=256), EINVAL), (dict(K=131072 + 128), EINVAL), (dict(io=0), EUNSUPPORTED),
    (dict(mode=2), EUNSUPPORTED), (dict(N=0), EINVAL), (dict(M=-1), EINVAL), (dict(n=0), EINVAL), (dict(n=65537), EINVAL),
    (dict(mr=0), EINVAL), (dict(mr=513), EINVAL), (dict(R=-1), EINVAL), (dict(R=(1 << 30) + 1), EINVAL),
    (dict(x=None), EINVAL), (dict(wq=None), EINVAL), (dict(ws=None), EINVAL), (dict(a=None), EINVAL),
    (dict(b=None), EINVAL), (dict(sc=None), EINVAL), (dict(off=None), EINVAL), (dict(idx=None), EINVAL),
    (dict(y=None), EINVAL), (dict(x=A + 8), EALIGN), (dict(wq=A + 4), EALIGN), (dict(y=A + 2), EALIGN),
    (dict(a=A + 2), EALIGN), (dict(w=A + 8), EALIGN), (dict(w=None), EWORKSPACE),
    (dict(wb=64 * 512 + 256 + 64 * 64 + 8 * 64 * 128 - 1), EWORKSPACE),
])
def test_refusals(B, kw, status):
    assert call(B, **kw) == status
    assert b"convrot_linear_lora" in B.lib().convrot_last_error()


def test_empty_and_workspace(B):
    assert call(B, M=0, x=None, wq=None, y=None, w=None, wb=0) == OK
    assert B.lib().convrot_last_error() == b""
    # slices of min(M, 2N) tokens: codes, scales, t rows (ranks are padded to 32), eight parts of their fp32 sums
    assert B.convrot_lora_workspace(64, 512, 64, 16) == 64 * 512 + 256 + 64 * 64 + 8 * 64 * 128
    assert B.convrot_lora_workspace(100, 512, 8, 40) == 16 * 512 + 256 + 16 * 128 + 8 * 16 * 256
    assert B.convrot_lora_workspace(64, 512, 64, 0) == 0 and B.convrot_lora_workspace(-1, 512, 64, 8) == 0


gpu = pytest.mark.gpu


def problem(M, K, N, io, ranks, row, bias, seed, run=None, none=0.2):
    """Adapters of the given ranks; tokens in runs of `run` tokens (1: each its own)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x = n(M, K)
    x[:, :: max(1, K // 3)] *= 20.0
    R = sum(ranks)
    index = torch.randint(0, len(ranks), (M,), generator=g, device=DEV)
    if run:
        index = index[torch.arange(M, device=DEV) // run]
    gone = torch.rand(M, generator=g, device=DEV) < none
    index = torch.where(gone, torch.where(torch.arange(M, device=DEV) % 2 == 0, -1, len(ranks)), index)
    off = torch.cumsum(torch.tensor([0] + list(ranks), device=DEV), 0)
    return dict(x=x.to(dt),
                wq=torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int8),
                w_scale=(0.5 + torch.rand(N if row else 1, generator=g, device=DEV)) * 2e-4,
                bias=n(N).to(dt) if bias else None, lora_a=(n(R, K) / K ** 0.5).to(dt), lora_b=(0.5 * n(R, N)).to(dt),
                lora_scale=0.5 + torch.rand(len(ranks), generator=g, device=DEV), offsets=off.to(torch.int32),
                index=index.to(torch.int32), max_rank=max(max(ranks), 1))


def reference(B, p, group):
    """The formula in 64 bits, and how far fp32 and the two roundings may be from it."""
    x, dt = p["x"], p["x"].dtype
    M, K = x.shape
    q, qs = B.convrot_rotate_quant_ex(x, group)
    prod = (q.double() @ p["wq"].double().t()) * qs.double()[:, None] * p["w_scale"].double()
    base = prod + (0 if p["bias"] is None else p["bias"].double())
    mag = prod.abs() + (0 if p["bias"] is None else p["bias"].double().abs())
    delta, t_lost = torch.zeros_like(base), torch.zeros_like(base)
    off = p["offsets"].tolist()
    for a in range(len(off) - 1):
        at = torch.nonzero(p["index"] == a).flatten()
        lo, hi = off[a], min(off[a + 1], off[a] + p["max_rank"])
        if not len(at) or hi <= lo:
            continue
        s, wa, wb = p["lora_scale"][a].double(), p["lora_a"][lo:hi].double(), p["lora_b"][lo:hi].double()
        t = s * (x[at].double() @ wa.t())
        delta[at] = t @ wb
        # t: half a step of the io type, and a sum in fp32 over at most K / 4 terms a wave and 16 parts
        lost = torch.finfo(dt).eps / 2 * t.abs() + (K / 4 + 20) * 2.0 ** -24 * s * (x[at].double().abs() @ wa.abs().t())
        t_lost[at] = lost @ wb.abs() + (hi - lo + 2) * 2.0 ** -24 * (t.abs() @ wb.abs())
    want = base + delta
    # fp32: the int32 sum, the scales, the multiply-add, the sum with the adapter's part
    tol = torch.finfo(dt).eps / 2 * want.abs() + 1.02 * t_lost + 5 * 2.0 ** -24 * (mag + delta.abs()) + 1e-7
    return want, tol


def check(B, p, group):
    got = B.convrot_linear_lora(**p, group=group)
    want, tol = reference(B, p, group)
    assert ((got.double() - want).abs() <= tol * 1.01).all()
    plain = B.convrot_linear_ex(p["x"], p["wq"], p["w_scale"], group, bias=p["bias"])
    none = (p["index"] < 0) | (p["index"] >= len(p["lora_scale"]))
    assert torch.equal(got[none], plain[none])
    return got


# one round of 256 x 128 or 256 x 192 tiles: few K, whole and ragged sides
@gpu
@pytest.mark.parametrize("io,row,bias", [("bf16", True, True), ("fp16", False, False)])
@pytest.mark.parametrize("M,K,N,ranks,run,group", [
    (257, 128, 14337, [16, 5], 100, 128), (1999, 256, 4095, [40] * 9, 50, 256), (2048, 384, 4096, [8], None, 128),
    (1301, 640, 4001, [64, 0, 33, 512], 7, 128), (2999, 128, 4090, [7, 300], 1000, 128), (400, 384, 28600, [16, 40, 9], 90, 128),
    (2112, 256, 4096, [1, 2, 3, 4, 5] * 20, 1, 256)])
def test_one_round(B, M, K, N, ranks, run, group, io, row, bias):
    check(B, problem(M, K, N, io, ranks, row, bias, M + K + N, run), group)


# every tile the call chooses from, ranks from 1 up, odd sizes, slices (M > 2N)
@gpu
@pytest.mark.parametrize("io,row,bias", [("bf16", False, True), ("fp16", True, False)])
@pytest.mark.parametrize("M,K,N,ranks,run,group", [
    (1, 128, 1, [1], None, 128), (1, 4096, 512, [16], None, 256), (7, 512, 100, [8, 0, 3], 1, 128),
    (16, 1024, 264, [16] * 16, 1, 256), (16, 2048, 8200, [16, 64, 5], 1, 128), (16, 4096, 8208, [8] * 20, 1, 256),
    (37, 640, 129, [33, 4], 5, 128), (64, 768, 200, [8] * 40, 1, 256), (100, 512, 8, [16, 32], 30, 128),
    (150, 512, 193, [64, 128, 1], 40, 256), (300, 1024, 520, [4] * 300, 1, 128), (523, 384, 250, [17, 512], 100, 128),
    (1100, 256, 577, [16, 48], 333, 256), (2500, 512, 1160, [64, 40, 8], 700, 128), (4700, 384, 1544, [24] * 5, 900, 128)])
def test_against_the_formula(B, M, K, N, ranks, run, group, io, row, bias):
    check(B, problem(M, K, N, io, ranks, row, bias, M + K + N, run), group)


@gpu
@pytest.mark.parametrize("M", [3, 16, 40, 200, 1500])
def test_a_token_does_not_see_the_others(B, M):
    """Its result stays when the others change their adapters, or those hold infinities and NaN."""
    p = problem(M, 512, 264, "bf16", [16, 8, 32, 24], False, True, M, 3, none=0.0)
    p["index"][M // 2] = 1
    want = B.convrot_linear_lora(**p, group=128)[M // 2]
    other = p["index"].clone()
    other[:M // 2] = 3
    other[M // 2 + 1:] = 0
    assert torch.equal(B.convrot_linear_lora(**dict(p, index=other), group=128)[M // 2], want)
    a, b, sc = p["lora_a"].clone(), p["lora_b"].clone(), p["lora_scale"].clone()
    a[:16], b[24:], sc[2] = float("nan"), float("inf"), float("-inf")     # adapter 1 is rows 16 to 23
    got = B.convrot_linear_lora(**dict(p, lora_a=a, lora_b=b, lora_scale=sc), group=128)
    mine = p["index"] == 1
    assert torch.equal(got[mine], B.convrot_linear_lora(**p, group=128)[mine])
    x = p["x"].clone()
    x[0, 3] = float("nan")
    assert torch.equal(B.convrot_linear_lora(**dict(p, x=x), group=128)[1:], B.convrot_linear_lora(**p, group=128)[1:])


@gpu
@pytest.mark.parametrize("M,N", [(1999, 4095), (3000, 4094)])
def test_infinities_of_others_in_one_round(B, M, N):
    """256 x 128 and 256 x 192 tiles: neighbours' infinities and NaN stay theirs."""
    p = problem(M, 256, N, "fp16", [16, 8, 32, 24], False, True, M, 3, none=0.1)
    want = B.convrot_linear_lora(**p, group=128)
    a, b, sc, x = p["lora_a"].clone(), p["lora_b"].clone(), p["lora_scale"].clone(), p["x"].clone()
    a[:16], b[24:], sc[2], x[7, 3] = float("nan"), float("inf"), float("-inf"), float("nan")
    got = B.convrot_linear_lora(**dict(p, lora_a=a, lora_b=b, lora_scale=sc, x=x), group=128)
    mine = (p["index"] != 0) & (p["index"] != 2) & (p["index"] != 3)
    mine[7] = False
    assert mine.sum() > M // 5 and torch.equal(got[mine], want[mine])


@gpu
@pytest.mark.parametrize("M,ranks", [(3, [5, 20]), (16, [17, 33]), (40, [5, 9, 12, 20, 3, 40]), (90, [5, 40]), (300, [7, 33])])
def test_infinities_are_the_formulas(B, M, ranks):
    """An infinite weight in an adapter's last row gives the infinity the sum has, not NaN from
    the padding behind it."""
    p = problem(M, 256, 40, "bf16", ranks, False, False, M, 2, none=0.0)
    last = p["offsets"][1:].long() - 1
    p["lora_b"][last, 3] = float("inf")
    got = B.convrot_linear_lora(**p, group=128)
    fine = torch.ones(40, dtype=torch.bool, device=DEV)
    fine[3] = False
    q = dict(p, lora_b=p["lora_b"].clone())
    q["lora_b"][last, 3] = 0.0
    assert torch.equal(got[:, fine], B.convrot_linear_lora(**q, group=128)[:, fine])
    a = p["index"].long()
    t = (p["lora_a"][last[a]].double() * p["x"].double()).sum(1)
    sure = t.abs() > 1e-3                    # far from a rounding to zero
    assert sure.sum() > M // 2
    assert torch.equal(got[sure, 3].double(), torch.where(t[sure] > 0, float("inf"), float("-inf")))


@gpu
@pytest.mark.parametrize("M", [16, 200])
def test_no_ranks_at_all_and_max_rank(B, M):
    p = problem(M, 256, 72, "fp16", [0, 0], False, True, 2, 4)
    assert p["lora_a"].shape[0] == 0
    assert torch.equal(check(B, p, 128), B.convrot_linear_ex(p["x"], p["wq"], p["w_scale"], 128, bias=p["bias"]))
    p = problem(M, 256, 72, "fp16", [40, 20], False, True, 2, 4)
    check(B, dict(p, max_rank=24), 128)            # rows past max_rank are not used
    check(B, dict(p, max_rank=512), 128)
    # offsets past the rows, and descending ones, are clamped
    p["offsets"] = torch.tensor([-5, 40, 1 << 30], dtype=torch.int32, device=DEV)
    q = dict(p, offsets=torch.tensor([0, 40, 60], dtype=torch.int32, device=DEV))
    assert torch.equal(B.convrot_linear_lora(**dict(p, max_rank=40), group=128),
                       B.convrot_linear_lora(**dict(q, max_rank=40), group=128))
    p["offsets"] = torch.tensor([50, 30, 1 << 30], dtype=torch.int32, device=DEV)     # adapter 0: none, 1: rows 30 on
    q = dict(p, offsets=torch.tensor([30, 30, 60], dtype=torch.int32, device=DEV))
    assert torch.equal(B.convrot_linear_lora(**dict(p, max_rank=40), group=128),
                       B.convrot_linear_lora(**dict(q, max_rank=40), group=128))


@gpu
def test_repeats_guards_streams_and_graphs(B):
    for M in (16, 130):
        p = problem(M, 1024, 200, "bf16", [16, 8, 40], True, True, 5, 2)
        want = B.convrot_linear_lora(**p, group=256)
        for _ in range(3):
            assert torch.equal(B.convrot_linear_lora(**p, group=256), want)
        buf = torch.full((M + 2, 200), 3.0, dtype=torch.bfloat16, device=DEV)
        need = B.convrot_lora_workspace(M, 1024, 200, 40)
        ws = torch.full((need + 512,), 77, dtype=torch.uint8, device=DEV)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            B.convrot_linear_lora(**p, group=256, out=buf[1:M + 1], workspace=ws[256:256 + need])
        st.synchronize()
        assert torch.equal(buf[1:M + 1], want) and (buf[[0, M + 1]] == 3).all()
        assert (ws[:256] == 77).all() and (ws[256 + need:] == 77).all()
        out = torch.empty_like(want)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.convrot_linear_lora(**p, group=256, out=out, workspace=ws)
        for k in range(3):
            p["index"].copy_(p["index"].roll(5))
            p["x"].mul_(0.75)
            ws.fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, B.convrot_linear_lora(**p, group=256))


@gpu
def test_binding_refuses(B):
    p = dict(problem(8, 256, 64, "bf16", [8, 8], False, True, 1), group=128)
    for kw in (dict(lora_a=p["lora_a"].float()), dict(lora_a=p["lora_a"][:, :128]), dict(lora_b=p["lora_b"].t()),
               dict(lora_b=p["lora_b"][:8]), dict(lora_scale=p["lora_scale"].double()), dict(offsets=p["offsets"][:2]),
               dict(index=p["index"].long()), dict(index=p["index"][:4]), dict(index=p["index"].cpu()),
               dict(out=p["x"]), dict(workspace=torch.empty(64, device=DEV))):
        with pytest.raises(ValueError):
            B.convrot_linear_lora(**dict(p, **kw))
    for kw in (dict(max_rank=0), dict(max_rank=513), dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(B.ConvrotError):
            B.convrot_linear_lora(**dict(p, **kw))
