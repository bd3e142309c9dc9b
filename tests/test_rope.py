"""convrot_rope and convrot_rope_frequencies: rotary positions against their formulas in 64 bits.

Tolerance of a turned value: half a step of the output type, and 8 fp32 steps of
scale (|a| + |b|): the turns left after the whole ones are dropped go to fp32 within 2^-26
(2 pi 2^-26 = 1.6 2^-24 radians), sine and cosine within 2 2^-24, their products with the
scale and the values and the sum 1 2^-24 each."""
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

def refused(B, **kw):
    a = dict(q=A, q_heads=4, q_stride=512, q_out=A, q_out_stride=512, k=A + 4096, k_heads=2, k_stride=512, k_out=A + 8192,
             k_out_stride=256, io=1, M=3, head_dim=128, rot_dim=64, layout=0, positions=A, freqs=A, scale=1.0, inverse=0)
    a.update(kw)
    return B.lib().convrot_rope(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(io=0), EUNSUPPORTED), (dict(io=3), EUNSUPPORTED), (dict(layout=2), EUNSUPPORTED), (dict(layout=-1), EUNSUPPORTED),
    (dict(M=-1), EINVAL), (dict(M=(1 << 30) + 1), EINVAL), (dict(head_dim=0), EINVAL), (dict(head_dim=4), EINVAL),
    (dict(head_dim=100), EINVAL), (dict(head_dim=1032), EINVAL), (dict(rot_dim=0), EINVAL), (dict(rot_dim=63), EINVAL),
    (dict(rot_dim=130), EINVAL), (dict(rot_dim=-2), EINVAL), (dict(q_heads=-1), EINVAL), (dict(k_heads=-1), EINVAL),
    (dict(q_heads=0, k_heads=0), EINVAL), (dict(q_heads=16384), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(q_stride=504), EINVAL), (dict(q_stride=516), EINVAL),
    (dict(k_out_stride=248), EINVAL), (dict(q=None), EINVAL), (dict(k_out=None), EINVAL), (dict(q_out=None), EINVAL),
    (dict(positions=None), EINVAL), (dict(freqs=None), EINVAL), (dict(q_out_stride=520), EINVAL),
    (dict(q=A + 8), EALIGN), (dict(q_out=A + 2), EALIGN), (dict(k=A + 4), EALIGN), (dict(k_out=A + 8), EALIGN),
])
def test_refusals(B, kw, status):
    assert refused(B, **kw) == status
    assert b"convrot_rope" in B.lib().convrot_last_error()


def test_takes_an_empty_batch_and_refuses_cpu_tensors(B):
    assert refused(B, M=0, q=None, k=None, q_out=None, k_out=None, positions=None, freqs=None) == OK
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.convrot_rope(x, None, torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))


# ---------------------------------------------------------------- frequencies (host)

@pytest.mark.parametrize("kw,status", [
    (dict(scaling=5), EUNSUPPORTED), (dict(scaling=-1), EUNSUPPORTED), (dict(rot=0), EINVAL), (dict(rot=7), EINVAL),
    (dict(rot=1026), EINVAL), (dict(base=1.0), EINVAL), (dict(base=math.inf), EINVAL), (dict(base=math.nan), EINVAL),
    (dict(scaling=1, factor=0.5), EINVAL), (dict(scaling=2, factor=math.nan), EINVAL), (dict(scaling=2, rot=2), EINVAL),
    (dict(scaling=2, base=1e300, factor=1e300), EINVAL),
    (dict(scaling=3, length=0.0), EINVAL), (dict(scaling=4, length=math.inf), EINVAL), (dict(scaling=3, low=0.0), EINVAL),
    (dict(scaling=4, low=4.0, high=4.0), EINVAL), (dict(scaling=3, high=math.inf), EINVAL), (dict(freqs=False), EINVAL),
])
def test_frequency_refusals(B, kw, status):
    a = dict(rot=64, base=1e4, scaling=0, factor=8.0, length=4096.0, low=1.0, high=32.0, freqs=True)
    a.update(kw)
    f, s = (ctypes.c_double * 512)(), ctypes.c_float()
    rc = B.lib().convrot_rope_frequencies(a["rot"], a["base"], a["scaling"], a["factor"], a["length"], a["low"], a["high"],
                                          f if a["freqs"] else None, ctypes.byref(s))
    assert rc == status and b"convrot_rope_frequencies" in B.lib().convrot_last_error()


def test_frequencies_follow_their_formulas(B):
    rot, base, factor, L = 128, 10000.0, 16.0, 4096.0
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
    close = lambda got, want: all(math.isclose(a, b, rel_tol=1e-14) for a, b in zip(got.tolist(), want))  # noqa: E731
    f, s = B.convrot_rope_frequencies(rot, base)
    assert f.dtype == torch.float64 and s == 1.0 and close(f, plain)
    f, s = B.convrot_rope_frequencies(rot, base, "linear", factor)
    assert s == 1.0 and close(f, [x / factor for x in plain])
    f, s = B.convrot_rope_frequencies(rot, base, "ntk", factor)
    # the slowest pair is interpolated in full, the fastest not at all
    assert s == 1.0 and f[0] == 1.0 and math.isclose(f[-1].item(), plain[-1] / factor, rel_tol=1e-12)
    f, s = B.convrot_rope_frequencies(rot, base, "yarn", factor, L)
    lo = math.floor(rot * math.log(L / (32 * 2 * math.pi)) / (2 * math.log(base)))
    hi = math.ceil(rot * math.log(L / (2 * math.pi)) / (2 * math.log(base)))
    assert (lo, hi) == (20, 46) and math.isclose(s, 0.1 * math.log(16) + 1, rel_tol=1e-7)
    assert close(f[:21], plain[:21]) and close(f[46:], [x / factor for x in plain[46:]])
    assert close(f[33:34], [plain[33] * 0.5 + plain[33] / factor * 0.5])
    f, s = B.convrot_rope_frequencies(rot, base, "bands", factor, L, 1.0, 4.0)
    for x, p in zip(f.tolist(), plain):
        turns = L * p / (2 * math.pi)
        k = min(max((turns - 1) / 3, 0), 1)
        assert math.isclose(x, p * k + p / factor * (1 - k), rel_tol=1e-13)
    # a factor of 1 scales nothing
    for kind in ("linear", "ntk", "yarn", "bands"):
        f, s = B.convrot_rope_frequencies(rot, base, kind, 1.0, L)
        assert s == 1.0 and close(f, plain)
    with pytest.raises(ValueError):
        B.convrot_rope_frequencies(rot, base, "other")


# ---------------------------------------------------------------- against the formulas

def check(got, x, positions, freqs, scale, layout, inverse=False):
    want, mag = ref.rope(x, positions, freqs, scale, layout, inverse)
    rot = 2 * freqs.shape[0]
    tol = torch.finfo(x.dtype).eps / 2 * want.abs() + 8 * 2.0 ** -24 * mag + 2.0 ** -25
    assert ((got.double() - want).abs() <= tol).all(), (got.double() - want).abs().max()
    assert torch.equal(got[..., rot:], x[..., rot:])


SHAPES = [(1, 32, 8, 128, 128), (5, 3, 1, 64, 64), (7, 4, 2, 80, 20), (300, 5, 5, 96, 24), (33, 2, 1, 256, 64),
          (2, 1, 1, 8, 2), (1030, 6, 2, 64, 32), (9, 7, 1, 1024, 1024), (4, 1, 3, 72, 60), (1, 1, 0, 16, 8), (2100, 2, 2, 64, 48)]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("M,Hq,Hk,D,rot", SHAPES)
def test_against_the_formula(B, M, Hq, Hk, D, rot, io, layout):
    g = torch.Generator(device=DEV)
    g.manual_seed(M + D + rot)
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    qkv = torch.randn(M, Hq + 2 * Hk + 1, D, generator=g, device=DEV).to(dt)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk] if Hk else None
    pos = torch.randint(1 - 2 ** 31, 2 ** 31 - 1, (M,), generator=g, device=DEV).to(torch.int32)
    pos[: M // 2] = torch.arange(M // 2, device=DEV, dtype=torch.int32)
    # 2^31 turns leave 2^-22 of one in 64 bits, which the formula in 64 bits shares only below 2^20
    pos = torch.where(pos.abs() > 2 ** 20, pos % 2 ** 20, pos)
    freqs, scale = B.convrot_rope_frequencies(rot, 10000.0, "yarn", 8.0, 4096.0, device=DEV)
    qo, ko = B.convrot_rope(q, k, pos, freqs, scale=scale, layout=layout)
    check(qo, q, pos, freqs, scale, layout)
    if Hk:
        check(ko, k, pos, freqs, scale, layout)
    # in place, in the rows of the projection: everything beside the two parts stays
    before = qkv.clone()
    a, b = B.convrot_rope(q, k, pos, freqs, scale=scale, layout=layout, q_out=q, k_out=k)
    assert a.data_ptr() == q.data_ptr() and torch.equal(q, qo) and (not Hk or torch.equal(k, ko))
    assert torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_is_the_inverse_turn(B, layout):
    """<turn(x), y> = <x, inverse(y)> in full, and differences of the formula along one direction."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    M, H, D, rot = 19, 3, 64, 48
    freqs, scale = B.convrot_rope_frequencies(rot, 500.0, "yarn", 4.0, 1000.0, device=DEV)
    pos = torch.randint(0, 5000, (M,), generator=g, device=DEV).to(torch.int32)
    x, y = (torch.randn(M, H, D, generator=g, device=DEV).to(torch.float16) for _ in range(2))
    grad, _ = B.convrot_rope(y, None, pos, freqs, scale=scale, layout=layout, inverse=True)
    check(grad, y, pos, freqs, scale, layout, inverse=True)
    t = x.double().requires_grad_()
    rot_dims = ref.rope(t, pos, freqs, scale, layout)[0]
    (rot_dims * y.double()).sum().backward()
    tol = torch.finfo(torch.float16).eps / 2 * t.grad.abs() + 8 * 2.0 ** -24 * 8 * scale + 2.0 ** -25
    assert ((grad.double() - t.grad).abs() <= tol).all()
    d = torch.randn(M, H, D, generator=g, device=DEV, dtype=torch.float64)
    up, down = (ref.rope(x.double() + e * d, pos, freqs, scale, layout)[0] for e in (1e-3, -1e-3))
    slope = ((up - down) * y.double()).sum() / 2e-3
    assert abs(slope - (grad.double() * d).sum()) <= (tol * d.abs()).sum() + 1e-8 * slope.abs()


@pytest.mark.gpu
def test_infinities_stay_in_their_pair(B):
    x = torch.randn(3, 2, 64, device=DEV).to(torch.bfloat16)
    x[1, 0, 5], x[1, 1, 60] = math.inf, math.nan
    freqs, _ = B.convrot_rope_frequencies(64, device=DEV)
    pos = torch.tensor([3, 70000, 9], dtype=torch.int32, device=DEV)
    got, _ = B.convrot_rope(x, None, pos, freqs)
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[1, 0, 5] = want[1, 0, 37] = want[1, 1, 60] = want[1, 1, 28] = True
    assert torch.equal(bad, want)


@pytest.mark.gpu
def test_captured_and_on_another_stream(B):
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    q, k = torch.randn(70, 4, 128, generator=g, device=DEV).half(), torch.randn(70, 2, 128, generator=g, device=DEV).half()
    pos = torch.arange(70, dtype=torch.int32, device=DEV)
    freqs, _ = B.convrot_rope_frequencies(128, device=DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    B.convrot_rope(q, k, pos, freqs, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.convrot_rope(q, k, pos, freqs, q_out=qo, k_out=ko)
    for i in range(3):
        q.normal_(generator=g), k.normal_(generator=g), pos.add_(1000 * i)
        graph.replay()
        torch.cuda.synchronize()
        a, b = B.convrot_rope(q, k, pos, freqs)
        assert torch.equal(a, qo) and torch.equal(b, ko)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b = B.convrot_rope(q, k, pos, freqs)
    side.synchronize()
    assert torch.equal(a, qo) and torch.equal(b, ko)


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit(B):
    q = torch.zeros(4, 2, 64, dtype=torch.float16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    f, _ = B.convrot_rope_frequencies(64, device=DEV)
    for bad in (dict(k=q[:3]), dict(k=q.bfloat16()), dict(positions=pos[:3]), dict(positions=pos.long()), dict(freqs=f.float()),
                dict(q=q.transpose(0, 1)), dict(q=q[:, :, ::2]), dict(layout="other"), dict(k_out=q), dict(q_out=q[:2]),
                dict(q_out=q[:1].expand(4, 2, 64))):
        args = {**dict(q=q, k=None, positions=pos, freqs=f), **bad}
        with pytest.raises(ValueError):
            B.convrot_rope(**args)
    with pytest.raises(B.ConvrotError):
        B.convrot_rope(q, None, pos, torch.zeros(40, dtype=torch.float64, device=DEV))
