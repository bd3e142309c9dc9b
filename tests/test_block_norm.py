"""convrot_block_norm: the step between two blocks, against its formulas in 64 bits.

The stored stream h' is rounded once from fp32, and the norm is that of the
stored values, so each of the two outputs is compared with what the formulas
give in 64 bits from the values the kernel itself read (its own h' for the
norm).  Tolerances: half a step of the output type relative to the value, plus
what fp32 loses before that rounding (see each test).  Codes are compared with
the codes of the 64-bit values: equal, or one apart where the value lies
within the fp32 error of a border between two codes.
"""
import ctypes
import math

import pytest
import torch

import oracle  # noqa: F401  (the tests share its build with the other modules)

OK, EINVAL, EUNSUPPORTED, EALIGN, EWORKSPACE = 0, -1, -2, -3, -4
A = 0x10000          # a fake, 16-byte aligned device address (never dereferenced)
DEV = "cuda:0"
EPS = 1e-6


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
    base = dict(io_dtype=1, group=0, post_norm=0, pre_norm=1, n_routes=0, eps=EPS, residual_scale=1.0, M=4, K=512,
                h=A, u=A + 4096, h_out=A + 8192, out=A + 16384, out_scale=A + 32768)
    base.update(kw)
    return B.lib().convrot_block_norm(ctypes.byref(B.Block(**base)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(io_dtype=0), EUNSUPPORTED), (dict(io_dtype=7), EUNSUPPORTED),
    (dict(group=64), EUNSUPPORTED), (dict(group=256, K=384), EINVAL), (dict(group=128, K=136), EINVAL),
    (dict(K=4), EINVAL), (dict(K=0), EINVAL), (dict(K=508), EINVAL), (dict(K=-8), EINVAL), (dict(K=32776), EUNSUPPORTED),
    (dict(group=128, K=32768 + 128), EUNSUPPORTED), (dict(M=-1), EINVAL), (dict(M=1 << 31), EINVAL),
    (dict(post_norm=3), EUNSUPPORTED), (dict(pre_norm=-1), EUNSUPPORTED),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(residual_scale=float("nan")), EINVAL), (dict(residual_scale=float("-inf")), EINVAL),
    (dict(n_routes=-1), EINVAL), (dict(n_routes=65), EINVAL), (dict(u_rows=-1), EINVAL),
    (dict(n_routes=2, u_rows=8), EINVAL), (dict(n_routes=2, u_rows=8, route_row=A), EINVAL),
    (dict(gate=A), EINVAL), (dict(n_mod=1), EINVAL), (dict(scale=A, n_mod=2, mod_stride=504), EINVAL),
    (dict(shift=A, n_mod=2, mod_stride=516), EINVAL),
    (dict(h=None), EINVAL), (dict(h_out=None), EINVAL), (dict(u=None, out=None), EINVAL),
    (dict(u=None, post_norm=1), EINVAL), (dict(u=None, residual_scale=2.0), EINVAL),
    (dict(u=None, gate=A, n_mod=1, mod_stride=512), EINVAL),
    (dict(group=128, out_scale=None), EINVAL),
    (dict(h=A + 8), EALIGN), (dict(u=A + 2), EALIGN), (dict(out=A + 4), EALIGN), (dict(h_out=A + 8), EALIGN),
    (dict(pre_weight=A + 8), EALIGN), (dict(post_weight=A + 8), EALIGN),
    (dict(shift=A + 8, n_mod=1, mod_stride=512), EALIGN),
])
def test_refusals(B, kw, status):
    assert refused(B, **kw) == status
    assert b"convrot_block_norm" in B.lib().convrot_last_error()


def test_refuses_null_and_takes_an_empty_batch(B):
    assert B.lib().convrot_block_norm(None, None) == EINVAL
    assert refused(B, M=0, h=None, u=None, h_out=None, out=None) == OK
    assert B.lib().convrot_last_error() == b""
    assert ctypes.sizeof(B.Block) == 176        # 7 words and a gap, 18 of 8 bytes


def test_binding_refuses_cpu_tensors(B):
    with pytest.raises(ValueError):
        B.convrot_block_norm(torch.zeros(2, 128, dtype=torch.bfloat16))


# ---------------------------------------------------------------- the formulas in 64 bits

def ref_norm(x, mag, kind, weight):
    """The normed x, and the magnitude of the terms that were added up to each value."""
    if kind == "none":
        return x, mag
    if kind == "layer":
        x, mag = x - x.mean(1, keepdim=True), mag + mag.mean(1, keepdim=True)
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    w = 1.0 if weight is None else weight.double()
    return x * r * w, mag * r * abs(w)


def ref_mod(t, index, M):
    """Rows of a modulation for each token; None where the token has none."""
    n = t.shape[0]
    index = torch.zeros(M, dtype=torch.int64, device=t.device) if index is None else index.long()
    good = (index >= 0) & (index < n)
    return t.double()[index.clamp(0, n - 1)], good[:, None]


def ref_h(c):
    h, u = c["h"].double(), c["u"].double()
    mag = u.abs()
    if c["routes"] is not None:
        row, weight = c["routes"]
        good = (row >= 0) & (row < u.shape[0])
        picked = u[row.long().clamp(0, max(0, u.shape[0] - 1))] if u.shape[0] else u.new_zeros(*row.shape, h.shape[1])
        terms = torch.where(good[:, :, None], picked, 0.0) * weight.double()[:, :, None]
        u, mag = terms.sum(1), terms.abs().sum(1)
    p, mag = ref_norm(u, mag, c["post_norm"], c["post_weight"])
    if c["gate"] is not None:
        g, good = ref_mod(c["gate"], c["mod_index"], h.shape[0])
        p, mag = torch.where(good, g * p, p), torch.where(good, g.abs() * mag, mag)
    h = c["residual_scale"] * h
    return h + p, h.abs() + mag


def ref_out(c, h):
    z, mag = ref_norm(h.double(), h.double().abs(), c["pre_norm"], c["pre_weight"])
    add = torch.zeros_like(z)
    for name in ("scale", "shift"):
        if c[name] is not None:
            m, good = ref_mod(c[name], c["mod_index"], h.shape[0])
            if name == "scale":
                z, mag = torch.where(good, z * (1 + m), z), torch.where(good, mag * (1 + m.abs()), mag)
            else:
                add = torch.where(good, m, add)
    return z + add, mag + add.abs()


def case(M, K, io, post="none", pre="rms", mods=0, routes=0, seed=0, spread=1.0, mean=0.0, weights=True, index=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000 * M + K + seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    h = n(M, K) * spread + mean
    h[:, :: max(1, K // 5)] *= 15.0
    P = M * routes + 3 if routes else M
    c = dict(h=h.to(dt), u=(n(P, K) + mean).to(dt), routes=None, post_norm=post, pre_norm=pre, post_weight=None,
             pre_weight=None, gate=None, scale=None, shift=None, mod_index=None, residual_scale=0.75, eps=EPS)
    if weights:
        c["post_weight"], c["pre_weight"] = (1 + 0.2 * n(K)).to(dt), (1 + 0.2 * n(K)).to(dt)
    if routes:
        row = torch.randint(-2, P + 2, (M, routes), generator=g, device=DEV).to(torch.int32)
        c["routes"] = (row, torch.softmax(n(M, routes), 1))
    if mods:
        mod = (0.4 * n(mods, 3 * K)).to(dt)
        c["gate"], c["scale"], c["shift"] = mod[:, :K], mod[:, K:2 * K], mod[:, 2 * K:]
        if index:
            c["mod_index"] = torch.randint(-1, mods + 1, (M,), generator=g, device=DEV).to(torch.int32)
    return c


# What fp32 loses before the rounding, in steps of 2^-24 of the terms' magnitude.
# A sum over the row adds up to 8 * 4 values in a lane, then ten levels of a
# tree: 42 steps of the sum of magnitudes, half of them through the square root
# of a sum of squares, once more for a layer norm's mean.  The root, the
# division, 1/K, the weight, the gate, the modulation and up to 5 routed rows
# add one each: under 21 + 42 + 16.
SLACK = 80


def close(got, want_mag, dt, what):
    """got = rnd(want): half a step of the value, and what fp32 lost before it."""
    want, mag = want_mag
    tiny = torch.finfo(dt).tiny * torch.finfo(dt).eps / 2      # half a subnormal step
    tol = torch.finfo(dt).eps / 2 * want.abs() + SLACK * 2.0 ** -24 * 1.01 * mag + tiny
    off = (got.double() - want).abs() / tol
    assert (off <= 1).all(), f"{what}: {int((off > 1).sum())} off, worst {float(off.max()):.2f} of the tolerance"


def check(B, c, group=0, **kw):
    dt = c["h"].dtype
    got = B.convrot_block_norm(**c, group=group, **kw)
    torch.cuda.synchronize()
    h = got[0]
    close(h, ref_h(c), dt, "h_out")
    if not group:
        close(got[1], ref_out(c, h), dt, "out")
    else:
        check_codes(got[1], got[2], *ref_out(c, h), group)
    return got


def rotate64(x, g):
    i = torch.arange(g, device=x.device)
    bits = i[:, None] & i[None, :]
    sign = torch.zeros_like(bits)
    for t in range(8):
        sign ^= (bits >> t) & 1
    H = (1.0 - 2.0 * sign.double()) / math.sqrt(g)
    return (x.reshape(-1, g) @ H).reshape(x.shape)


def check_codes(q, s, z, mag, group):
    """Codes and scales of the rotated z: the scale within the fp32 error of the
    row's largest value, each code the nearest one to v / s up to that error."""
    v = rotate64(z, group)
    # fp32 error of a rotated value: SLACK steps of each term, averaged by the
    # orthogonal rotation (2-norm of the block's terms), and log2 g roundings
    lost = (SLACK + 9) * 2.0 ** -24 * mag.reshape(-1, group).norm(dim=1).repeat_interleave(group).reshape(z.shape)
    amax = v.abs().amax(1)
    worst = lost.amax(1)
    assert ((s.double() * 127 - amax).abs() <= worst + 2.0 ** -22 * amax).all(), "scale"
    safe = torch.where(s > 0, s.double(), 1.0)[:, None]
    t = v / safe
    assert ((q.double() - t.clamp(-127, 127)).abs() <= 0.5 + lost / safe + 2.0 ** -22 * t.abs() + 1e-9).all(), "codes"
    assert (q[s == 0] == 0).all()


gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K", [(1, 8), (3, 504), (5, 512), (2, 520), (7, 1000), (4, 2048), (3, 2056), (130, 4096),
                                 (2, 8192), (3, 12288), (2, 16392), (1, 32768)])
def test_rms_both_sides(B, M, K, io):
    check(B, case(M, K, io, post="rms", pre="rms"))


@gpu
@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("mods,routes", [(0, 0), (3, 0), (0, 2), (2, 5)])
def test_kinds(B, post, pre, mods, routes, io):
    check(B, case(33, 776, io, post=post, pre=pre, mods=mods, routes=routes))


@gpu
@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("K,group", [(128, 128), (256, 256), (640, 128), (768, 256), (2048, 256), (2176, 128),
                                     (4096, 128), (6144, 256), (8192, 128), (12288, 256), (16512, 128), (32768, 256)])
def test_codes(B, K, group, io):
    check(B, case(9, K, io, post="rms", pre="layer", mods=2), group=group)
    check(B, case(5, K, io, post="none", pre="rms", routes=3, seed=1), group=group)


@gpu
@pytest.mark.parametrize("group", [128, 256])
def test_codes_of_a_plain_stream_are_rotate_quants(B, group):
    # no norm, no modulation: the same values rotated in the same order
    c = case(37, 2048, "bf16", pre="none", weights=False)
    h, q, s = B.convrot_block_norm(c["h"], pre_norm="none", group=group)
    q2, s2 = B.convrot_rotate_quant(c["h"], group)
    assert h is c["h"] and torch.equal(q, q2) and torch.equal(s, s2)


@gpu
def test_norm_alone_equals_the_second_half(B):
    """The norm of h' is that of the stored stream: fused and apart, the same bytes."""
    c = case(50, 1536, "bf16", post="layer", pre="rms", mods=3)
    h, z = B.convrot_block_norm(**c)
    again, z2 = B.convrot_block_norm(h, pre_norm="rms", pre_weight=c["pre_weight"], scale=c["scale"], shift=c["shift"],
                                     mod_index=c["mod_index"], eps=EPS)
    assert again is h and torch.equal(z, z2)
    only = B.convrot_block_norm(**c, want_out=False)
    assert torch.equal(only, h)


@gpu
def test_layer_norm_with_a_far_mean(B):
    """A mean of 200 beside a spread of 1: the variance is that of the centred
    values, and what is lost stays within some steps of the mean."""
    c = case(20, 4096, "bf16", post="none", pre="layer", weights=False)
    c["h"] = (200 + torch.randn(20, 4096, device=DEV)).to(torch.bfloat16)
    c["u"] = torch.zeros_like(c["u"])
    c["residual_scale"] = 1.0
    h, z = check(B, c)
    assert torch.equal(h, c["h"])


@gpu
def test_zero_rows_and_nothing_routed(B):
    c = case(6, 1024, "bf16", post="rms", pre="rms", routes=2, weights=False)
    c["h"][1] = 0
    c["routes"][0][1] = -1                       # token 1: no row, a zero stream
    c["routes"][0][2] = 1 << 30                  # token 2: rows out of range only
    h, z = check(B, c)
    assert (h[1] == 0).all() and (z[1] == 0).all()
    h, q, s = B.convrot_block_norm(**c, group=128)
    assert (q[1] == 0).all() and s[1] == 0
    # no rows at all to route to
    c["u"] = c["u"][:0]
    h, _ = B.convrot_block_norm(**c)
    assert torch.equal(h, (0.75 * c["h"].float()).to(torch.bfloat16))


@gpu
def test_non_finite_rows_stay_alone(B):
    c = case(8, 2048, "fp16", post="rms", pre="layer", mods=2)
    clean = B.convrot_block_norm(**c)
    c["h"] = c["h"].clone()
    c["h"][2, 5], c["h"][5, 7], c["u"][6, 9] = float("inf"), float("nan"), float("-inf")
    got = B.convrot_block_norm(**c)
    rows = [0, 1, 3, 4, 7]
    assert torch.equal(got[0][rows], clean[0][rows]) and torch.equal(got[1][rows], clean[1][rows])
    assert torch.isnan(got[1][5]).any() and not torch.isfinite(got[0][2, 5])


@gpu
def test_in_place_strides_streams_and_bounds(B):
    c = case(65, 1160, "bf16", post="rms", pre="rms", mods=4)
    want = B.convrot_block_norm(**c)
    # a single row of modulation: a chunk whose own stride is not a multiple of 8
    one = dict(c, gate=c["gate"][:1], scale=c["scale"][:1], shift=c["shift"][:1], mod_index=None)
    check(B, one)
    # in place, on a stream of its own, between guard rows that stay as they were
    buf = torch.full((67, 1160), 7.0, dtype=torch.bfloat16, device=DEV)
    out = torch.full((67, 1160), 9.0, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        buf[1:66] = c["h"]
        d = dict(c, h=buf[1:66])
        B.convrot_block_norm(**d, h_out=buf[1:66], out=out[1:66])
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(buf[1:66], want[0]) and torch.equal(out[1:66], want[1])
    assert (buf[[0, 66]] == 7).all() and (out[[0, 66]] == 9).all()


@gpu
def test_more_rows_than_one_grid_dimension(B):
    """2^24 workgroups of 256 threads would be 2^32 threads along x."""
    M, K = (1 << 24) + 3, 8
    h = (torch.arange(M, device=DEV, dtype=torch.int32) % 251).to(torch.bfloat16)[:, None].expand(M, K).contiguous()
    _, z = B.convrot_block_norm(h, pre_norm="rms")
    few = torch.tensor([0, 1, 250, (1 << 20) - 1, 1 << 20, (1 << 24) - 1, 1 << 24, M - 1], device=DEV)
    _, want = B.convrot_block_norm(h[few].contiguous(), pre_norm="rms")
    assert torch.equal(z[few], want) and int((z != 0).sum()) == int((h != 0).sum())


@gpu
def test_captured_and_replayed(B):
    c = case(40, 2048, "bf16", post="rms", pre="layer", mods=2, routes=4)
    h, q, s = B.convrot_block_norm(**c, group=128)
    bufs = [torch.empty_like(t) for t in (h, q, s)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.convrot_block_norm(**c, group=128, h_out=bufs[0], out=bufs[1], out_scale=bufs[2])
    for k in range(3):
        c["h"].mul_(0.5 + k)
        want = B.convrot_block_norm(**c, group=128)
        for b in bufs:
            b.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bufs, want))


@gpu
def test_binding_refuses(B):
    c = case(4, 512, "bf16", mods=2, routes=2)
    for kw in (dict(u=c["u"][:2], routes=None), dict(routes=(c["routes"][0].long(), c["routes"][1])),
               dict(gate=c["gate"].float()), dict(gate=c["gate"].contiguous()), dict(scale=c["scale"][:1]),
               dict(pre_norm="batch"), dict(pre_weight=c["pre_weight"][:256]), dict(mod_index=c["mod_index"][:3]),
               dict(u=None), dict(u=None, routes=None, h_out=c["h"]),
               dict(gate=None, scale=None, shift=None)):
        with pytest.raises(ValueError):
            B.convrot_block_norm(**dict(c, **kw))
    with pytest.raises(B.ConvrotError):
        B.convrot_block_norm(**dict(c, eps=-1.0))
