"""A transformer block through the layer and the operators around it, as a server runs it: the
norm before, the projection with each request's adapter, the norm between, the routed experts
and the sum of their rows with the norm after -- against the same block in 64 bits.

Each step's codes are those of its own input, so the 64-bit block takes the codes and the
rounded tensors at the joints from the run (they are checked step by step elsewhere) and
compares every joint with what the formulas make of the joint before.  Norms as in
test_block_norm; the layers' outputs within half a step of the io type, the adapters' rounded
first product and a few fp32 steps.
"""
import pytest
import torch

from tests.test_block_norm import close, ref_h, ref_out
from tests.test_linear_lora import reference as lora_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def B():
    from w8a8_rotated_int8_convrot_amd import binding
    binding.lib()
    return binding


def model(io, K, F, E, group, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float16
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    q = lambda *s: (n(*s) * 28).round().clamp(-127, 127).to(torch.int8)  # noqa: E731
    ranks = [8, 24, 16]
    off = torch.tensor([0, 8, 32, 48], dtype=torch.int32, device=DEV)
    w = dict(norm1=(1 + 0.1 * n(K)).to(dt), norm2=(1 + 0.1 * n(K)).to(dt), norm3=(1 + 0.1 * n(K)).to(dt),
             mod=(0.3 * n(3, 3 * K)).to(dt), proj=q(K, K), proj_s=torch.full((1,), 0.03 / 28 / K ** 0.5 * 32, device=DEV),
             a=(n(sum(ranks), K) / K ** 0.5).to(dt), b=(0.2 * n(sum(ranks), K)).to(dt),
             s=0.5 + torch.rand(3, generator=g, device=DEV), off=off, up=q(E, F, K),
             up_s=(0.5 + torch.rand(E, F, generator=g, device=DEV)) / (28 * K ** 0.5), down=q(E, K, F),
             down_s=(0.5 + torch.rand(E, generator=g, device=DEV)) / (28 * F ** 0.5), group=group)
    return g, dt, w


def route(g, M, E, top):
    """Rows sorted by expert: their tokens, the offsets, and each token's rows and weights."""
    logits = torch.randn(M, E, generator=g, device=DEV)
    weight, chosen = torch.topk(torch.softmax(logits, 1), top)
    expert, order = torch.sort(chosen.reshape(-1), stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.cumsum(torch.bincount(expert, minlength=E), 0)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=DEV)
    return off, (order // top).to(torch.int32), pos.view(M, top).to(torch.int32), weight.contiguous()


def block(B, w, h, index, r):
    """One block; returns the tensors at its joints."""
    off, rows, pos, weight = r
    K, grp = h.shape[1], w["group"]
    _, x = B.convrot_block_norm(h, pre_weight=w["norm1"])
    attn = B.convrot_linear_lora(x, w["proj"], w["proj_s"], grp, w["a"], w["b"], w["s"], w["off"], index, 24)
    gate, scale, shift = w["mod"][:, :K], w["mod"][:, K:2 * K], w["mod"][:, 2 * K:]
    h1, y = B.convrot_block_norm(h, attn, post_norm="rms", post_weight=w["norm2"], gate=gate, scale=scale, shift=shift,
                                 mod_index=index, pre_norm="layer")
    up = B.convrot_grouped_linear(y, w["up"], w["up_s"], grp, off, rows=rows)
    act = torch.nn.functional.silu(up.float()).to(h.dtype)
    down = B.convrot_grouped_linear(act, w["down"], w["down_s"], grp, off)
    h2, codes, s = B.convrot_block_norm(h1, down, routes=(pos, weight), pre_weight=w["norm3"], group=grp)
    return dict(x=x, attn=attn, h1=h1, y=y, up=up, act=act, down=down, h2=h2, codes=codes, s=s)


def norm_case(**kw):
    base = dict(routes=None, post_norm="none", pre_norm="rms", post_weight=None, pre_weight=None, gate=None, scale=None,
                shift=None, mod_index=None, residual_scale=1.0, eps=1e-6)
    return {**base, **kw}


def expert_rows(B, x, wq, ws, grp, off, rows):
    """The grouped layer from its codes in 64 bits, and its tolerance."""
    q, qs = B.convrot_rotate_quant_ex(x, grp)
    owner = torch.searchsorted(off[1:].contiguous(), torch.arange(rows.numel(), device=DEV, dtype=torch.int32), right=True)
    out = torch.stack([wq[e].double() @ q[m].double() for e, m in zip(owner.tolist(), rows.tolist())])
    ws = ws if ws.dim() == 2 else ws[:, None]
    want = out * qs.double()[rows.long()][:, None] * ws.double()[owner]
    return want, (torch.finfo(x.dtype).eps / 2 + 4 * 2.0 ** -24) * want.abs() + 1e-7


@pytest.mark.parametrize("io,M,K,F,E,top,group", [("bf16", 70, 512, 384, 6, 2, 128), ("fp16", 300, 1280, 256, 9, 3, 256),
                                                  ("bf16", 1, 768, 512, 4, 2, 128), ("fp16", 16, 512, 768, 8, 4, 256)])
def test_block(B, io, M, K, F, E, top, group):
    g, dt, w = model(io, K, F, E, group, M + K)
    h = torch.randn(M, K, generator=g, device=DEV)
    h[:, ::K // 4] *= 15
    h = h.to(dt)
    index = (torch.arange(M, device=DEV) * 3 // M).to(torch.int32)
    r = route(g, M, E, top)
    off, rows, pos, weight = r
    got = block(B, w, h, index, r)
    gate, scale, shift = w["mod"][:, :K], w["mod"][:, K:2 * K], w["mod"][:, 2 * K:]

    close(got["x"], ref_out(norm_case(pre_weight=w["norm1"]), h), dt, "norm before")
    want, tol = lora_reference(B, dict(x=got["x"], wq=w["proj"], w_scale=w["proj_s"], bias=None, lora_a=w["a"],
                                       lora_b=w["b"], lora_scale=w["s"], offsets=w["off"], index=index, max_rank=24), group)
    assert ((got["attn"].double() - want).abs() <= tol * 1.01).all()
    c = norm_case(h=h, u=got["attn"], post_norm="rms", post_weight=w["norm2"], gate=gate, scale=scale, shift=shift,
                  mod_index=index, pre_norm="layer")
    close(got["h1"], ref_h(c), dt, "stream after the projection")
    close(got["y"], ref_out(c, got["h1"]), dt, "norm between")
    want, tol = expert_rows(B, got["y"], w["up"], w["up_s"], group, off, rows)
    assert ((got["up"].double() - want).abs() <= tol * 1.01).all()
    want, tol = expert_rows(B, got["act"], w["down"], w["down_s"], group, off, torch.arange(M * top, device=DEV))
    assert ((got["down"].double() - want).abs() <= tol * 1.01).all()
    c = norm_case(h=got["h1"], u=got["down"], routes=(pos, weight), pre_weight=w["norm3"])
    close(got["h2"], ref_h(c), dt, "stream after the experts")
    # the codes are the next layer's input: its product from them, and from the norm's 16-bit values
    y = B.convrot_gemm_dequant_ex(got["codes"], got["s"], w["proj"], w["proj_s"], out_dtype=dt)
    _, z = B.convrot_block_norm(got["h2"], pre_weight=w["norm3"])
    y2 = B.convrot_linear_ex(z, w["proj"], w["proj_s"], group)
    assert (y.double() - y2.double()).norm() <= 0.02 * y2.double().norm()
    # the whole block again, and captured
    again = block(B, w, h, index, r)
    assert all(torch.equal(again[k], v) for k, v in got.items())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block(B, w, h, index, r)
    for k in range(3):
        h.mul_(0.9)
        o, rw, p, wt = route(g, M, E, top)
        for a, b in zip(r, (o, rw, p, wt)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        now = block(B, w, h, index, r)
        assert all(torch.equal(held[n], v) for n, v in now.items())
