"""convrot_linear_lora: the adapters' first product keeps more bits than the io type has.

The result is compared with the formula in 64 bits.  What may lie between them, apart from the
rounding of the output and the fp32 sums (as in test_linear_lora): token by token t is an fp32
value, 2^-24 of it; in a list it is two parts of the io type, each off by half a step of what it
stands for, 2^-16 of t in bf16 and 2^-22 in fp16, there also 2^-39 of the largest t of the
token (the parts of a scaled t between 2^14 and 2^15, and half the smallest step, 2^-25).
One rounding of t to the io type would be off by 2^-8 and 2^-11, and out of fp16's range.
"""
import pytest
import torch

from tests.test_linear_lora import DEV, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from w8a8_rotated_int8_convrot_amd import binding
    binding.lib()
    return binding


def want_and_tol(B, p, group):
    x, dt = p["x"], p["x"].dtype
    M, K = x.shape
    q, qs = B.convrot_rotate_quant_ex(x, group)
    prod = (q.double() @ p["wq"].double().t()) * qs.double()[:, None] * p["w_scale"].double()
    bias = 0.0 if p["bias"] is None else p["bias"].double()
    want, mag, lost = prod + bias, prod.abs() + abs(bias), torch.zeros_like(prod)
    off = p["offsets"].tolist()
    by_token = M <= 16           # and some larger batches, whose bound is the list's here
    for a in range(len(off) - 1):
        at = torch.nonzero(p["index"] == a).flatten()
        lo, hi = off[a], off[a + 1]
        if not len(at) or hi == lo:
            continue
        s, wa, wb = p["lora_scale"][a].double(), p["lora_a"][lo:hi].double(), p["lora_b"][lo:hi].double()
        t = s * (x[at].double() @ wa.t())
        held = 2.0 ** -24 * t.abs()
        if not by_token:
            held = 2.0 ** -16 * t.abs() if dt == torch.bfloat16 else 2.0 ** -22 * t.abs() + 2.0 ** -39 * t.abs().amax(1, True)
        held += (K / 4 + 20) * 2.0 ** -24 * s * (x[at].double().abs() @ wa.abs().t())     # the fp32 sum over K
        want[at] += t @ wb
        # the fp32 sum over the ranks, two products each
        lost[at] = held @ wb.abs() + (2 * (hi - lo) + 4) * 2.0 ** -24 * (t.abs() @ wb.abs())
        mag[at] += (t @ wb).abs()
    tol = torch.finfo(dt).eps / 2 * want.abs() + 1.02 * lost + 5 * 2.0 ** -24 * mag
    return want, tol * 1.01 + (2.0 ** -24 if dt == torch.float16 else 0.0)


def close(B, p, group):
    want, tol = want_and_tol(B, p, group)
    got = B.convrot_linear_lora(**p, group=group).double()
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= tol).all()


# token by token and as a list, in every tile the call chooses from; K is short, so that the fp32 sums' bound is
# far below the roundings'
SHAPES = [(5, 256, 130, [40, 64], 1), (16, 256, 200, [16] * 16, 1), (90, 256, 72, [64, 33, 5, 8, 16, 40] * 3, 7),
          (37, 256, 5244, [8, 40, 64, 3, 16, 20] * 3, 3), (60, 128, 9000, [8, 40, 64, 3, 16, 20] * 4, 5),
          (97, 128, 15790, [8, 40, 64, 3, 16, 20] * 3, 9), (97, 128, 9000, [8, 40, 64, 3, 16, 20], 9),
          (40, 256, 136, [64, 33], 9), (100, 384, 2000, [64, 8], 30),
          (85, 256, 3132, [48, 64], 20), (120, 256, 8200, [48, 64], 50), (226, 128, 20434, [33, 64], 60),
          (300, 256, 520, [64, 40, 128], 11), (1000, 256, 2600, [64, 40, 32], 300), (559, 256, 13260, [40, 64], 100),
          (1999, 256, 4095, [40] * 9, 50), (2999, 128, 4090, [64, 100], 1000), (4700, 256, 3000, [64] * 5, 900),
          (4700, 640, 3001, [64] * 5, 900), (4333, 384, 8200, [24, 70, 100], 700)]


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N,ranks,run", SHAPES)
def test_more_bits_than_the_io_type(B, M, K, N, ranks, run, io):
    p = problem(M, K, N, io, ranks, False, False, M + N, run)
    p["w_scale"] *= 1e-3               # the layer's own part, and with it the output's steps, small
    close(B, p, 128)


@pytest.mark.parametrize("M,K,N,ranks,run", SHAPES)
def test_first_products_outside_fp16(B, M, K, N, ranks, run):
    """t of some millions, and of some 1e-8: the formula's fp32 holds them, fp16 does not."""
    p = problem(M, K, N, "fp16", ranks, True, True, M + N, run)
    high = dict(p, lora_a=(p["lora_a"].float() * 16384).to(torch.float16), lora_scale=p["lora_scale"] * 16,
                lora_b=(p["lora_b"].float() * 2.0 ** -14).to(torch.float16))
    t = high["x"].double() @ high["lora_a"].double().t() * 8
    assert t.abs().max() > 1e6
    close(B, high, 128)
    low = dict(p, lora_scale=p["lora_scale"] * 2.0 ** -33, lora_b=(p["lora_b"].float() * 4096).to(torch.float16),
               w_scale=p["w_scale"] * 1e-9, bias=None)
    close(B, low, 128)


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N", [(40, 72), (300, 520), (1999, 4095), (2999, 4090), (4700, 3001)])
def test_the_second_parts_leave_infinities_alone(B, M, N, io):
    """Infinite weights of B give the infinity of t's sign in their column, NaN gives NaN, and the
    other columns keep their bytes."""
    p = problem(M, 384, N, io, [16, 40], False, False, M, 5, none=0.0)
    off = p["offsets"].tolist()
    one = dict(p, lora_b=p["lora_b"].clone())
    one["lora_b"][off[0] + 3, 7] = one["lora_b"][off[1] + 33, 7] = float("-inf")
    one["lora_b"][off[0] + 1, 9] = one["lora_b"][off[1] + 35, 9] = float("nan")
    got, plain = B.convrot_linear_lora(**one, group=128), B.convrot_linear_lora(**p, group=128)
    rest = torch.ones(N, dtype=torch.bool, device=DEV)
    rest[[7, 9]] = False
    assert torch.equal(got[:, rest], plain[:, rest])
    assert got[:, 9].isnan().all()
    row = torch.where(p["index"] == 0, off[0] + 3, off[1] + 33).long()
    t = (p["lora_a"][row].double() * p["x"].double()).sum(1)
    sure = t.abs() > 1e-3
    assert torch.equal(got[sure, 7].double(), torch.where(t[sure] > 0, float("-inf"), float("inf")))


@pytest.mark.parametrize("io", ["bf16", "fp16"])
@pytest.mark.parametrize("M,ranks", [(7, [8, 16]), (100, [8] * 6), (100, [8, 16]), (300, [8, 16])])
def test_tokens_without_an_adapter_keep_the_sign_of_a_zero(B, M, ranks, io):
    """A scale product that underflows to zero and a bias of -0 give zeros of both signs, and a token
    without an adapter, or with one of no rows, gets the layer's own."""
    p = problem(M, 256, 72, io, ranks + [0], False, True, M, 1, none=0.5)
    p["w_scale"] *= 1e-37
    p["x"] *= 1e-6
    p["bias"] = torch.full_like(p["bias"], -0.0)
    got = B.convrot_linear_lora(**p, group=128)
    plain = B.convrot_linear_ex(p["x"], p["wq"], p["w_scale"], 128, bias=p["bias"])
    none = (p["index"] < 0) | (p["index"] >= len(ranks))
    zeros = plain[none]
    assert (zeros == 0).all() and torch.signbit(zeros).any() and not torch.signbit(zeros).all()
    assert torch.equal(got[none].view(torch.int16), zeros.view(torch.int16))


@pytest.mark.parametrize("M,N,ranks", [(12, 1030, [16] * 12), (100, 2048, [64] * 14), (700, 4096, [64, 40]),
                                       (2999, 4090, [64, 100]), (4700, 3001, [64] * 5)])
def test_two_streams_and_two_graphs(B, M, N, ranks):
    """t lies in the call's own workspace: two calls at once, and two graphs replayed in turn with
    eager calls between them, give what each gives alone."""
    ps = [problem(M, 512, N, "fp16", ranks, False, True, s, 50) for s in (1, 2)]
    want = [B.convrot_linear_lora(**p, group=128) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    outs = []
    for p, s in zip(ps, streams):
        with torch.cuda.stream(s):
            outs.append(B.convrot_linear_lora(**p, group=128))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs, outs = [], []
    for p in ps:
        outs.append(torch.empty_like(want[0]))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            B.convrot_linear_lora(**p, group=128, out=outs[-1])
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.fill_(9)
            g.replay()
        assert torch.equal(B.convrot_linear_lora(**ps[0], group=128), want[0])
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
