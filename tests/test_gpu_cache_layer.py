"""Attention over the cache between two layers, as a server runs it: the projection to queries, keys
and values, their rotary positions in its rows, the new tokens into the cache, the attention over
it and the projection back -- prompts, single tokens, a fork and a captured step, joint by joint
against the formulas in 64 bits (tests/_cache.py).

Tolerances at the joints as in test_rope, test_cache_attention and, for the layers, half a step
of the type and a few of fp32; the pages byte by byte."""
import pytest
import torch

from tests import _cache as ref
from tests.test_rope import check as check_rope

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def B():
    from w8a8_rotated_int8_convrot_amd import binding
    binding.lib()
    return binding


class Layer:
    def __init__(self, B, K, Hq, Hk, D, rot, page, io, seqs, tokens, window=0, layout="half", group=128):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(K + D + Hq)
        self.B, self.K, self.Hq, self.Hk, self.D, self.page, self.window, self.layout = B, K, Hq, Hk, D, page, window, layout
        self.dt = torch.bfloat16 if io == "bf16" else torch.float16
        self.group = group
        self.w_in, self.s_in = self.weight((Hq + 2 * Hk) * D, K)
        self.w_out, self.s_out = self.weight(K, Hq * D)
        self.freqs, self.factor = B.convrot_rope_frequencies(rot, 10000.0, "yarn", 4.0, 4096.0, device=DEV)
        cols = (tokens + page - 1) // page
        # every other page spare: a fork takes them
        self.pages = torch.full((2 * seqs * cols, B.convrot_cache_page_bytes(page, Hk, D)), 255, dtype=torch.uint8, device=DEV)
        order = torch.randperm(2 * seqs * cols, generator=self.g, device=DEV).to(torch.int32)
        self.table, self.spare = order[:seqs * cols].view(seqs, cols).contiguous(), order[seqs * cols:].tolist()

    def weight(self, n, k):
        q = (28 * torch.randn(n, k, generator=self.g, device=DEV)).round().clamp(-127, 127).to(torch.int8)
        return q, torch.full((n,), 1.5 / 28 / k ** 0.5, device=DEV)

    def rows(self, M):
        return torch.randn(M, self.K, generator=self.g, device=DEV).to(self.dt)

    def run(self, x, starts, offsets, positions):
        """The step; returns its joints (the projection's rows before the turn among them)."""
        B, D = self.B, self.D
        qkv = B.convrot_linear_ex(x, self.w_in, self.s_in, self.group)
        plain = qkv.clone()
        rows = qkv.view(x.shape[0], -1, D)
        q, k, v = rows.split((self.Hq, self.Hk, self.Hk), 1)
        B.convrot_rope(q, k, positions, self.freqs, scale=self.factor, layout=self.layout, q_out=q, k_out=k)
        B.convrot_cache_append(self.pages, self.table, starts, offsets, k, v, self.page)
        a = B.convrot_cache_attention(q, self.pages, self.table, starts, offsets, self.Hk, self.page, window=self.window)
        y = B.convrot_linear_ex(a.view(x.shape[0], -1), self.w_out, self.s_out, self.group)
        return dict(plain=plain, qkv=qkv, a=a, y=y)

    def step(self, starts, lens):
        """A step from eager arguments, with every joint checked."""
        M = sum(lens)
        t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        ends = [sum(lens[:i]) for i in range(len(lens) + 1)]
        positions = torch.cat([torch.arange(s, s + n, device=DEV) for s, n in zip(starts, lens)]).to(torch.int32)
        x, starts, offsets = self.rows(M), t(starts), t(ends)
        before = self.pages.cpu()
        self.check(before, x, starts, offsets, positions, self.run(x, starts, offsets, positions))

    def layer(self, x, w, s, got):
        codes, scales = self.B.convrot_rotate_quant_ex(x, self.group)
        want = (codes.double() @ w.double().t()) * scales.double()[:, None] * s.double()
        tol = torch.finfo(self.dt).eps / 2 * want.abs() + 4 * 2.0 ** -24 * want.abs() + 2.0 ** -25
        assert ((got.double() - want).abs() <= 1.01 * tol).all()

    def check(self, before, x, starts, offsets, positions, j):
        M, D, Hq, Hk = x.shape[0], self.D, self.Hq, self.Hk
        self.layer(x, self.w_in, self.s_in, j["plain"])
        plain, rows = j["plain"].view(M, -1, D), j["qkv"].view(M, -1, D)
        check_rope(rows[:, :Hq + Hk], plain[:, :Hq + Hk], positions, self.freqs, self.factor, self.layout)
        assert torch.equal(rows[:, Hq + Hk:], plain[:, Hq + Hk:])
        ref.write(before, self.page, Hk, D, self.table.cpu(), starts.cpu(), offsets.cpu(), rows[:, Hq:Hq + Hk].cpu(),
                  rows[:, Hq + Hk:].cpu())
        assert torch.equal(self.pages.cpu(), before), "pages"
        want, tol = ref.attention(rows[:, :Hq], self.pages, self.page, Hk, self.table, starts, offsets, D ** -0.5, True, self.window)
        assert ((j["a"].double() - want).abs() <= tol).all(), "attention"
        self.layer(j["a"].view(M, -1), self.w_out, self.s_out, j["y"])


@pytest.mark.parametrize("K,Hq,Hk,D,rot,page,io,window,layout", [
    (512, 8, 2, 128, 128, 64, "bf16", 0, "half"), (256, 6, 6, 64, 32, 32, "fp16", 40, "interleaved"),
    (1024, 4, 1, 256, 64, 128, "bf16", 0, "interleaved"), (512, 4, 2, 128, 64, 256, "fp16", 300, "half")])
def test_prompts_tokens_fork_and_graph(B, K, Hq, Hk, D, rot, page, io, window, layout):
    m = Layer(B, K, Hq, Hk, D, rot, page, io, 3, 1400, window, layout)
    m.step([0, 0, 0], [333, 70, 0])                        # two prompts, a sequence that has none yet
    m.step([333, 70, 0], [1, 1, 129])                      # tokens beside a prompt's first piece
    m.step([334, 71, 129], [5, 1, 900])                    # drafts, a token, the long rest
    # the third becomes a fork of the first: its full pages shared, the last one copied
    full, last = 339 // page, int(m.table[0, 339 // page])
    to = m.spare[0]
    B.convrot_cache_copy(m.pages, [(last, to)])
    m.table[2, :full] = m.table[0, :full]
    m.table[2, full] = to
    assert torch.equal(m.pages[to], m.pages[last])
    m.step([335, 72, 335], [1, 1, 1])                      # two drafts dropped again: written over
    m.step([336, 73, 336], [1, 1, 1])
    # a token's step captured, its arguments on the GPU moving on
    x, pos = m.rows(3), torch.tensor([337, 74, 337], dtype=torch.int32, device=DEV)
    starts, offsets = pos.clone(), torch.arange(4, dtype=torch.int32, device=DEV)
    held_pages = m.pages.clone()
    m.run(x, starts, offsets, pos)                         # the workspaces' first use
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = m.run(x, starts, offsets, pos)
    m.pages.copy_(held_pages)
    for _ in range(3):
        x.copy_(m.rows(3))
        before = m.pages.cpu()
        graph.replay()
        torch.cuda.synchronize()
        m.check(before, x, starts, offsets, pos, held)
        after, got = m.pages.clone(), {k: v.clone() for k, v in held.items()}
        now = m.run(x, starts, offsets, pos)               # the same rows over themselves
        assert torch.equal(after, m.pages) and all(torch.equal(got[k], v) for k, v in now.items())
        starts.add_(1)
        pos.add_(1)
