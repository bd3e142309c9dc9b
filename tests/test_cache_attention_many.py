"""convrot_cache_attention with more long sequences in a call than a grid has third coordinates: every
one has its rows written."""
import pytest
import torch

from tests import _cache as ref
from tests.test_cache_attention import DEV, B, filled  # noqa: F401


def test_operands_are_for_all_long_sequences_or_none(B):  # noqa: F811
    """97 tokens of 8 query heads on 1 a sequence, over the 768 rows and more than the CUs' number of
    tiles: operands of 128 tokens, 256 bytes each, for each sequence, as long as there are
    65535 at most; past that the workspace holds none (and no parts: there are tiles enough)."""
    f = B.convrot_cache_attention_workspace
    assert f(65535 * 97, 8, 1, 64, 65535, 128) >= 65535 * 128 * 256
    assert f(65536 * 97, 8, 1, 64, 65536, 128) == 0
    assert f(70000 * 97, 8, 1, 64, 70000, 128) == 0


@pytest.mark.gpu
def test_more_long_sequences_than_a_grid_has_slots(B):  # noqa: F811
    """Sequences of 25 tokens, 32 query heads of 64 on 1, that repeat three: all rows are written, each
    as its like among the first three."""
    n, tokens, H, D, page, seqs = 25, 25, 32, 64, 32, 65537
    g, pages, table, _, _ = filled(31, [(0, n)] * 3, 1, D, page)
    q = torch.randn(3, tokens, H, D, generator=g, device=DEV).to(torch.bfloat16)
    starts, offsets = torch.zeros(3, dtype=torch.int32, device=DEV), torch.arange(4, dtype=torch.int32, device=DEV) * tokens
    want, tol = ref.attention(q.flatten(0, 1), pages, page, 1, table, starts, offsets, D ** -0.5)
    like = torch.arange(seqs, device=DEV) % 3
    rows = q[like].flatten(0, 1)
    out = torch.full_like(rows, 55.0)
    B.convrot_cache_attention(rows, pages, table[like].contiguous(), torch.zeros(seqs, dtype=torch.int32, device=DEV),
                              torch.arange(seqs + 1, dtype=torch.int32, device=DEV) * tokens, 1, page, out=out)
    out = out.view(seqs, tokens, H, D)
    assert ((out[:3].flatten(0, 1).double() - want).abs() <= tol).all()
    for i in range(3):
        assert (out[i::3] == out[i]).all()
