"""convrot_cache_copy captured: the lists are the call's, what pages hold is the replay's."""
import pytest
import torch

from tests.test_kv_cache import DEV, B  # noqa: F401


@pytest.mark.gpu
def test_captured_copies_of_what_is_there(B):  # noqa: F811
    pairs = [(i, 700 + i) for i in range(300)] + [(5, 690)]       # two launches
    pages = torch.randint(0, 256, (2, 1024, 64), dtype=torch.uint8, device=DEV)
    B.convrot_cache_copy(pages, pairs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.convrot_cache_copy(pages, pairs)
    src, dst = torch.tensor(pairs, device=DEV).t()
    del pairs
    for _ in range(3):
        pages.random_(0, 256)
        want = pages.clone()
        want[:, dst] = pages[:, src]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pages, want)
        eager = torch.randint(0, 256, (2, 1024, 64), dtype=torch.uint8, device=DEV)
        B.convrot_cache_copy(eager, [(1, 2)])
        assert torch.equal(eager[:, 2], eager[:, 1])
