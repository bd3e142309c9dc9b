"""Workspace sizes of the operators around the layer: 0 for a size that the call refuses, so that
no product of sizes wraps round to a small number (host code only)."""
import pytest

BIG = 1 << 30


@pytest.fixture(scope="module")
def B():
    import os
    from w8a8_rotated_int8_convrot_amd import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    binding.lib()
    return binding


@pytest.mark.parametrize("M,K", [(BIG + 1, 128), (1 << 62, 1 << 17), ((1 << 63) - 1, 128), (4, 131072 + 128), (4, 1 << 62)])
def test_grouped(B, M, K):
    assert B.convrot_grouped_workspace(M, K) == 0


@pytest.mark.parametrize("M,K,N,rank", [(BIG + 1, 128, BIG, 8), (1 << 62, 128, 8, 8), (8, 1 << 60, 8, 8), (8, 128, BIG + 1, 8),
                                        (8, 128, 1 << 62, 8), (8, 128, 8, 513), (8, 128, 0, 8)])
def test_lora(B, M, K, N, rank):
    assert B.convrot_lora_workspace(M, K, N, rank) == 0


def test_the_largest_sizes_do_not_wrap(B):
    assert B.convrot_grouped_workspace(BIG, 131072) == BIG * 131072 + BIG * 4
    # codes, scales, 512 ranks' 16-bit and fp32 words a token
    assert B.convrot_lora_workspace(BIG, 131072, BIG, 512) == BIG * 131072 + BIG * 4 + BIG * 1024 + BIG * 2048
