"""A workspace sized for the largest batch serves every smaller one (CPU: sizes and the checks of the C ABI)."""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from moe_decode_tail_gb300 import build as cuda_build

FAKE = 0x7F0000000000
GB = 1 << 30

# fake device addresses: only where no GPU is visible, so that a missing check can never launch on them
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: host-only")


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return mt.lib()


def chunk(routes):
    return 1024 * (1 if routes <= 128 * 1024 else 4 if routes <= 512 * 1024 else 16)


ROUTES = sorted({n + d for n in (1, 1024, 4096, 33 * 1024, 131072, 135168, 262144, 524288, 540672, 1048576, 2097152)
                 for d in (-1, 0, 1, 8) if 0 <= n + d <= 1 << 21})


def test_sort_workspace_never_shrinks(lib):
    for E in (1, 7, 128, 1024):
        sizes = [lib.moe_tail_sort_workspace_bytes(n, 1, E) for n in ROUTES]
        assert sizes == sorted(sizes)
        # and holds a row of counts for each thread block of a sort
        assert all(size >= 4 * E * -(-n // chunk(n)) for n, size in zip(ROUTES, sizes))
    for K in (2, 8, 32):
        sizes = [lib.moe_tail_sort_workspace_bytes(n // K, K, 128) for n in ROUTES]
        assert sizes == sorted(sizes)


def test_product_workspace_never_shrinks(lib):
    rows = sorted({n + d for n in (1, 16, 32, 64, 256, 1024, 4096, 8192, 16384, 32768, 1 << 20, 1 << 22) for d in (-1, 0, 1)
                   if 0 <= n + d <= 1 << 22})
    for E in (1, 2, 16, 128, 1024):
        for D in (16, 4096):
            sizes = [lib.moe_tail_expert_product_workspace_bytes(n, E, 256, D) for n in rows]
            assert sizes == sorted(sizes) and sizes[0] > 0


@host_only
@pytest.mark.parametrize("most,fewer", [(131080, 131072), (131080, 40000), (524296, 524288), (1 << 21, 131072)])
def test_a_sort_workspace_of_a_larger_batch_is_accepted(lib, most, fewer):
    size = lib.moe_tail_sort_workspace_bytes(most, 1, 128)
    p = lambda i: FAKE + 64 * GB * i  # noqa: E731
    # as far as the first CUDA call
    assert lib.moe_tail_sort_routes(p(0), fewer, 1, 128, p(1), p(2), p(3), p(4), size, None) in (2, 3)
