"""Workspaces of the operators of a mixed batch by size alone: what serves a call serves every smaller one.  Each size is compared with
the largest of all smaller ones, over the borders where the kernels' plans change."""
import pytest


@pytest.fixture(scope="module")
def tq():
    import bit_quantized_matvec_amd as m

    return m


def grows(sizes):
    assert all(a > 0 for a in sizes)
    drops = [(i, a, b) for i, (a, b) in enumerate(zip(sizes, sizes[1:])) if b < a]
    assert not drops, drops[:5]


@pytest.mark.parametrize("n,rank,cols", [(1, 8, 8), (5, 64, 5120), (24, 32, 5120), (4, 64, 5120), (3, 16, 6144), (300, 128, 2048), (7, 256, 7168), (40, 72, 264)])
def test_adapter_workspaces_grow_with_tokens(tq, n, rank, cols):
    grows([tq.adapter_workspace_bytes(t, n, rank, cols) for t in range(1, 13_000)] + [tq.adapter_workspace_bytes(t, n, rank, cols) for t in (50_000, 2**20)])


@pytest.mark.parametrize("tokens", [1, 64, 65, 700, 2047, 2048, 9000])
def test_adapter_workspaces_grow_with_adapters_ranks_and_columns(tq, tokens):
    size = tq.adapter_workspace_bytes
    grows([size(tokens, n, 32, 5120) for n in range(1, 3000)])
    grows([size(tokens, 24, rank, 5120) for rank in range(8, 257, 8)])
    grows([size(tokens, 24, 64, cols) for cols in range(8, 20_000, 8)])


def test_an_adapter_workspace_serves_smaller_calls(tq):
    size, n = tq.adapter_workspace_bytes, [(t, a, r, c) for t in (1, 65, 1375, 1500, 2048, 7000) for a in (1, 24) for r in (8, 64, 72, 256) for c in (8, 1024, 5120)]
    for large in n:
        for small in n:
            if all(s <= b for s, b in zip(small, large)):
                assert size(*small) <= size(*large), (small, large)


def test_sample_workspaces_grow(tq):
    size = tq.sample_workspace_bytes
    borders = [b + i for b in (262_137, 262_144, 266_233, 266_240, 532_473, 532_480, 2**20 - 8) for i in range(-9, 9)]
    for rows in (1, 3, 1024, 5000):
        grows([size(rows, v) for v in sorted({*range(1, 2**20 + 1, 1013), *borders, 2**20})])
    for vocab in (1, 4089, 4090, 131_072, 262_144, 270_000, 540_000, 2**20):
        grows([size(rows, vocab) for rows in range(1, 3000)])
