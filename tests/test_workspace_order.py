"""A workspace for the most rows serves fewer: its size never falls with the rows."""
import random

import pytest

import tcgen05_tmem_bf16_gb300 as gbf

WIDTHS = (8, 64, 256, 320, 584, 1000, 1024, 2048, 2232, 4096, 8192)
HIDDEN = (8, 136, 544, 1408, 2728, 4096, 5632, 14336, 28672)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tcgen05_tmem_bf16_gb300 import build
    build.build()
    return gbf.load()


def rows(seed):
    """Both sides of the tiles' and paths' edges, and others."""
    edges = [e + d for e in (16, 32, 64, 128, 256, 512, 1024, 1536, 2048, 4096, 8192, 65536) for d in (-1, 0, 1)]
    rng = random.Random(seed)
    return sorted({0, 1, 2, 2 ** 18 + 1, 2 ** 20, *edges, *(int(2 ** rng.uniform(0, 17)) for _ in range(60))})


@pytest.mark.parametrize("D", WIDTHS)
def test_mlp_grad(D):
    for F in HIDDEN:
        sizes = [gbf.gbf_workspace_size("mlp_grad", M, D, F, True) for M in rows(D + F)]
        assert sizes[0] == 0 and all(a <= b for a, b in zip(sizes, sizes[1:])), (D, F)
