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


VOCABULARIES = (1, 10, 1000, 32000, 50001, 131072, 2 ** 21 + 3)


@pytest.mark.parametrize("D", (8, 64, 1000, 2056, 4096, 8192))
@pytest.mark.parametrize("grad", [False, True])
def test_linear_distill_and_linear_ce(D, grad):
    for V in VOCABULARIES:
        for K in (1, 20, 1024):
            sizes = [gbf.linear_distill_workspace_size(M, V, D, K, grad) for M in rows(V + K)]
            assert all(0 < a <= b for a, b in zip(sizes, sizes[1:])), (V, K)
        sizes = [gbf.gbf_workspace_size("linear_ce_grad" if grad else "linear_ce", M, V, D, True) for M in rows(V)]
        assert all(0 < a <= b for a, b in zip(sizes, sizes[1:])), V


@pytest.mark.parametrize("D", (8, 256, 1024, 1032, 2048, 4096, 8192, 2 ** 21))
def test_embedding_grad(D):
    many = sorted({*rows(D), 2432, 2433, 4864, 4865, 9728, 9729})
    sizes = [gbf.gbf_workspace_size("embedding_grad", M, 32000, D, True) for M in many]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
