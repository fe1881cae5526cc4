"""Which kernel the gated block that is trained takes, at the sizes by which the tests on the
GPU run each of its forms: a changed estimate must not silently leave one untested."""
import pytest

import tcgen05_tmem_bf16_gb300 as gbf

PAIRS = 76
# forward: CTA pairs, units of one and of two row tiles, two rounds and more; 2056 columns of
# K are more than a ring; more than 8 units of rows make two groups of the raster
ROUNDS = [(513, 2056, 8200, "pair_1tile"), (2500, 1544, 2056, "pair_1tile"), (4500, 2056, 1032, "pair_1tile"),
          (1700, 1032, 7176, "pair_2tiles"), (2500, 2056, 5128, "pair_2tiles"), (4610, 1032, 2568, "pair_2tiles")]
# the gradient's dh
GRAD_ROUNDS = [(1300, 136, 8200, "pair_1tile"), (4610, 136, 2056, "pair_1tile"), (2500, 136, 8200, "pair_2tiles"),
               (4610, 136, 4104, "pair_2tiles")]


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tcgen05_tmem_bf16_gb300 import build
    build.build()
    return gbf.load()


@pytest.mark.parametrize("M,D,F,path", ROUNDS)
def test_forward(M, D, F, path):
    got, units = gbf.gbf_debug_mlp_path(M, D, F)
    assert got == path and units > 2 * PAIRS


@pytest.mark.parametrize("M,D,F,path", GRAD_ROUNDS)
def test_gradient(M, D, F, path):
    got, units = gbf.gbf_debug_mlp_path(M, D, F, True)
    assert got == path and units > 2 * PAIRS


@pytest.mark.parametrize("sizes,path", [((16, 264, 520), "swap_splitk"), ((1300, 72, 4104), "persistent"),
                                        ((513, 136, 1032), "pair_1tile"), ((1800, 1032, 4104), "pair_2tiles")])
def test_forward_of_the_tests_with_nan(sizes, path):
    from test_mlp_train_nan_gpu import FORWARD
    assert sizes in FORWARD and gbf.gbf_debug_mlp_path(*sizes)[0] == path


@pytest.mark.parametrize("sizes", [(0, 64, 64), (4, 12, 64), (4, 64, 0), (-1, 64, 64), (2 ** 24 + 1, 64, 64)])
def test_refused(sizes):
    assert gbf.gbf_debug_mlp_path(*sizes) == ("rejected", 0) == gbf.gbf_debug_mlp_path(*sizes, True)
