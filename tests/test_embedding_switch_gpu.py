"""The table's gradient at the number of positions where it begins to sort them
(1025), for every kind of ids.  Inputs, reference and tolerances are those of
test_embedding_gpu.py."""
import pytest

import test_embedding_gpu as embedding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1023, 1024, 1025])
@pytest.mark.parametrize("V,D", [(1, 8), (1500, 1032), (300000, 64)])
@pytest.mark.parametrize("kind", ["random", "mixed", "same", "unknown"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_where_sorting_begins(cuda_lib, M, V, D, kind, accumulate):
    embedding.test_gradient(cuda_lib, M, V, D, kind, accumulate)
