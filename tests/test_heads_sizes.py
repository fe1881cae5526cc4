"""Workspace sizes of the linear cross entropy for sizes that its entry points
refuse: none, and no crash of the process that asks (each in one of its own).
No GPU needed."""
import subprocess
import sys

import pytest

import tcgen05_tmem_bf16_gb300 as gbf

SHAPE = 3
P = 0x10000  # an address that is never followed


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tcgen05_tmem_bf16_gb300 import build
    build.build()
    return gbf.load()


@pytest.mark.parametrize("op", ["linear_ce", "linear_ce_grad"])
@pytest.mark.parametrize("sizes", [
    (4, 32000, 0), (0, 32000, 0), (256, 2000, 0), (1, 1024, 0), (300, 1024, 0), (4, 0, 64), (300, 0, 64),
    (4, 10, 12), (4, 10, 4), (2 ** 24 + 1, 10, 16), (4, 2 ** 26 + 1, 16), (4, 10, 2 ** 20 + 8), (2 ** 24, 2 ** 26, 16),
    (2 ** 24, 10, 2 ** 20), (4, 2 ** 26, 2 ** 20), (2 ** 62, 2 ** 62, 2 ** 62)])
def test_no_workspace_for_refused_sizes(op, sizes):
    M, V, D = sizes
    ask = f"import tcgen05_tmem_bf16_gb300 as g; print(g.gbf_workspace_size({op!r}, {M}, {V}, {D}, True))"
    got = subprocess.run([sys.executable, "-c", ask], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and got.stdout.strip() == "0"
    ends = dict(M=M, V=V, D=D, workspace=P, workspace_bytes=1 << 62, stream=0, raise_on_error=False)
    if op == "linear_ce":
        assert gbf.linear_ce(P, P, P, P, P, None, **ends) == SHAPE
    else:
        assert gbf.linear_ce_grad(P, P, P, P, None, P, P, **ends) == SHAPE


@pytest.mark.parametrize("op", ["linear_ce", "linear_ce_grad"])
@pytest.mark.parametrize("sizes", [(0, 1, 8), (1, 1, 8), (128, 2 ** 26, 8), (129, 1000, 2 ** 20), (2 ** 24, 1000, 8)])
def test_a_workspace_for_the_others(op, sizes):
    assert gbf.gbf_workspace_size(op, *sizes, True) > 0
