"""The layer for a few tokens at its limits: matrices next to 2^31 bytes, as shared experts
beside small routed ones, and every expert of 1024 chosen; against the 64-bit definition."""
import pytest
import torch

from test_gpu_few import BF, F32, Case, xm  # noqa: F401  (xm is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,hs,size", [("bf16", 16376, 2), ("f32", 8184, 4), ("mx8", 32736, 1)])
def test_matrices_next_to_the_limit(xm, kind, hs, size):  # noqa: F811
    d = 65536
    assert 2 ** 31 - 2 ** 23 < d * hs * size < 2 ** 31
    c = Case(xm, 3, d, 8, 2, 32, hs, dt=F32 if kind == "f32" else BF, mx8=kind == "mx8")
    c.splain = None
    torch.cuda.empty_cache()
    c.run().check(kind)


@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("T", [1, 64])
def test_every_one_of_1024_experts(xm, kind, T):  # noqa: F811
    Case(xm, T, 96, 1024, 1024, 32, 32, dt=F32 if kind == "f32" else BF, mx8=kind == "mx8", bias=True).run().check(kind)
