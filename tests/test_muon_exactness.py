"""How exact the Newton-Schulz products are, type by type."""
import pytest

from test_muon import distance, exact, matrices


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(20, 30), (64, 512), (500, 40), (64, 8192), (3, 3000, 30), (70, 90), (300, 200)])
@pytest.mark.parametrize("ratio", [1e-8, 1e-12, 1e-16])
def test_a_norm_far_below_eps(tgs_gpu, shape, ratio):
    """X stays tiny and every step multiplies it by the first coefficient, near enough."""
    x = matrices(shape, seed=sum(shape)) * (1e-3 * ratio)
    got = tgs_gpu.newton_schulz(x.cuda(), eps=1e-3)
    assert distance(got, exact(x, eps=1e-3)) <= 2.0**-18
