"""Weights of the attention over a paged cache where their rounding, the running maximum and values that are not finite
show: against the fp64 oracle, with the bounds of attention_util but for the weights' term, which is said at each test."""
import pytest

from tests.test_gpu_attention import KINDS, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1.4e-45, 1e-39, 1.5e-38, 3e-38])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_scales_that_are_tiny(scale, dtype, kind):
    """Scales down to the least number of fp32: all keys count alike, in tiles, pieces and their join."""
    check(50, [150, 1, 40], [60, 70, 2500], 4, 2, 64, 16, kind, dtype, scale=scale)
    check(51, [40], [100], 2, 1, 256, 16, kind, dtype, scale=scale, causal=False)
