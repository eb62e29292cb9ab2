"""The root-mean-square norm with and without residual and weight in each of its forms: one and two vectors a lane of a wave, one,
two and four of a block a row."""
import pytest

from test_gpu_rms import inputs, parity

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("C", [504, 1016, 1032, 2056, 4104])
def test_optional_inputs(C, dtype, residual, weight):
    parity(f"{C}", inputs(2, 13, C, dtype, residual, weight), dtype)
