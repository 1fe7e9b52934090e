"""The 8-bit product's waits: a warp gives up together (see test_warp_waits)."""
import pytest

from tests.test_warp_waits import test_a_warp_gives_up_together as gives_up_together


@pytest.mark.parametrize("name", ["mx8_gemm.cu"])
def test_a_warp_of_the_product_gives_up_together(name):
    gives_up_together(name)
