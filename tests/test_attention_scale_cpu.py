"""Refused scales of attention's scores, checked on the host."""
import pytest

from tests.test_attention_abi_cpu import attend
from tests.test_rows_abi_cpu import INVALID, refused


@pytest.mark.parametrize("scale", [2.0 ** 127 * (1 + 2.0 ** -23), -3e38, float("nan"), float("-inf")])
def test_scales_whose_powers_of_two_leave_float32(scale):
    refused(lambda: attend(scale=scale), INVALID, "scale")
