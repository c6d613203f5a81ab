"""The issue loops' bounded wait is given up, or not, by a whole warp: the self-test
has half a warp's lanes wait on a barrier whose phase is complete and the other half
on one that nothing arrives on, and reports in bit 1 of the error word whether any
lane left with another answer than the rest."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

TIMEOUT = 5
WAIT_TEST_CODE = 7


@pytest.mark.parametrize("limit_us", [50, 5_000])
def test_lanes_of_a_warp_give_up_together(gemm_mod, limit_us):
    lib = gemm_mod.lib
    gemm_mod.check_device_error()
    assert lib.gemm_selftest_wait_timeout(limit_us, None) == 0
    torch.cuda.synchronize()
    word = ctypes.c_uint32(0)
    assert lib.gemm_check_device_error(ctypes.byref(word)) == TIMEOUT
    assert (word.value >> 8) & 0xFF == WAIT_TEST_CODE
    assert not word.value & 2, "lanes of one warp disagreed about a wait"
    assert gemm_mod.check_device_error() == 0
