"""What the test hooks of the block-scaled products refuse. CPU only."""
import pytest

import paged_quantized_expert_gb300 as pqe


@pytest.mark.parametrize("who,block", [(-1, 0), (7, 0), (1 << 30, 0), (1, -1)])
def test_expiry_refuses(who, block):
    assert pqe.load().pqe_test_set_matmul_expiry(who, block) == pqe.PQE_ERR_INVALID_ARG


def test_expiry_takes_each_role():
    lib = pqe.load()
    for who in range(1, 7):
        assert lib.pqe_test_set_matmul_expiry(who, (1 << 31) - 1) == 0
    assert lib.pqe_test_set_matmul_expiry(0, 0) == 0
