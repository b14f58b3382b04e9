"""Block-scaled products into rows that end inside 16 bytes and lie 16-byte aligned, as columns of a wider result or rows with room
behind them: what lies behind each row stays as it was."""
import pytest
import torch

from test_gpu_fp8_block import KERNELS, check, inputs, kernel  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(pqe, M, N, K, dtype, room):
    a = inputs(M, N, K, N)
    each = 8 if dtype is torch.bfloat16 else 4
    wide = -(-N // each) * each + room
    buf = torch.full((M + 1, wide), 7.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pqe.fp8_block_matmul(*a, buf[:M, :N], status)
    check(buf[:M, :N], *a)
    assert (buf[:M, N:] == 7).all() and (buf[M] == 7).all() and status.item() == 0


@pytest.mark.parametrize("kernel", KERNELS, indirect=True, ids=lambda k: f"{k[0]}-{k[1]}")
@pytest.mark.parametrize("N", [1, 3, 7, 9, 133, 255, 257, 318, 1003])
def test_every_kernel_and_rest(cuda_lib, kernel, N):  # noqa: F811
    for dtype in (torch.bfloat16, torch.float32):
        for room in (0, 16):
            run(cuda_lib, 150, N, 272, dtype, room)


@pytest.mark.parametrize("rest", range(8))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(383, 2672, 1040), (64, 20000, 512), (2050, 1280, 256)])
def test_every_rest_by_the_choice_of_kernel(cuda_lib, M, N, K, dtype, rest):
    run(cuda_lib, M, N + rest, K, dtype, 8)


def test_two_products_side_by_side(cuda_lib):
    """Columns of one result from two calls, the second first: neither touches the other's."""
    M, K = 700, 640
    a, b = inputs(M, 1283, K, 1), inputs(M, 400, K, 2)
    out = torch.full((M, 1688), float("nan"), dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cuda_lib.fp8_block_matmul(*b, out[:, 1283:1683], status)
    cuda_lib.fp8_block_matmul(*a, out[:, :1283], status)
    check(out[:, :1283], *a)
    check(out[:, 1283:1683], *b)
    assert status.item() == 0
