"""Test hooks of the block-scaled products: the choice of kernel, and waits that expire with no GPU fault. A hook makes one role of a
kernel give up its waits from one of its blocks on, while the others run into a short limit. The call comes back and says so,
the loads under way have landed before its CTAs end, and the next call is right."""
import threading
import time

import pytest
import torch

from test_gpu_fp8_block import check, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"

LOADS, SECOND_LOADS, MMA, SCALES, SUMS, PARTS = 1, 2, 3, 4, 5, 6


@pytest.fixture
def hooks(cuda_lib):
    cuda_lib.pqe_set_wait_limit(2000)
    yield cuda_lib
    cuda_lib.pqe_test_set_matmul_kernel(0, 0)
    cuda_lib.pqe_test_set_matmul_expiry(0, 0)
    cuda_lib.pqe_set_wait_limit(0)


def expires(pqe, kernel, who, block, sizes):
    """Three calls whose waits expire, each followed by one that is right."""
    a = inputs(*sizes, 3)
    out = torch.empty(sizes[:2], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pqe.pqe_test_set_matmul_kernel(*kernel)
    for _ in range(3):
        pqe.pqe_test_set_matmul_expiry(who, block)
        torch.cuda.synchronize()
        t = time.perf_counter()
        pqe.fp8_block_matmul(*a, out, status)
        torch.cuda.synchronize()
        assert time.perf_counter() - t < 10
        assert status.item() == pqe.PQE_STATUS_TIMEOUT
        pqe.pqe_test_set_matmul_expiry(0, 0)
        status.zero_()
        out.fill_(float("nan"))
        pqe.pqe_set_wait_limit(0)
        pqe.fp8_block_matmul(*a, out, status)
        check(out, *a)
        assert status.item() == 0
        pqe.pqe_set_wait_limit(2000)


@pytest.mark.parametrize("who", [LOADS, SECOND_LOADS, MMA, SCALES, SUMS])
@pytest.mark.parametrize("kernel", [(128, 128), (256, 128), (256, 256)], ids=lambda k: f"{k[0]}-{k[1]}")
def test_many_rows(hooks, kernel, who):
    """From the first block on, inside the ring's first round, later, and at the last block of a tile."""
    if who == SECOND_LOADS and kernel[0] == 128:
        pytest.skip("one CTA a tile")
    for block in (0, 2, 7, 15):
        expires(hooks, kernel, who, block, (300, 700, 2048))


@pytest.mark.parametrize("who", [LOADS, SECOND_LOADS, MMA, SCALES, SUMS])
def test_many_rows_in_a_later_tile(hooks, who):
    """1413 tiles of four blocks on 76 pairs."""
    expires(hooks, (256, 128), who, 30, (2050, 20000, 512))


@pytest.mark.parametrize("who", [LOADS, MMA, SUMS])
@pytest.mark.parametrize("kernel", [(16, 0), (16, 1), (16, 2), (32, 0), (32, 1), (32, 2), (32, 3)], ids=lambda k: f"{k[0]}-{k[1]}")
def test_few_rows(hooks, kernel, who):
    """From a CTA's first block on, inside the ring's first round, and (33 blocks of K, shared by up to eight) at its last or one near it."""
    for block in (0, 2, max(3, (33 >> kernel[1]) - 1)):
        expires(hooks, kernel, who, block, (60, 700, 4224))


@pytest.mark.parametrize("who,block", [(LOADS, 40), (MMA, 41), (SUMS, 42)])
def test_few_rows_in_a_later_tile(hooks, who, block):
    """3282 tiles of four blocks on 304 CTAs: ten or eleven each."""
    expires(hooks, (32, 0), who, block, (33 * 5, 70000, 512))


@pytest.mark.parametrize("kernel", [(16, 1), (16, 2), (32, 1), (32, 2), (32, 3)], ids=lambda k: f"{k[0]}-{k[1]}")
def test_parts_of_a_cluster(hooks, kernel):
    """The wait for the parts gives up in all CTAs of a cluster, in all but the first, and in the last alone."""
    for first in {0, 1, (1 << kernel[1]) - 1}:
        expires(hooks, kernel, PARTS, first, (60, 700, 4224))


@pytest.mark.parametrize("kernel", [(128, 128), (256, 128), (256, 256)], ids=lambda k: f"{k[0]}-{k[1]}")
def test_scales_of_many_blocks(hooks, kernel):
    """Several tiles a CTA, 64 blocks each, whose scales differ by up to 2^24: every slot of scales is used anew many times. A scale
    of another block would show in the bound, one that came late from run to run."""
    a = inputs(2300, 5000, 8192, 6)
    outs = [torch.full((2300, 5000), float("nan"), device=DEV) for _ in range(4)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    hooks.pqe_set_wait_limit(0)
    hooks.pqe_test_set_matmul_kernel(*kernel)
    for o in outs:
        hooks.fp8_block_matmul(*a, o, status)
    check(outs[0], *a)
    assert all(torch.equal(o, outs[0]) for o in outs) and status.item() == 0


def test_nobody_gives_up(hooks):
    """The hook at a block that no CTA reaches, or for a role that the kernel does not have, changes nothing."""
    a = inputs(300, 700, 2048, 4)
    out = torch.empty((300, 700), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    hooks.pqe_set_wait_limit(0)
    for kernel, who, block in (((256, 256), LOADS, 16), ((256, 128), MMA, 16), ((128, 128), SECOND_LOADS, 0)):
        hooks.pqe_test_set_matmul_kernel(*kernel)
        hooks.pqe_test_set_matmul_expiry(who, block)
        out.fill_(float("nan"))
        hooks.fp8_block_matmul(*a, out, status)
        check(out, *a)
    assert status.item() == 0


def test_kernel_hook_set_while_calls_are_made(cuda_lib):
    """A call sees one choice or another, never the tile of one with the split of the other, which no kernel takes."""
    a = inputs(40, 300, 1024, 5)
    out = torch.empty((40, 300), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    done = threading.Event()

    def turn():
        while not done.is_set():
            for kernel in ((32, 3), (256, 256), (16, 0), (128, 128), (32, 0), (256, 128)):
                cuda_lib.pqe_test_set_matmul_kernel(*kernel)

    t = threading.Thread(target=turn)
    t.start()
    try:
        for _ in range(200):
            out.fill_(float("nan"))
            for _ in range(20):
                cuda_lib.fp8_block_matmul(*a, out, status)
            check(out, *a)
    finally:
        done.set()
        t.join()
        cuda_lib.pqe_test_set_matmul_kernel(0, 0)
    assert status.item() == 0


def test_hook_refuses(cuda_lib):
    for bad in ((-1, 0), (7, 0), (1, -1)):
        with pytest.raises(cuda_lib.PqeError):
            cuda_lib.pqe_test_set_matmul_expiry(*bad)
