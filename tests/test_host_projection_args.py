"""Refusals of the block-scaled products and of sampling: bad arguments return PQE_ERR_INVALID_ARG before any launch. CPU only."""
import pytest
import torch

import paged_quantized_expert_gb300 as pqe

BAD = pqe.PQE_ERR_INVALID_ARG
A = 4096  # an aligned address that is never read


def _refused(fn, ok, i, v):
    assert fn(*(v if j == i else x for j, x in enumerate(ok))) == BAD


@pytest.mark.parametrize("i,v", [(0, None), (0, A + 8), (1, 120), (1, 132), (2, -1), (3, 0), (3, 8), (3, 120), (3, 32784), (4, None), (4, A + 8),
                                 (5, None), (5, A + 2)])
def test_quantize_arguments(i, v):
    _refused(pqe.load().fp8_block_quantize, [A, 128, 1, 128, A, A, None], i, v)


@pytest.mark.parametrize("i,v", [(0, None), (0, A + 2), (1, 0), (2, 0), (2, -4), (3, None), (4, None), (4, A + 1)])
def test_quantize_tiles_arguments(i, v):
    _refused(pqe.load().pqe_quantize_fp8_blocks, [A, 4, 4, A, A, None], i, v)


@pytest.mark.parametrize("i,v", [(1, 65535 * 128 + 1), (1, (1 << 31) - 1), (2, (1 << 31) - 127), (2, (1 << 31) - 1)])
def test_quantize_tiles_beyond_the_grid_or_an_index(i, v):
    _refused(pqe.load().pqe_quantize_fp8_blocks, [A, 4, 4, A, A, None], i, v)


@pytest.mark.parametrize("i,v", [(0, None), (0, A + 8), (1, 112), (1, 136), (2, None), (2, A + 2), (3, None), (3, A + 8), (4, None), (4, A + 1), (5, -1),
                                 (5, (1 << 28) + 1), (6, 0), (6, -3), (6, (1 << 22) + 1), (7, 0), (7, 8), (7, 130), (7, 32784), (8, None), (8, A + 2), (9, 63), (11, None),
                                 (11, A + 2)])
def test_matmul_arguments(i, v):
    _refused(pqe.load().fp8_block_matmul, [A, 128, A, A, A, 2, 64, 128, A, 64, 1, A, None], i, v)


@pytest.mark.parametrize("i,v", [(0, None), (0, A + 2), (2, 99), (3, -1), (4, 0), (4, 368641), (5, A + 2), (6, A + 1), (7, A + 2), (8, A + 3), (9, None),
                                 (9, A + 2), (10, None), (10, A + 1), (11, A + 2), (12, None), (12, A + 2)])
def test_sample_arguments(i, v):
    _refused(pqe.load().sample_tokens, [A, 1, 100, 2, 100, None, None, None, None, A, A, None, A, None], i, v)


def test_bf16_logits_may_start_at_any_element():
    # the same address is refused for fp32 and not for bf16, where the next argument is
    lib = pqe.load()
    ok = [A + 2, 0, 100, 2, 100, None, None, None, None, None, A, None, A, None]
    assert lib.sample_tokens(*ok) == BAD
    assert lib.sample_tokens(*[A + 1] + ok[1:9] + [A] + ok[10:]) == BAD


def test_without_work():
    lib = pqe.load()
    assert lib.fp8_block_quantize(None, 0, 0, 128, None, None, None) == 0
    assert lib.fp8_block_matmul(None, 0, None, None, None, 0, 64, 128, None, 0, 0, None, None) == 0
    assert lib.sample_tokens(None, 0, 0, 0, 100, None, None, None, None, None, None, None, None, None) == 0


def test_matmul_kernel_hook():
    lib = pqe.load()
    for tile, split in ((1, 0), (16, 3), (16, -1), (32, 4), (64, 0), (128, 256), (128, 0), (256, 0), (256, 64), (0, 1)):
        assert lib.pqe_test_set_matmul_kernel(tile, split) == BAD
    assert lib.pqe_test_set_matmul_kernel(0, 0) == 0


def test_norm_takes_the_format():
    ok = [A, 64, A, 64, A, 1e-6, 1, 64, A, A, A, A, 2, None]
    for i, v in ((11, None), (11, A + 2), (12, 3)):
        _refused(pqe.load().add_rms_norm, ok, i, v)


E4 = torch.float8_e4m3fn


def _z(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype)


def test_binding_refuses_tensors_that_do_not_fit():
    x, xs, w, ws = _z(3, 256, dtype=E4), _z(3, 2), _z(130, 256, dtype=E4), _z(2, 2)
    out, st = _z(3, 130), _z(1, dtype=torch.int32)
    bf = _z(3, 256, dtype=torch.bfloat16)
    for bad in ((x[:, :128], xs, w, ws, out, st), (x, xs[:2], w, ws, out, st), (x, xs, w, ws[:1], out, st), (x, xs, w, ws, out[:2], st),
                (x, xs.double(), w, ws, out, st), (x.float(), xs, w, ws, out, st), (x, xs, w, ws, out.half(), st), (x, xs, w, ws, out, _z(1)),
                (x, xs, w.T.contiguous().T, ws, out, st), (x, xs, w, ws, _z(130, 3).T, st), (_z(256, 3, dtype=E4).T, xs, w, ws, out, st),
                (x, xs, w, ws, out, st)):  # the last one fits, and lies on the CPU
        with pytest.raises(ValueError):
            pqe.fp8_block_matmul(*bad)
    for bad in ((bf.float(), x, xs), (bf, x[:2], xs), (bf, x, xs[:1]), (bf, bf, xs), (bf, x, xs)):
        with pytest.raises(ValueError):
            pqe.fp8_block_quantize(*bad)
    for bad in ((w.float().double(), w, ws), (w.float(), w[:3], ws), (w.float(), w, ws[:1]), (w.float(), w, ws)):
        with pytest.raises(ValueError):
            pqe.pqe_quantize_fp8_blocks(*bad)
    with pytest.raises(ValueError):
        pqe.add_rms_norm(bf, None, bf[0], 1e-6, None, None, x, xs[:2], pqe.PQE_Q8_B128)
    l, u, tok = _z(3, 50), _z(3), _z(3, dtype=torch.int32)
    for bad in ((l.half(), u, tok, st), (l, u[:2], tok, st), (l, u, tok[:2], st), (l, u, u, st), (l, u.double(), tok, st), (_z(50, 3).T, u, tok, st),
                (l, u, tok, u), (l, u, tok, st)):
        with pytest.raises(ValueError):
            pqe.sample_tokens(*bad)
    for kw in (dict(temperature=u[:1]), dict(top_k=u), dict(top_p=tok), dict(min_p=u.double()), dict(logprobs=u[:2])):
        with pytest.raises(ValueError):
            pqe.sample_tokens(l, u, tok, st, **kw)
