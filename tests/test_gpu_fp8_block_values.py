"""Special values through the block quantisers of weights and of the residual norm: what is not a number or not finite stays in its
tile or block, and sizes at the ends of fp32 keep their codes."""
import pytest
import torch

import attention_ref as ref
from test_gpu_fp8_block import tiles

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4 = torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


def test_weights_that_are_not_finite(cuda_lib):
    """NaN: the tile's scale and codes are NaN. Infinity: the scale is, the infinity's own code is NaN (their quotient), all others 0."""
    rows, cols = 300, 400
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.randn((rows, cols), generator=g, device=DEV)
    clean = w.clone()
    w[5, 130] = NAN
    w[299, 399] = -NAN
    w[128, 0] = INF
    w[200, 100] = -INF
    w[10, 384], w[11, 385] = INF, NAN  # both: NaN
    q = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
    s = torch.empty((3, 4), device=DEV)
    cuda_lib.pqe_quantize_fp8_blocks(w, q, s)
    wq, ws = (t.to(DEV) for t in tiles(clean, 128))
    f = q.view(E4).float()
    bad = {(0, 1): NAN, (2, 3): NAN, (0, 3): NAN, (1, 0): INF}
    for i in range(3):
        for j in range(4):
            at = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
            if (i, j) not in bad:
                assert s[i, j] == ws[i, j] and torch.equal(q[at], wq.view(torch.uint8)[at])
            elif bad[i, j] == INF:
                assert s[i, j] == INF
                assert torch.equal(torch.isnan(f[at]), torch.isinf(w[at])) and (f[at][~torch.isinf(w[at])] == 0).all()
            else:
                assert torch.isnan(s[i, j]) and torch.isnan(f[at]).all()


@pytest.mark.parametrize("top", [3.4e38, 1e38, 2.0 ** 100, 2.0 ** -100, 2.0 ** -126, 1e-40, 2.0 ** -149])
def test_weights_at_the_ends_of_fp32(cuda_lib, top):
    """Bit for bit with IEEE divisions, subnormal scales and a scale that fp32 does not hold (1 then) among them."""
    g = torch.Generator().manual_seed(2)
    w = ((2 * torch.rand((130, 260), generator=g, dtype=torch.float64) - 1) * top).float()
    w[0, 0], w[129, 259] = top, -top
    q = torch.empty((130, 260), dtype=torch.uint8, device=DEV)
    s = torch.empty((2, 3), device=DEV)
    cuda_lib.pqe_quantize_fp8_blocks(w.to(DEV), q, s)
    wq, ws = tiles(w, 128)
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu(), wq.view(torch.uint8))


def norm(pqe, x, r, w):
    T, H = x.shape
    q = torch.empty((T, H), dtype=torch.uint8, device=DEV)
    s = torch.empty((T, -(-H // 128)), device=DEV)
    pqe.add_rms_norm(x, r, w, 1e-6, None, None, q, s, pqe.PQE_Q8_B128)
    return q.view(E4).float(), s


# (rows enough for the kernel with a warp a row, and few)
@pytest.mark.parametrize("T,H", [(3, 2208), (1300, 2208), (5, 416), (2000, 416), (2, 8224)])
def test_norm_of_values_that_are_not_finite(cuda_lib, T, H):
    """A NaN in x or the residual makes its whole row NaN; an infinity there the infinity's block, where 0 times it is NaN, the others
    are zeros with scale 1. A NaN or an infinity in the weight is its own block's, in every row
    (an infinity times a sum of exactly 0 is NaN too)."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x, r = (torch.randn((T, H), generator=g, device=DEV).bfloat16() for _ in range(2))
    w = (1 + 0.3 * torch.randn(H, generator=g, device=DEV)).bfloat16()
    clean, clean_s = norm(cuda_lib, x, r, w)
    x1, r1 = x.clone(), r.clone()
    x1[0, 200] = NAN
    r1[1, H - 1] = -INF
    f, s = norm(cuda_lib, x1, r1, w)
    last = (H - 1) // 128
    assert torch.isnan(s[0]).all() and torch.isnan(f[0]).all()
    assert torch.isnan(s[1, last]) and torch.isnan(f[1, 128 * last:]).all()
    assert (s[1, :last] == 1).all() and (f[1, :128 * last] == 0).all()
    assert torch.equal(s[2:], clean_s[2:]) and torch.equal(f[2:], clean[2:])
    w1 = w.clone()
    w1[130] = NAN
    w1[H - 2] = INF
    f, s = norm(cuda_lib, x, r, w1)
    assert torch.isnan(s[:, 1]).all() and torch.isnan(f[:, 128:256]).all()
    assert torch.isnan(f[:, H - 2]).all()
    zero = x[:, H - 2].float() + r[:, H - 2].float() == 0  # times infinity: NaN, as is its whole block then
    assert torch.isnan(s[zero, last]).all() and torch.isnan(f[zero, 128 * last:]).all()
    assert torch.isinf(s[~zero, last]).all() and (f[~zero, 128 * last:H - 2] == 0).all() and (f[~zero, H - 1] == 0).all()
    rest = torch.ones(H, dtype=torch.bool, device=DEV)
    rest[128:256] = rest[128 * last:] = False
    assert torch.equal(f[:, rest], clean[:, rest])


@pytest.mark.parametrize("T", [4, 1300])
@pytest.mark.parametrize("power", [120, 99, -99, -115])
def test_norm_of_weights_far_from_one(cuda_lib, T, power):
    """Block codes where amax is outside 2^-100 to 2^100 and where it is at these borders, by the bounds of other sizes: fp32 work
    under 2^-16 relative, a code within 2^-4 of y or half its smallest step."""
    H = 544
    g = torch.Generator(device=DEV).manual_seed(power + 200)
    x, r = (torch.randn((T, H), generator=g, device=DEV).bfloat16() for _ in range(2))
    w = ((1 + 0.3 * torch.randn(H, generator=g, device=DEV)) * 2.0 ** power).bfloat16()
    f, s = norm(cuda_lib, x, r, w)
    _, y = ref.norm(x, r, w, 1e-6)
    amax = torch.stack([b.abs().amax(1) for b in y.split(128, 1)], 1)
    assert ((s.double() - amax / 448).abs() <= 2.0 ** -16 * amax / 448).all()
    scale = s.double().repeat_interleave(128, 1)[:, :H]
    assert ((f.double() * scale - y).abs() <= (1 + 2.0 ** -8) * (2.0 ** -4 * y.abs() + 2.0 ** -10 * scale)).all()
