"""add_rms_norm against the 64-bit statement.

Bounds, with u = 2^-8 (bf16's unit roundoff): the fp32 work adds at most about
(H/512 + 20) * 2^-24 < 2^-17 relative, so sum_out and y_out lie within u * (1 + 2^-8) of the
exact values, scales within 2^-16 relative; a code's value times its scale lies within 2^-4 of
y (E4M3's unit roundoff) plus half its smallest step, 2^-10 scales, both with 2^-8 to spare for a
code that a scale's last bit moves."""
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


def _inputs(T, H, seed, big=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, H), generator=g, device=DEV) * big
    r = 4 * torch.randn((T, H), generator=g, device=DEV) * (1 + 20 * (torch.rand(H, generator=g, device=DEV) < 0.02)) * big
    w = 1 + 0.3 * torch.randn(H, generator=g, device=DEV)
    return x.bfloat16(), r.bfloat16(), w.bfloat16()


def _check_q(q, s, y, fmt_row):
    y = y.cpu()
    if fmt_row:
        want = y.abs().amax(-1) / 448
        want = torch.where(want == 0, 1.0, want)
        assert ((s.double().cpu() - want).abs() <= 2.0 ** -16 * want).all()
        scale = s.double().cpu()[:, None]
    else:
        b = y.unflatten(-1, (-1, 32)).abs().amax(-1)
        e = torch.where(b == 0, 0, torch.frexp(b).exponent - 1 - 8 + 127).clamp(0, 254)
        diff = (s.cpu().long() - e).abs()
        near = (torch.frexp(b).mantissa - 0.5).abs() < 2.0 ** -15  # amax at a power of two: either side of it
        near |= (torch.frexp(b).mantissa - 1.0).abs() < 2.0 ** -15
        assert (diff <= near).all()
        scale = ref.pow2(s.cpu().long() - 127).repeat_interleave(32, -1)
    got = q.view(torch.float8_e4m3fn).double().cpu() * scale
    sat = torch.where(y.abs() > 448 * scale, torch.sign(y) * 448 * scale, y)
    assert ((got - sat).abs() <= (1 + U) * (2.0 ** -4 * sat.abs() + 2.0 ** -10 * scale)).all()


@pytest.mark.parametrize("T,H", [(1, 32), (3, 64), (1, 2048), (64, 2048), (5, 2560), (33, 96), (2, 4096), (3, 4128), (7, 8192),
                                 (2, 16384), (1, 16352), (4099, 256), (300, 5120)])
@pytest.mark.parametrize("fmt", ["row", "mx"])
def test_all_outputs(cuda_lib, T, H, fmt):
    pqe = cuda_lib
    x, r, w = _inputs(T, H, T + H)
    res, y = (torch.empty((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.empty((T, H), dtype=torch.uint8, device=DEV)
    row = fmt == "row"
    s = torch.empty(T, dtype=torch.float32, device=DEV) if row else torch.empty((T, H // 32), dtype=torch.uint8, device=DEV)
    pqe.add_rms_norm(x, r, w, 1e-6, res, y, q, s, pqe.PQE_Q8_ROW if row else pqe.PQE_Q8_MX)
    h64, y64 = ref.norm(x, r, w, 1e-6)
    assert ((res.double() - h64).abs() <= U * (1 + U) * h64.abs()).all()
    assert ((y.double() - y64).abs() <= U * (1 + U) * y64.abs()).all()
    _check_q(q, s, y64, row)


def test_optional_inputs_and_outputs(cuda_lib):
    pqe = cuda_lib
    T, H = 9, 512
    x, r, w = _inputs(T, H, 4)
    full = [torch.empty((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    q, s = torch.empty((T, H), dtype=torch.uint8, device=DEV), torch.empty(T, dtype=torch.float32, device=DEV)
    pqe.add_rms_norm(x, r, w, 1e-5, full[0], full[1], q, s)
    for outs in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        a = torch.empty_like(full[0]) if outs[0] else None
        b = torch.empty_like(full[0]) if outs[1] else None
        c, d = (torch.empty_like(q), torch.empty_like(s)) if outs[2] else (None, None)
        pqe.add_rms_norm(x, r, w, 1e-5, a, b, c, d)
        for got, want in ((a, full[0]), (b, full[1]), (c, q), (d, s)):
            assert got is None or torch.equal(got, want)
    # no residual: the norm alone
    y = torch.empty_like(full[0])
    pqe.add_rms_norm(x, None, w, 1e-5, None, y)
    _, y64 = ref.norm(x, None, w, 1e-5)
    assert ((y.double() - y64).abs() <= U * (1 + U) * y64.abs()).all()


def test_strided_rows_and_residual_in_place(cuda_lib):
    pqe = cuda_lib
    T, H = 37, 256
    wide, r, w = _inputs(T, 2 * H + 64, 6)[0], *_inputs(T, H, 7)[1:]
    x = wide[:, 64:64 + H]
    h64, y64 = ref.norm(x, r, w, 1e-6)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    pqe.add_rms_norm(x, r, w, 1e-6, r, y)  # the residual's rows take the sum
    assert ((r.double() - h64).abs() <= U * (1 + U) * h64.abs()).all()
    assert ((y.double() - y64).abs() <= U * (1 + U) * y64.abs()).all()


@pytest.mark.parametrize("fmt", ["row", "mx"])
def test_special_rows(cuda_lib, fmt):
    """A zero row, a row with a NaN, with an infinity, rows of huge and tiny values."""
    pqe = cuda_lib
    T, H = 6, 128
    x, r, w = _inputs(T, H, 9)
    x[0], r[0] = 0, 0
    x[1, 5] = float("nan")
    x[2, 40] = float("inf")
    x[3] = 3e18
    x[4], r[4] = 1e-30, 0
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    q = torch.empty((T, H), dtype=torch.uint8, device=DEV)
    row = fmt == "row"
    s = torch.empty(T, dtype=torch.float32, device=DEV) if row else torch.empty((T, H // 32), dtype=torch.uint8, device=DEV)
    pqe.add_rms_norm(x, r, w, 1e-6, None, y, q, s, pqe.PQE_Q8_ROW if row else pqe.PQE_Q8_MX)
    _, y64 = ref.norm(x, r, w, 1e-6)
    ok = [0, 3, 4, 5]
    assert ((y[ok].double() - y64[ok]).abs() <= U * (1 + U) * y64[ok].abs()).all()
    _check_q(q[ok], s[ok], y64[ok], row)
    assert torch.isnan(y[1]).all() and torch.isnan(q[1].view(torch.float8_e4m3fn).float()).all()
    assert (torch.isnan(s[1]) if row else s[1] == 255).all()
    # the infinity itself becomes NaN, the rest of its row zero
    assert torch.isnan(y[2, 40]) and (y[2, :40] == 0).all()
    if row:
        assert torch.isnan(s[2])
    else:
        assert s[2].tolist() == [0, 255, 0, 0]


def test_row_scale_below_fp32(cuda_lib):
    """y so small that max|y| / 448 is 0 in fp32: scale 1 and codes of zero, no 0 / 0."""
    T, H = 3, 64
    x = torch.ones((T, H), dtype=torch.bfloat16, device=DEV)
    x[:, ::2] = 0
    w = torch.full((H,), 2.0 ** -133, dtype=torch.bfloat16, device=DEV)  # bf16's smallest
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    q = torch.full((T, H), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.empty(T, dtype=torch.float32, device=DEV)
    cuda_lib.add_rms_norm(x, None, w, 1e8, None, y, q, s)  # y = 1e-4 * 2^-133, under 448 * 2^-150
    assert (y == 0).all() and (s == 1).all() and (q & 0x7F == 0).all()


def test_stream_and_graph(cuda_lib):
    pqe = cuda_lib
    T, H = 8, 2048
    x, r, w = _inputs(T, H, 12)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pqe.add_rms_norm(x, r, w, 1e-6, None, y)
    x.copy_(_inputs(T, H, 13)[0])
    g.replay()
    torch.cuda.synchronize()
    _, y64 = ref.norm(x, r, w, 1e-6)
    assert ((y.double() - y64).abs() <= U * (1 + U) * y64.abs()).all()
