"""kv_paged_attention at the ends of its ranges: widest windows, longest caches, what a masked token or a
token of no weight may hold. Bounds as in test_gpu_kv_attention.py, whose cases and comparison are used; where one
is wider, its derivation stands at the test."""
import pytest
import torch

import attention_ref as ref
from test_gpu_kv_attention import DEV, U, Case, compare, floor

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=["few", "many"])
def kernel(request, cuda_lib):
    cuda_lib.pqe_test_set_attention_kernel({"few": 1, "many": 2}[request.param])
    yield request.param
    cuda_lib.pqe_test_set_attention_kernel(0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ms,lens", [([6, 300], [1, 200]), ([70, 3], [67, 0]), ([140], [129])])
def test_widest_window_and_more_queries_than_tokens(cuda_lib, ms, lens, d):
    """A window that stands for none, where the first queries' positions are below zero: they see nothing, the others all
    tokens up to their own."""
    c = Case(cuda_lib, ms, lens, 8, 2, d, 16, seed=d)
    c.check(window=2 ** 31 - 1)
    wide, wide_lse = c.run(window=2 ** 31 - 1)
    none, none_lse = c.run()
    assert torch.equal(wide, none) and torch.equal(wide_lse, none_lse)


def _repeated(pqe, length, m, seed=0):
    """A sequence of `length` tokens whose block table names three pages of 1024 tokens over and over: pages, table, rows."""
    n_kv, d, page = 1, 64, 1024
    g = torch.Generator(device=DEV).manual_seed(seed)
    mem, cache = pqe.alloc_kv_cache(3, page, n_kv, d)
    at = torch.arange(3 * page, device=DEV)
    ref.put(mem, at, *(torch.randn((3 * page, n_kv, d), generator=g, device=DEV).bfloat16() for _ in range(2)), page)
    table = (torch.arange(-(-length // page), device=DEV, dtype=torch.int32) % 3)[None].contiguous()
    q = torch.randn((m, 4, d), generator=g, device=DEV).bfloat16()
    i32 = dict(dtype=torch.int32, device=DEV)
    return mem, cache, table, q, torch.tensor([0, m], **i32), torch.tensor([length], **i32), torch.zeros(1, **i32)


def _run(pqe, cache, table, q, offsets, lens, status, **kw):
    m, n_q, d = q.shape
    out, lse = torch.empty_like(q), torch.empty((m, n_q), device=DEV)
    ws = torch.empty(pqe.kv_paged_attention_workspace_size(1, m, m, n_q, cache.n_kv, d), dtype=torch.uint8, device=DEV)
    pqe.kv_paged_attention(cache, q, offsets, lens, table, m, d ** -0.5, out, ws, status, lse=lse, **kw)
    return out, lse


@pytest.mark.parametrize("m", [1, 5, 90])
@pytest.mark.parametrize("length", [2 ** 30 - 17, 2 ** 30 + 16, 2 ** 30 + 70001, 2 ** 31 - 2 ** 16])
def test_more_than_2_30_tokens(cuda_lib, length, m):
    """The window's tokens of a sequence whose token numbers pass 2^30, up to the longest that a table may describe."""
    window, page = 5000, 1024
    mem, cache, table, q, offsets, lens, status = _repeated(cuda_lib, length, m)
    out, lse = _run(cuda_lib, cache, table, q, offsets, lens, status, window=window)
    first = length - (window + m - 1)
    at = torch.arange(first, length, device=DEV)
    kv = [ref.get(mem, at // page % 3 * page + at % page, page, 1, 64)]
    compare(out, lse, *ref.attend(q, [m], [length - first], kv, 64 ** -0.5, window=window), floor(kv))
    assert status.item() == 0


def test_every_one_of_more_than_2_30_tokens(cuda_lib, kernel):
    """All tokens of 349526 rounds over three pages: the result of one round. The sums' own rounding counts here: a share of the
    work adds up to 2^20 tokens in fp32, 16 at a time, with 2^-23 each (a sum may be cut off rather than rounded)."""
    if kernel == "many":
        pytest.skip("one query row: about a second on the kernel for many")
    rounds, page = 349526, 1024
    length = rounds * 3 * page
    assert length > 2 ** 30
    mem, cache, table, q, offsets, lens, status = _repeated(cuda_lib, length, 1)
    out, lse = _run(cuda_lib, cache, table, q, offsets, lens, status)
    kv = [ref.get(mem, torch.arange(3 * page, device=DEV), page, 1, 64)]
    o, a, l = ref.attend(q, [1], [3 * page], kv, 64 ** -0.5)
    off = (out.double() - o).abs() - (U * (1 + U) * o.abs() + (2.0 ** -9 + 2 * 2 ** 16 * 2.0 ** -23) * a)
    assert not (off > 0).any(), off.max().item()
    assert not ((lse.double() - l - torch.log(torch.tensor(float(rounds), dtype=torch.float64))).abs() > 2.0 ** -6).any()
    assert status.item() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [1, 4, 90])
@pytest.mark.parametrize("n", [150, 5000])
def test_nan_values_of_no_weight(cuda_lib, m, n, d):
    """A token whose V block is NaN and whose score lies so far below the others that its probability is 0 in any format:
    0 * NaN is NaN, on both kernels. Rows that do not see it are as without it."""
    c = Case(cuda_lib, [m, m], [n, 40 + m], 8, 2, d, 16, seed=n + m)
    bad = n - 1 - m // 2  # some of the queries come before it
    c.q[:, :, 0] = 32.0
    k, v = ref.get(c.mem, c.slots[0][bad:bad + 1], 16, 2, d)
    k[:, :, 0] = -2048.0  # a score of -65536 / sqrt(d)
    v[0, 1, 40] = float("nan")
    ref.put(c.mem, c.slots[0][bad:bad + 1], k.bfloat16(), v.bfloat16(), 16)
    out, lse = c.run()
    kv = c.kv()
    o, a, l = ref.attend(c.q, c.ms, c.lens, kv, c.scale)
    hit = torch.isnan(o)
    assert hit[m - 1 - m // 2:m, 4:, 32:64].all() and hit.sum() == (m // 2 + 1) * 4 * 32
    assert torch.equal(torch.isnan(out), hit) and not torch.isnan(lse).any()
    # scores within 2^10 for the tokens that count: their fp32 sums are off by 2^-13 at most, which moves a probability by less
    # than 2^-11 (its share in A)
    compare(out, lse, o, a, l, floor(kv))
