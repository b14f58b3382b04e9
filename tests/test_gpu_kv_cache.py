"""kv_cache_write and kv_cache_read against the 64-bit statement: every byte of the
cache and every value read back is equal (a power-of-two scale makes v / X exact, so
the code is the only rounding and both sides define it)."""
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _rows(n, heads, d, seed, spread=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, heads, d), generator=g, device=DEV)
    if spread:  # magnitudes over bf16's range
        x = x * torch.exp2(torch.randint(-40, 40, (n, heads, d // 32, 1), generator=g, device=DEV).float()).expand(
            n, heads, d // 32, 32).reshape(n, heads, d)
    return x.bfloat16()


def _check(pqe, n, n_kv, d, page, slots, k, v, n_pages):
    mem, cache = pqe.alloc_kv_cache(n_pages, page, n_kv, d)
    mem.fill_(0x5A)  # what is not written stays
    want = mem.clone()
    status = _status()
    pqe.kv_cache_write(cache, k, v, slots, status)
    keep = slots >= 0
    ref.put(want, slots[keep], k[keep], v[keep], page)
    assert torch.equal(mem, want)
    ko = torch.full((n, n_kv, d), 7.0, dtype=torch.bfloat16, device=DEV)
    vo = ko.clone()
    pqe.kv_cache_read(cache, slots, ko, vo, status)
    kr, vr = ref.get(want, slots.clamp(min=0), page, n_kv, d)
    z = keep[:, None, None]
    for got, exp in ((ko, kr), (vo, vr)):
        exp = torch.where(z, exp, 0.0)
        assert torch.equal(torch.nan_to_num(got.double(), nan=123.0), torch.nan_to_num(exp, nan=123.0))
    assert status.item() == 0


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("n,n_kv,d", [(1, 1, 64), (1, 8, 128), (5, 3, 64), (17, 4, 128), (64, 4, 128), (333, 2, 64), (1000, 8, 128)])
@pytest.mark.parametrize("order", ["run", "offset", "scattered"])
def test_write_and_read_back(cuda_lib, page, n, n_kv, d, order):
    n_pages = -(-(n + 40) // page) + 2
    g = torch.Generator(device=DEV).manual_seed(n * 31 + page)
    if order == "scattered":
        slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:n]
    else:  # a prompt's tokens, from a place inside a page on, its pages in any order
        at = torch.arange(n, device=DEV) + (0 if order == "run" else 21)
        slots = torch.randperm(n_pages, generator=g, device=DEV)[at // page] * page + at % page
    if n > 4:
        slots[[0, n // 2]] = -1
    _check(cuda_lib, n, n_kv, d, page, slots, _rows(n, n_kv, d, n), _rows(n, n_kv, d, n + 1), n_pages)


def test_many_tokens(cuda_lib):
    n, n_kv, d, page = 20011, 4, 128, 64
    n_pages = n // page + 2
    slots = torch.arange(n, device=DEV) + 5
    _check(cuda_lib, n, n_kv, d, page, slots, _rows(n, n_kv, d, 1), _rows(n, n_kv, d, 2), n_pages)


def test_special_values(cuda_lib):
    """All-zero blocks, subnormal ones, ties between codes, the largest finite values, and blocks with NaN or infinities."""
    n, n_kv, d, page = 16, 1, 128, 16
    k = torch.zeros((n, n_kv, d), dtype=torch.bfloat16, device=DEV)
    tiny = torch.finfo(torch.bfloat16).smallest_normal
    k[1, 0, :32] = torch.tensor([tiny / 128 * i for i in range(32)])
    k[2, 0, :32] = tiny
    k[3, 0, :8] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0])
    k[4, 0, 32] = torch.finfo(torch.bfloat16).max
    k[5, 0, 33:36] = torch.tensor([1.0, float("nan"), 2.0])
    k[6, 0, 64] = float("inf")
    k[7, 0, 127] = float("-inf")
    k[7, 0, 0] = 3.0
    k[8, 0, :32] = -0.0
    _check(cuda_lib, n, n_kv, d, page, torch.arange(n, device=DEV), k, k.flip(0).contiguous(), 1)


@pytest.mark.parametrize("n", [1, 70])
def test_rows_inside_a_fused_projection(cuda_lib, n):
    n_kv, d, page = 2, 64, 32
    fused = _rows(n, 12, d, 3)  # 8 query heads, 2 of K, 2 of V
    _check(cuda_lib, n, n_kv, d, page, torch.arange(n, device=DEV) + 3, fused[:, 8:10], fused[:, 10:], 4)


def test_slots_beyond_the_cache(cuda_lib):
    pqe = cuda_lib
    n_kv, d, page, n_pages = 2, 64, 16, 3
    mem, cache = pqe.alloc_kv_cache(n_pages, page, n_kv, d)
    k = _rows(4, n_kv, d, 5)
    slots = torch.tensor([n_pages * page, 1 << 40, 7, (1 << 62) + 3], device=DEV)
    status = _status()
    pqe.kv_cache_write(cache, k, k, slots, status)
    assert status.item() == pqe.PQE_STATUS_BAD_PAGE
    want = torch.zeros_like(mem)
    ref.put(want, slots[2:3], k[2:3], k[2:3], page)
    assert torch.equal(mem, want)
    status.zero_()
    ko = torch.ones_like(k)
    pqe.kv_cache_read(cache, slots, ko, None, status)
    assert status.item() == pqe.PQE_STATUS_BAD_PAGE
    assert torch.equal(ko[[0, 1, 3]], torch.zeros_like(ko[:3])) and ko[2].abs().sum() > 0


def test_cache_beyond_32_bit_offsets(cuda_lib):
    pqe = cuda_lib
    n_kv, d, page = 8, 128, 64
    n_pages = (5 << 30) // pqe.pqe_kv_page_bytes(page, n_kv, d)
    mem = torch.empty(n_pages * pqe.pqe_kv_page_bytes(page, n_kv, d), dtype=torch.uint8, device=DEV)
    cache = pqe.make_kv_cache(mem, n_pages, page, n_kv, d)
    slots = torch.cat([torch.arange(40, device=DEV) + (n_pages - 1) * page, torch.arange(40, device=DEV)])
    k, v = _rows(80, n_kv, d, 8), _rows(80, n_kv, d, 9)
    status = _status()
    pqe.kv_cache_write(cache, k, v, slots, status)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    pqe.kv_cache_read(cache, slots, ko, vo, status)
    for got, x in ((ko, k), (vo, v)):
        assert torch.equal(got.double(), ref.values(*ref.mxfp4(x)))
    assert status.item() == 0


def test_other_stream_and_graph(cuda_lib):
    pqe = cuda_lib
    n_kv, d, page, n = 4, 128, 16, 33
    mem, cache = pqe.alloc_kv_cache(8, page, n_kv, d)
    k, v = _rows(n, n_kv, d, 11), _rows(n, n_kv, d, 12)
    slots, status = torch.arange(n, device=DEV) + 2, _status()
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pqe.kv_cache_write(cache, k, v, slots, status)
        pqe.kv_cache_read(cache, slots, ko, vo, status)
    torch.cuda.synchronize()
    assert torch.equal(ko.double(), ref.values(*ref.mxfp4(k)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pqe.kv_cache_write(cache, k, v, slots, status)
        pqe.kv_cache_read(cache, slots, ko, vo, status)
    k.copy_(_rows(n, n_kv, d, 13))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ko.double(), ref.values(*ref.mxfp4(k)))
    assert torch.equal(vo.double(), ref.values(*ref.mxfp4(v)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [16, 6400])
def test_two_tokens_of_one_slot(cuda_lib, n, d):
    """Two rows with the same slot among 16 of one block: that place holds either one's bytes, every other place its own
    token's, and the place that no row has keeps what it held."""
    n_kv, page = 8, 32
    slots = torch.arange(n, device=DEV)
    slots[9::16] = slots[4::16]  # place 9 of each block has no row, place 4 two
    k, v = _rows(n, n_kv, d, 3), _rows(n, n_kv, d, 4)
    k[9::16], v[9::16] = k[4::16], v[4::16]  # equal rows: the bytes are then determined
    mem, cache = cuda_lib.alloc_kv_cache(n // page + 1, page, n_kv, d)
    mem.fill_(0x5A)
    want = mem.clone()
    ref.put(want, slots, k, v, page)
    status = _status()
    cuda_lib.kv_cache_write(cache, k, v, slots, status)
    assert torch.equal(mem, want)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    cuda_lib.kv_cache_read(cache, slots, ko, vo, status)
    kr, vr = ref.get(want, slots, page, n_kv, d)
    assert torch.equal(ko.double(), kr) and torch.equal(vo.double(), vr) and status.item() == 0
