"""Refusals of the attention-side calls: bad arguments return PQE_ERR_INVALID_ARG before any launch. CPU only."""
import ctypes as C

import pytest
import torch

import paged_quantized_expert_gb300 as pqe

BAD = pqe.PQE_ERR_INVALID_ARG
A = 4096  # a 256-byte aligned address that is never read


def _cache(**kw):
    f = dict(pages=A, page_stride=pqe.pqe_kv_page_bytes(16, 2, 64), n_pages=4, page_size=16, n_kv=2, d=64) | kw
    return C.byref(pqe.pqe_kv_cache(*(f[n] for n, _ in pqe.pqe_kv_cache._fields_)))


def test_page_bytes():
    pqe.load()
    assert pqe.pqe_kv_page_bytes(16, 1, 128) == 17 * 128
    assert pqe.pqe_kv_page_bytes(64, 8, 64) == 8 * 4 * 17 * 64
    for bad in ((8, 1, 64), (24, 1, 64), (2048, 1, 64), (16, 0, 64), (16, 257, 64), (16, 1, 96), (16, 1, 256)):
        assert pqe.pqe_kv_page_bytes(*bad) == 0


BAD_CACHES = [dict(pages=None), dict(pages=A + 8), dict(page_stride=16), dict(page_stride=pqe.pqe_kv_page_bytes(16, 2, 64) + 8),
              dict(n_pages=0), dict(page_size=48), dict(n_kv=0), dict(d=80)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches(kw):
    lib = pqe.load()
    c = _cache(**kw)
    assert lib.kv_cache_write(c, A, A, 128, 128, A, 1, A, None) == BAD
    assert lib.kv_cache_read(c, A, 1, A, A, A, None) == BAD
    assert _attend(lib, c) == BAD


def test_write_and_read_arguments():
    lib = pqe.load()
    ok = [_cache(), A, A, 128, 128, A, 1, A, None]
    for i, v in ((0, None), (1, None), (2, None), (1, A + 2), (2, A + 8), (3, 120), (4, 0), (3, 132), (5, None), (5, A + 4), (6, -1), (7, None)):
        assert lib.kv_cache_write(*(v if j == i else x for j, x in enumerate(ok))) == BAD
    ok = [_cache(), A, 1, A, A, A, None]
    for i, v in ((0, None), (1, None), (2, -1), (3, A + 8), (5, None)):
        assert lib.kv_cache_read(*(v if j == i else x for j, x in enumerate(ok))) == BAD
    assert lib.kv_cache_read(_cache(), A, 1, None, None, A, None) == BAD
    assert lib.kv_cache_write(_cache(), None, None, 0, 0, None, 0, None, None) == 0  # no tokens: nothing to do
    assert lib.kv_cache_read(_cache(), None, 0, None, None, None, None) == 0


NAMES = ("q", "q_stride", "offsets", "lens", "table", "max_pages", "B", "total_q", "max_q", "n_q", "scale", "causal", "window", "out", "lse",
         "ws", "ws_bytes", "status", "stream")


def _attend(lib, cache=None, **kw):
    f = dict(q=A, q_stride=4 * 64, offsets=A, lens=A, table=A, max_pages=3, B=1, total_q=1, max_q=1, n_q=4, scale=0.1, causal=1, window=0,
             out=A, lse=None, ws=A, ws_bytes=1 << 40, status=A, stream=None) | kw
    return lib.kv_paged_attention(cache or _cache(), *(f[n] for n in NAMES))


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=A + 8), dict(q_stride=248), dict(q_stride=260), dict(offsets=None), dict(lens=None),
                                dict(table=None), dict(max_pages=0), dict(max_pages=1 << 28), dict(B=-1), dict(total_q=-1), dict(max_q=-1),
                                dict(max_q=0), dict(n_q=3), dict(n_q=0), dict(n_q=2048), dict(scale=float("nan")), dict(scale=float("inf")),
                                dict(window=-1), dict(causal=0, window=4), dict(out=None), dict(out=A + 4), dict(lse=A + 2), dict(ws=None),
                                dict(ws=A + 16), dict(ws_bytes=0), dict(status=None)])
def test_attention_arguments(kw):
    assert _attend(pqe.load(), **kw) == BAD


def test_attention_without_work():
    lib = pqe.load()
    assert _attend(lib, B=0, q=None) == 0 and _attend(lib, total_q=0, q=None) == 0
    assert pqe.kv_paged_attention_workspace_size(1, 1, 1, 3, 2, 64) == 0
    assert pqe.kv_paged_attention_workspace_size(1, 1, 1, 4, 2, 80) == 0
    assert pqe.kv_paged_attention_workspace_size(-1, 1, 1, 4, 2, 64) == 0
    assert pqe.kv_paged_attention_workspace_size(64, 64, 1, 16, 4, 128) > 0


@pytest.mark.parametrize("i,v", [(0, None), (0, A + 8), (1, 60), (1, 68), (2, A + 2), (3, 60), (4, None), (5, -1.0), (6, -1), (7, 0), (7, 48),
                                 (7, 32768), (8, A + 2), (9, A + 4), (10, A + 4), (11, None), (11, A + 2), (12, 7), (12, -1)])
def test_norm_arguments(i, v):
    lib = pqe.load()
    ok = [A, 64, A, 64, A, 1e-6, 1, 64, A, A, A, A, 0, None]
    assert lib.add_rms_norm(*(v if j == i else x for j, x in enumerate(ok))) == BAD


def test_norm_without_outputs_or_rows():
    lib = pqe.load()
    assert lib.add_rms_norm(A, 64, None, 0, A, 1e-6, 1, 64, None, None, None, None, 0, None) == BAD
    assert lib.add_rms_norm(None, 64, None, 0, None, 1e-6, 0, 64, None, None, None, None, 0, None) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    mem = torch.zeros(100, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pqe.make_kv_cache(mem, 1, 16, 2, 64)
    with pytest.raises(pqe.PqeError):
        pqe.make_kv_cache(mem, 1, 16, 2, 96)
    x = torch.zeros((2, 64), dtype=torch.float32)
    w = torch.ones(64, dtype=torch.bfloat16)
    y = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pqe.add_rms_norm(x, None, w, 1e-6, None, y)
    with pytest.raises(ValueError):
        pqe.add_rms_norm(y, None, w, 1e-6, None, y[:1])
    with pytest.raises(ValueError):
        pqe.add_rms_norm(y, None, w, 1e-6, None, None, torch.zeros((2, 64), dtype=torch.uint8), torch.zeros(1))
    mem, cache = pqe.alloc_kv_cache(4, 16, 2, 64, device="cpu")
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pqe.kv_cache_write(cache, k, k[:2], torch.zeros(3, dtype=torch.int64), st)
    with pytest.raises(ValueError):
        pqe.kv_cache_write(cache, k, k, torch.zeros(3, dtype=torch.int32), st)
    with pytest.raises(ValueError):
        pqe.kv_cache_write(cache, k[..., ::2], k, torch.zeros(3, dtype=torch.int64), st)
