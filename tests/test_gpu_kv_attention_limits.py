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


def _unlike(c, window, hit, least=2.0 ** -32):
    """Rows marked in `hit` see a token out of scale with the others: finite is all that is asked of them. The others are held to
    the bound of what they see themselves: n 2^-32 of the largest |v| among their tokens, since V's factors, up to 2^8 below
    the largest of the tile's rows, meet probabilities in f16."""
    out, lse = c.run(window=window)
    assert c.status.item() == 0
    kv = c.kv()
    o, a, l = ref.attend(c.q, c.ms, c.lens, kv, c.scale, True, window)
    rest, start = torch.zeros(c.total, dtype=torch.float64, device=DEV), 0
    for m, n, (k, v) in zip(c.ms, c.lens, kv):
        for i in range(m):
            pos = n - m + i
            seen = v[max(pos - window + 1, 0) if window else 0:max(pos + 1, 0)]
            rest[start + i] = len(seen) * least * seen.abs().max() if len(seen) else 0.0
        start += m
    keep = ~hit
    assert torch.isfinite(out[hit]).all() and torch.isfinite(lse[hit]).all()
    off = (out.double() - o).abs() - (U * (1 + U) * o.abs() + 2.0 ** -9 * a + rest[:, None, None])
    assert not (off[keep] > 0).any(), off[keep].max().item()
    assert torch.equal(lse[keep] == float("-inf"), l[keep] == float("-inf"))
    both = keep[:, None] & (l != float("-inf"))
    assert not ((lse.double() - l).abs() > 2.0 ** -11 * (1 + l.abs()))[both].any()


def _grow(c, b, token, power, k=False, v=False, block=None):
    """Token `token` of sequence b 2^power times as large: its K, its V, or one 32-channel block of them."""
    at = c.slots[b][token:token + 1]
    rows = list(ref.get(c.mem, at, c.page, c.n_kv, c.d))
    part = slice(None) if block is None else slice(32 * block, 32 * block + 32)
    for x, use in zip(rows, (k, v)):
        if use:
            x[..., part] *= 2.0 ** power
    ref.put(c.mem, at, *(x.bfloat16() for x in rows), c.page)


def _sees(c, b, token, window):
    """Which rows see the token."""
    hit = torch.zeros(c.total, dtype=torch.bool, device=DEV)
    start = sum(c.ms[:b])
    for i in range(c.ms[b]):
        pos = c.lens[b] - c.ms[b] + i
        hit[start + i] = token <= pos and (not window or token > pos - window)
    return hit


POWERS = [4, 7, 8, 9, 11, 13, 14, 24, 40, 90]


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [2, 5, 100])
def test_large_values_that_a_query_does_not_see(cuda_lib, m, d, power):
    """A token that comes after some of the queries, with V far above all others: nothing of it reaches those. One sequence of many
    cached tokens, one of none but the queries' own; all channels, and one block of them."""
    for lens, block in (([300, m], None), ([5000, 70 + m], 1)):
        c = Case(cuda_lib, [m, m], lens, 8, 2, d, 16, seed=m)
        hit = torch.zeros(c.total, dtype=torch.bool, device=DEV)
        for b, token in ((0, lens[0] - 1), (1, lens[1] - 1 - m // 3)):
            _grow(c, b, token, power, v=True, block=block)
            hit |= _sees(c, b, token, 0)
        assert hit.any() and not hit.all()
        _unlike(c, 0, hit)


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("d,page", [(64, 32), (128, 16)])
@pytest.mark.parametrize("m,window", [(2, 30), (5, 17), (100, 40), (100, 3), (3, 3000)])
def test_large_values_before_the_window(cuda_lib, m, window, d, page, power):
    """Tokens that some queries' windows no longer hold, and one that none does, with V (and K, of the last) far above all others."""
    n = 700 if window < 700 else 5000
    c = Case(cuda_lib, [m, m], [n, m + 20], 8, 2, d, page, seed=window)
    first = n - m - window + 1  # the first query's first token
    _grow(c, 0, first, power, v=True)  # that only the first query sees
    _grow(c, 0, first - 1, power, k=True, v=True)  # that none does
    _grow(c, 1, 4, power, v=True)
    hit = _sees(c, 0, first, window) | _sees(c, 1, 4, window)
    assert hit.any() and not hit.all()
    _unlike(c, window, hit)


@pytest.mark.parametrize("m", [4, 40])
def test_queries_that_see_only_small_values(cuda_lib, m):
    """First tokens with V of zero and of almost nothing, and heads whose values differ by 2^60."""
    c = Case(cuda_lib, [m, m], [m, 30 + m], 8, 2, 128, 16, seed=9)
    for b in (0, 1):
        for token, power in ((0, None), (1, -40), (2, -20)):
            at = c.slots[b][token:token + 1]
            k, v = ref.get(c.mem, at, 16, 2, 128)
            v = v * (0.0 if power is None else 2.0 ** power)
            v[:, 1] *= 2.0 ** -60
            ref.put(c.mem, at, k.bfloat16(), v.bfloat16(), 16)
    _unlike(c, 0, torch.zeros(c.total, dtype=torch.bool, device=DEV))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [2, 60])
def test_rows_out_of_scale_keep_the_other_rules(cuda_lib, m, d):
    """Beside a token that only the last query sees and that is 2^40 larger: a bad table entry, NaN in K and V blocks, a query that
    is not finite, strided queries; equal bits every time."""
    n = 300
    c = Case(cuda_lib, [m, m], [n, n], 8, 2, d, 16, seed=m + d)
    for b in (0, 1):
        _grow(c, b, n - 1, 40, v=True)
    c.q[m, 3, 5] = float("nan")
    at = c.slots[1][[7, n - 1 - m // 2]]
    k, v = ref.get(c.mem, at, 16, 2, d)
    v[0, 0, 33] = float("nan")  # all queries see it
    k[1, 1, 0] = float("inf")  # some of them
    ref.put(c.mem, at, k.bfloat16(), v.bfloat16(), 16)
    kv = c.kv()
    c.table[0, 3] = c.n_pages  # 16 tokens of the first sequence are gone
    here = torch.ones(n, dtype=torch.bool, device=DEV)
    here[48:64] = False
    kv[0] = tuple(x[here] for x in kv[0])
    fused = torch.zeros((2 * m, 12, d), dtype=torch.bfloat16, device=DEV)
    fused[:, 2:10] = c.q
    out, lse = c.run(q=fused[:, 2:10])
    assert c.status.item() == cuda_lib.PQE_STATUS_BAD_PAGE
    o, a, l = ref.attend(c.q, c.ms, [n - 16, n], kv, c.scale)
    o[m, 3] = l[m, 3] = float("nan")  # (the statement's own 0 * NaN leaves nothing else of that row)
    keep = torch.ones(2 * m, dtype=torch.bool, device=DEV)
    keep[[m - 1, 2 * m - 1]] = False
    least = n * 2.0 ** -32 * max(torch.nan_to_num(v[:-1]).abs().max().item() for _, v in kv)
    compare(out[keep], lse[keep], o[keep], a[keep], l[keep], least)
    for _ in range(3):
        again, lse2 = c.run()
        assert torch.equal(torch.nan_to_num(again, nan=7.0), torch.nan_to_num(out, nan=7.0))
        assert torch.equal(torch.nan_to_num(lse2, nan=7.0), torch.nan_to_num(lse, nan=7.0))


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [2, 5, 100, 300])
def test_large_keys_that_a_query_does_not_see(cuda_lib, m, d, power):
    """As the values: scores of the queries before the token keep their own K blocks."""
    for lens, block in (([300 + m, m], None), ([5000, 70 + m], 1)):
        c = Case(cuda_lib, [m, m], lens, 8, 2, d, 16, seed=m)
        hit = torch.zeros(c.total, dtype=torch.bool, device=DEV)
        for b, token in ((0, lens[0] - 1), (1, lens[1] - 1 - m // 3)):
            _grow(c, b, token, power, k=True, block=block)
            hit |= _sees(c, b, token, 0)
        assert hit.any() and not hit.all()
        _unlike(c, 0, hit)


@pytest.mark.parametrize("power", [24, 40, 90])
@pytest.mark.parametrize("d,page", [(64, 32), (128, 16)])
@pytest.mark.parametrize("m,window", [(1, 30), (5, 18), (100, 40), (3, 3000), (300, 129)])
def test_large_values_that_no_query_sees(cuda_lib, m, window, d, page, power):
    """The tokens just before the first query's window, in the same block of 16 as tokens that it sees (of one sequence at least), with K
    and V far above all others: every row is as without them."""
    n = 700 if window < 700 else 5000
    c = Case(cuda_lib, [m, m], [n, n + 5], 8, 2, d, page, seed=window)
    for b in (0, 1):
        first = c.lens[b] - m - window + 1
        for token in range(first // 16 * 16, first):
            _grow(c, b, token, power, k=True, v=True)
    _unlike(c, window, torch.zeros(c.total, dtype=torch.bool, device=DEV))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [1, 5, 100])
@pytest.mark.parametrize("power", [16, 20, 24, 28, 40, 80])
def test_scores_of_any_size(cuda_lib, m, d, power):
    """Scores of 2^power times a few units, of either sign: a row is its largest score's token alone. The scores' fp32 sums (of d
    products, and of d / 32 scaled blocks) are off by (d + 4) 2^-24 sum |q k| scale at most: rows whose two largest are nearer than
    twice that and 2^6 more are not asked for. (Those left have p below 2^-64 for every other token.)"""
    for sign in (1, -1):
        c = Case(cuda_lib, [m, m], [400, 100 + m], 8, 2, d, 16, seed=power)
        if sign < 0:  # all scores below zero
            c.q = c.q.abs()
            for s in c.slots:
                k, v = ref.get(c.mem, s, 16, 2, d)
                ref.put(c.mem, s, -k.abs().bfloat16(), v.bfloat16(), 16)
        c.scale = 2.0 ** power
        out, lse = c.run()
        assert c.status.item() == 0 and torch.isfinite(out).all() and torch.isfinite(lse).all()
        kv = c.kv()
        o, a, l = ref.attend(c.q, c.ms, c.lens, kv, c.scale)
        assert not ((lse.double() - l).abs() > 2.0 ** -11 * (1 + l.abs())).any()
        clear, start = torch.zeros((c.total, 8), dtype=torch.bool, device=DEV), 0
        for n, (k, v) in zip(c.lens, kv):
            q = c.q[start:start + m].double().view(m, 2, 4, d)
            see = torch.arange(n, device=DEV)[None] <= n - m + torch.arange(m, device=DEV)[:, None]
            z = torch.einsum("mhgd,jhd->mhgj", q, k).masked_fill(~see[:, None, None], float("-inf")) * c.scale
            size = torch.einsum("mhgd,jhd->mhgj", q.abs(), k.abs()).masked_fill(~see[:, None, None], 0.0).amax(-1) * c.scale
            top = z.topk(2, -1).values
            clear[start:start + m] = (top[..., 0] - top[..., 1] > 2 * (d + 4) * 2.0 ** -24 * size + 64).view(m, 8)
            start += m
        assert clear.float().mean() > 0.9
        assert not ((out.double() - o).abs() > U * (1 + U) * o.abs() + 2.0 ** -9 * a + floor(kv))[clear].any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [1, 3, 100])
def test_waits_that_expire(cuda_lib, m, d):
    """Every wait for data gives up without a poll: the call comes back, says so in its status, and the next one is right. (The
    waits for what is in flight keep their own limit, so that nothing lands in a block that has ended.)"""
    c = Case(cuda_lib, [m, m], [2000, 3000], 8, 2, d, 16)
    want, l = c.run()
    for _ in range(3):
        try:
            cuda_lib.pqe_test_set_attention_polls(0)
            c.run()
            torch.cuda.synchronize()
        finally:
            cuda_lib.pqe_test_set_attention_polls(-1)
        assert c.status.item() == cuda_lib.PQE_STATUS_TIMEOUT
        c.status.zero_()
        again, l2 = c.run()
        assert c.status.item() == 0 and torch.equal(again, want) and torch.equal(l2, l)


def test_polls_hook_rejects_less(cuda_lib):
    with pytest.raises(cuda_lib.PqeError):
        cuda_lib.pqe_test_set_attention_polls(-2)
