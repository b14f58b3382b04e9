"""kv_paged_attention against the 64-bit statement.

Bound, before any run: with u = 2^-8 (bf16's unit roundoff) for the output's own rounding; the
probabilities' rounding to f16 is 2^-11 relative per term; a score's fp32 sum of d products is off
by at most d * 2^-24 * sum |q k| * scale, under 2^-12 for these inputs (sum |q k| * scale < 32), which
moves a probability and the sum by as much each. A probability under 2^-33 of its row's largest may
count as zero: n tokens' together add at most n * 2^-33 of the largest |v|. So |out - exact| <=
u (1 + u) |exact| + 2^-9 A + n 2^-33 max|v| with A = sum_j p_j |v_j|, and |lse - exact| <=
2^-11 (1 + |exact|)."""
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


@pytest.fixture(autouse=True, params=["few", "many", "choice"])
def kernel(request, cuda_lib):
    """Every case on the kernel for few query rows, on the one for many, and on the library's choice."""
    if request.param == "choice" and request.node.originalname not in CHOSEN:
        pytest.skip("the two kernels themselves cover it")
    cuda_lib.pqe_test_set_attention_kernel({"few": 1, "many": 2, "choice": 0}[request.param])
    yield request.param
    cuda_lib.pqe_test_set_attention_kernel(0)


CHOSEN = ("test_single_tokens_beside_a_prompt", "test_other_stream_and_graph_follow_the_lengths", "test_many_sequences",
          "test_max_q_only_chooses_the_kernel")


class Case:
    """Sequences in a paged cache whose every other byte is 0xFF: scales of NaN where no token was written."""

    def __init__(self, pqe, ms, lens, n_q, n_kv, d, page, seed=0, big=None, q_big=1.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.pqe, self.ms, self.lens, self.n_q, self.n_kv, self.d, self.page = pqe, ms, lens, n_q, n_kv, d, page
        need = [-(-n // page) for n in lens]
        self.n_pages, self.width = sum(need) + 3, max(max(need), 1) + 1
        perm = torch.randperm(self.n_pages, generator=g, device=DEV)
        self.table = torch.full((len(lens), self.width), 1 << 30, dtype=torch.int32, device=DEV)  # never looked at
        self.mem = torch.full((self.n_pages * pqe.pqe_kv_page_bytes(page, n_kv, d),), 255, dtype=torch.uint8, device=DEV)
        self.cache = pqe.make_kv_cache(self.mem, self.n_pages, page, n_kv, d)
        self.slots, used = [], 0
        for b, n in enumerate(need):
            own = perm[used:used + n]
            self.table[b, :n] = own.int()
            at = torch.arange(lens[b], device=DEV)
            self.slots.append(own[at // page] * page + at % page)
            used += n
        big = big or (lambda x: x)
        for s in self.slots:
            if len(s):
                rows = torch.randn((2, len(s), n_kv, d), generator=g, device=DEV)
                ref.put(self.mem, s, big(rows[0]).bfloat16(), big(rows[1]).bfloat16(), page)
        self.total = sum(ms)
        self.q = (torch.randn((self.total, n_q, d), generator=g, device=DEV) * q_big).bfloat16()
        self.scale = d ** -0.5
        self.offsets = torch.tensor([sum(ms[:i]) for i in range(len(ms) + 1)], dtype=torch.int32, device=DEV)
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def kv(self):
        return [ref.get(self.mem, s, self.page, self.n_kv, self.d) for s in self.slots]

    def run(self, lse=True, q=None, max_q=None, **kw):
        pqe = self.pqe
        q = self.q if q is None else q
        out = torch.full((q.shape[0], self.n_q, self.d), 99.0, dtype=torch.bfloat16, device=DEV)
        l = torch.full((q.shape[0], self.n_q), 99.0, dtype=torch.float32, device=DEV) if lse else None
        max_q = max(self.ms) if max_q is None else max_q
        ws = torch.full((pqe.kv_paged_attention_workspace_size(len(self.lens), q.shape[0], max_q, self.n_q, self.n_kv, self.d),),
                        255, dtype=torch.uint8, device=DEV)
        pqe.kv_paged_attention(self.cache, q, self.offsets, self.kv_lens, self.table, max_q, self.scale, out, ws, self.status,
                               lse=l, **kw)
        return out, l

    def check(self, causal=True, window=0):
        out, lse = self.run(causal=causal, window=window)
        assert self.status.item() == 0
        o, a, l = ref.attend(self.q, self.ms, self.lens, self.kv(), self.scale, causal, window)
        compare(out, lse, o, a, l, floor(self.kv()))


def floor(kv):
    """n 2^-33 max|v|, the largest over the sequences."""
    return max((k.shape[0] * 2.0 ** -33 * torch.nan_to_num(v).abs().max().item() for k, v in kv if len(k)), default=0.0)


def compare(out, lse, o, a, l, least=0.0):
    out = out.double()
    assert torch.equal(torch.isnan(out), torch.isnan(o))
    off = (out - o).abs() - (U * (1 + U) * o.abs() + 2.0 ** -9 * a + least)
    assert not (off > 0).any(), off.max().item()
    empty = l == float("-inf")
    assert torch.equal(lse == float("-inf"), empty) and torch.equal(torch.isnan(lse), torch.isnan(l))
    assert not ((lse.double() - l).abs() > 2.0 ** -11 * (1 + l.abs())).any()
    assert (out[empty] == 0).all()


HEADS = [(1, 1), (4, 4), (16, 4), (20, 4), (3, 1), (14, 2), (32, 2), (40, 1), (8, 8)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q,n_kv", HEADS)
def test_single_tokens(cuda_lib, d, n_q, n_kv):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 200, 517]
    Case(cuda_lib, [1] * len(lens), lens, n_q, n_kv, d, 16, seed=n_q).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("d", [64, 128])
def test_page_sizes(cuda_lib, page, d):
    lens = [1, 31, 33, 64, 100, 129, 1025, 1100]
    Case(cuda_lib, [1, 2, 1, 3, 1, 5, 2, 1], lens, 12, 3, d, page, seed=page).check()


@pytest.mark.parametrize("m", [2, 3, 5, 7, 8, 16, 17, 33])
@pytest.mark.parametrize("d,n_q,n_kv", [(64, 8, 2), (128, 5, 1), (128, 8, 8)])
def test_few_tokens(cuda_lib, m, d, n_q, n_kv):
    lens = [m, m + 1, 70, 300, 129]
    Case(cuda_lib, [m, m - 1, min(m, 70), 1, m], lens, n_q, n_kv, d, 32, seed=m).check()


@pytest.mark.parametrize("d,n_q,n_kv,page", [(64, 4, 1, 16), (128, 8, 2, 64), (128, 3, 3, 128), (64, 10, 2, 32), (128, 16, 1, 16)])
@pytest.mark.parametrize("window", [0, 1, 40, 200])
def test_prompts(cuda_lib, d, n_q, n_kv, page, window):
    ms = [100, 1, 257, 64, 130, 31]
    lens = [100, 1, 400, 512, 131, 1000]
    Case(cuda_lib, ms, lens, n_q, n_kv, d, page, seed=d + window).check(window=window)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 300])
def test_window_single(cuda_lib, window):
    Case(cuda_lib, [1, 1, 3, 1], [1, 64, 333, 1000], 8, 2, 128, 16, seed=window).check(window=window)


@pytest.mark.parametrize("ms", [[1, 1, 1], [4, 2, 7], [90, 3, 140]])
def test_not_causal(cuda_lib, ms):
    Case(cuda_lib, ms, [130, 3, 257], 8, 2, 64, 16).check(causal=False)


@pytest.mark.parametrize("ms,lens", [([1, 1, 1], [0, 5, 0]), ([3, 4, 2], [1, 0, 2]), ([0, 2, 0, 1], [50, 60, 0, 1]), ([70, 90], [20, 0]),
                                     ([1], [0]), ([200], [0])])
def test_rows_that_see_nothing(cuda_lib, ms, lens):
    """No cached token, more queries than cached tokens, sequences without queries."""
    Case(cuda_lib, ms, lens, 8, 2, 128, 16).check()
    Case(cuda_lib, ms, lens, 8, 2, 64, 32).check(window=3)


@pytest.mark.parametrize("m", [1, 5, 80])
def test_long_axis(cuda_lib, m):
    """Few rows over many tokens: the work is split along the cache and joined."""
    Case(cuda_lib, [m, m], [20011, 4096], 8, 2, 128, 64, seed=m).check()


def test_many_sequences(cuda_lib):
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 300, (700,), generator=g).tolist()
    ms = [int(x) for x in torch.randint(0, 4, (700,), generator=g)]
    Case(cuda_lib, ms, lens, 4, 2, 64, 16).check()


@pytest.mark.parametrize("m", [1, 40])
def test_scales_far_apart(cuda_lib, m):
    """Channels and tokens whose magnitudes differ by up to 2^16; scores stay of order one, so that every token counts."""
    def big(x):
        e = torch.arange(x.shape[-1], device=DEV) // 32 % 4 * 4
        t = torch.arange(x.shape[0], device=DEV) % 5 - 4
        return x * torch.exp2(e.float()) * torch.exp2(t.float())[:, None, None]
    c = Case(cuda_lib, [m, m], [333, 64 + m], 8, 2, 128, 16, big=big)
    c.scale = 2.0 ** -12
    c.check()


@pytest.mark.parametrize("m", [1, 40])
@pytest.mark.parametrize("power", [-90, -30, 30, 90])
def test_magnitudes(cuda_lib, m, power):
    """K, V and q of any magnitude that bf16 holds: the scale brings the scores back."""
    c = Case(cuda_lib, [m], [200], 4, 1, 64, 16, big=lambda x: x * 2.0 ** power, q_big=2.0 ** (-power // 2))
    c.scale = 2.0 ** (-power + power // 2) / 8
    c.check()


@pytest.mark.parametrize("m", [1, 6, 100])
def test_peaked_rows(cuda_lib, m):
    """Scores of several hundred: the running maximum moves by far more than a float's range allows unscaled."""
    c = Case(cuda_lib, [m, m], [400, 150], 8, 2, 128, 16, big=lambda x: x * 4)
    c.scale = 1.0
    out, lse = c.run()
    o, a, l = ref.attend(c.q, c.ms, c.lens, c.kv(), c.scale)
    # scores up to about 1000 lie within 2^-24 * (d + 2) * sum |q k| (under 2^13) of the exact: 0.06 at worst for the sums'
    # order, far less in practice; held to 2^-7 here, on the probabilities and so on A
    assert not ((out.double() - o).abs() > U * (1 + U) * o.abs() + 2.0 ** -6 * a + floor(c.kv())).any()
    assert not ((lse.double() - l).abs() > 2.0 ** -7 + 2.0 ** -20 * l.abs()).any()


@pytest.mark.parametrize("m", [1, 4, 90])
def test_nan_tokens_reach_only_what_sees_them(cuda_lib, m):
    """A token whose V (or K) held a NaN: rows that see it turn to NaN (its channels' block for V, all for K), others do not."""
    d, page, n = 128, 16, 150
    for which in ("k", "v"):
        c = Case(cuda_lib, [m, m], [n, 40 + m], 8, 2, d, page, seed=3)
        rows = torch.zeros((1, 2, d), device=DEV)
        rows[0, 1, 40] = float("nan")
        bad = n - 1 - m // 2  # some of the queries come before it
        k0, v0 = ref.get(c.mem, c.slots[0][bad:bad + 1], page, 2, d)
        k, v = (rows + k0, v0) if which == "k" else (k0, rows + v0)
        ref.put(c.mem, c.slots[0][bad:bad + 1], k, v, page)
        out, lse = c.run()
        kv = c.kv()
        o, a, l = ref.attend(c.q, c.ms, c.lens, kv, c.scale)
        compare(out, lse, o, a, l, floor(kv))
        assert torch.isnan(o).any() and not torch.isnan(o).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [1, 4, 90])
def test_nan_scales_with_any_codes(cuda_lib, m, d):
    """A scale byte of 255 is NaN whatever the block's codes are (a cache filled elsewhere may hold other ones than zero), also
    where the block's product with q is below zero."""
    page, n = 16, 150
    for which, sign in (("k", 1), ("k", -1), ("v", 1)):
        c = Case(cuda_lib, [m, m], [n, 40 + m], 8, 2, d, page, seed=5)
        c.q = (sign * c.q.abs()).bfloat16()
        bad = n - 1 - m // 2
        slot = c.slots[0][bad].item()
        block = slot // page * cuda_lib.pqe_kv_page_bytes(page, 2, d) + 17 * d  # head 1's only block of the page
        t = slot % page
        if which == "k":
            c.mem[block + t * (d // 2):block + (t + 1) * (d // 2)] = 0x77  # codes of 6
            c.mem[block + 16 * d + t * (d // 32) + 1] = 255
        else:
            c.mem[block + 16 * d + d // 2 + (t % 8) // 2 * (d // 8) + 4 + t % 2 + 2 * (t // 8)] = 255
        kv = c.kv()
        assert torch.isnan(kv[0][0 if which == "k" else 1][bad, 1, 32:64]).all()
        out, lse = c.run()
        o, a, l = ref.attend(c.q, c.ms, c.lens, kv, c.scale)
        compare(out, lse, o, a, l, floor(kv))
        assert torch.isnan(o).any() and not torch.isnan(o).all()


@pytest.mark.parametrize("m", [1, 70])
def test_query_that_is_not_finite(cuda_lib, m):
    c = Case(cuda_lib, [m, m], [100, 90], 8, 2, 64, 16)
    want, _ = c.run()
    c.q[0, 3, 5] = float("nan")
    c.q[m, 1, 0] = float("inf")
    out, lse = c.run()
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
    hit[0, 3] = hit[m, 1] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], want[~hit])


@pytest.mark.parametrize("m", [1, 3, 100])
def test_bad_table_entries_and_lengths(cuda_lib, m):
    pqe = cuda_lib
    c = Case(pqe, [m, m, m], [200, 150, 120], 8, 2, 64, 16)
    want, _ = c.run()
    for value in (-1, c.n_pages, 1 << 30):
        c.status.zero_()
        held = c.table[1, 3].item()
        c.table[1, 3] = value
        out, lse = c.run()
        assert c.status.item() == pqe.PQE_STATUS_BAD_PAGE
        assert torch.equal(out[:m], want[:m]) and torch.equal(out[2 * m:], want[2 * m:])
        # the page's tokens count as masked: as if they were not there
        kv = c.kv()
        keep = torch.ones(150, dtype=torch.bool, device=DEV)
        keep[48:64] = False
        if m == 1:
            o, a, l = ref.attend(c.q[m:2 * m], [m], [134], [(kv[1][0][keep], kv[1][1][keep])], c.scale)
            compare(out[m:2 * m], lse[m:2 * m], o, a, l)
        c.table[1, 3] = held
    c.status.zero_()
    c.kv_lens[1] = c.width * 16 + 5  # beyond the table: cut, and its entries past the sequence's own are bad
    out, _ = c.run()
    assert c.status.item() == pqe.PQE_STATUS_BAD_PAGE
    assert torch.equal(out[:m], want[:m]) and torch.equal(out[2 * m:], want[2 * m:])


@pytest.mark.parametrize("m", [1, 80])
def test_strided_queries_and_spare_rows(cuda_lib, m):
    c = Case(cuda_lib, [m, m], [100, 200], 8, 2, 64, 16)
    want, _ = c.run()
    fused = torch.zeros((2 * m + 3, 12 * 64), dtype=torch.bfloat16, device=DEV)
    fused[:2 * m, :8 * 64] = c.q.flatten(1)
    out, lse = c.run(q=fused.view(-1, 12, 64)[:, :8])
    assert torch.equal(out[:2 * m], want)
    assert (out[2 * m:] == 99.0).all() and (lse[2 * m:] == 99.0).all()  # rows of no sequence stay as they are


def test_cache_beyond_32_bit_offsets(cuda_lib):
    pqe = cuda_lib
    n_kv, d, page, n = 8, 128, 64, 300
    nb = pqe.pqe_kv_page_bytes(page, n_kv, d)
    n_pages = (5 << 30) // nb
    mem = torch.empty(n_pages * nb, dtype=torch.uint8, device=DEV)
    cache = pqe.make_kv_cache(mem, n_pages, page, n_kv, d)
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2, 0, n_pages - 7]], dtype=torch.int32, device=DEV)
    at = torch.arange(n, device=DEV)
    slots = table[0].long()[at // page] * page + at % page
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn((n, n_kv, d), generator=g, device=DEV).bfloat16() for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pqe.kv_cache_write(cache, k, v, slots, status)
    kv = [(ref.values(*ref.mxfp4(k)), ref.values(*ref.mxfp4(v)))]
    for m in (1, 100):
        q = torch.randn((m, 16, d), generator=g, device=DEV).bfloat16()
        out, lse = torch.empty_like(q), torch.empty((m, 16), device=DEV)
        ws = torch.empty(pqe.kv_paged_attention_workspace_size(1, m, m, 16, n_kv, d), dtype=torch.uint8, device=DEV)
        pqe.kv_paged_attention(cache, q, torch.tensor([0, m], dtype=torch.int32, device=DEV),
                               torch.tensor([n], dtype=torch.int32, device=DEV), table, m, d ** -0.5, out, ws, status, lse=lse)
        compare(out, lse, *ref.attend(q, [m], [n], kv, d ** -0.5))
    assert status.item() == 0


@pytest.mark.parametrize("m", [1, 100])
def test_same_bits_every_time(cuda_lib, m):
    c = Case(cuda_lib, [m, 1, m], [5000, 1, 333], 16, 2, 128, 16)
    first, l1 = c.run()
    for _ in range(5):
        out, l2 = c.run()
        assert torch.equal(out, first) and torch.equal(l1, l2)


@pytest.mark.parametrize("m", [1, 100])
def test_other_stream_and_graph_follow_the_lengths(cuda_lib, m):
    c = Case(cuda_lib, [m, m], [300, 200], 8, 2, 128, 16)
    want, _ = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, _ = c.run()
    s.synchronize()
    assert torch.equal(out, want)
    pqe = cuda_lib
    out = torch.empty_like(c.q)
    ws = torch.empty(pqe.kv_paged_attention_workspace_size(2, c.total, m, 8, 2, 128), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pqe.kv_paged_attention(c.cache, c.q, c.offsets, c.kv_lens, c.table, m, c.scale, out, ws, c.status)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    c.kv_lens[0], c.lens[0] = 250, 250
    c.slots[0] = c.slots[0][:250]
    graph.replay()
    torch.cuda.synchronize()
    o, a, _ = ref.attend(c.q, c.ms, c.lens, c.kv(), c.scale)
    assert not ((out.double() - o).abs() > U * (1 + U) * o.abs() + 2.0 ** -9 * a).any()


def test_max_q_only_chooses_the_kernel(cuda_lib):
    """The same call under another bound on the queries: both kernels agree within the bound."""
    c = Case(cuda_lib, [40, 1, 33], [300, 70, 33], 8, 2, 128, 16)
    o, a, l = ref.attend(c.q, c.ms, c.lens, c.kv(), c.scale)
    for max_q in (40, 1000):
        out, lse = c.run(max_q=max_q)
        compare(out, lse, o, a, l)


@pytest.mark.parametrize("m", [1, 4, 100])
def test_pages_before_the_window_may_be_gone(cuda_lib, m):
    c = Case(cuda_lib, [m, m], [700, 333], 8, 2, 128, 16)
    want, _ = c.run(window=50)
    c.table[0, :(700 - m - 50 + 1) // 16] = -1
    c.table[1, :(333 - m - 50 + 1) // 16] = 1 << 29
    c.check(window=50)
    out, _ = c.run(window=50)
    assert torch.equal(out, want) and c.status.item() == 0


def test_one_call_and_single_tokens_agree(cuda_lib):
    """The same queries as one call of 40 a sequence and as calls of one."""
    c = Case(cuda_lib, [40, 40], [300, 70], 8, 2, 64, 16)
    o, a, l = ref.attend(c.q, c.ms, c.lens, c.kv(), c.scale)
    out, lse = c.run()
    compare(out, lse, o, a, l, floor(c.kv()))
    single = Case(cuda_lib, [1, 1], [300, 70], 8, 2, 64, 16)
    for i in (0, 17, 39):
        single.q = c.q[[i, 40 + i]].contiguous()
        single.kv_lens.copy_(torch.tensor([300 - 39 + i, 70 - 39 + i]))
        single.mem, single.cache, single.table = c.mem, c.cache, c.table
        got, gl = single.run()
        compare(got, gl, o[[i, 40 + i]], a[[i, 40 + i]], l[[i, 40 + i]], floor(c.kv()))


@pytest.mark.parametrize("m", [1, 3, 100])
def test_waits_that_run_out(cuda_lib, m):
    """With a limit of one poll the waits for data give up before it is there (or, rarely, just find it): the call comes back,
    says so in its status, and the next call is right."""
    pqe = cuda_lib
    c = Case(pqe, [m, m], [2000, 3000], 8, 2, 128, 16)
    want, l = c.run()
    try:
        assert pqe.lib().pqe_set_wait_limit(1) == 0
        out, _ = c.run()
        torch.cuda.synchronize()
    finally:
        pqe.lib().pqe_set_wait_limit(0)
    assert c.status.item() in (0, pqe.PQE_STATUS_TIMEOUT)
    if c.status.item() == 0:
        assert torch.equal(out, want)
    c.status.zero_()
    again, l2 = c.run()
    assert c.status.item() == 0 and torch.equal(again, want) and torch.equal(l2, l)


def test_many_prompts_in_one_call(cuda_lib):
    """More sequences than a block has threads, with and without queries, in the kernel for many rows."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 60, (1100,), generator=g).tolist()
    ms = [min(int(x), n) if i % 3 else 0 for i, (x, n) in enumerate(zip(torch.randint(0, 40, (1100,), generator=g), lens))]
    ms[500], lens[500] = 70, 80
    Case(cuda_lib, ms, lens, 2, 1, 64, 16).check()


@pytest.mark.parametrize("n_q,n_kv,d", [(8, 2, 128), (16, 1, 64), (4, 4, 64)])
def test_single_tokens_beside_a_prompt(cuda_lib, n_q, n_kv, d):
    """One call with a prompt's chunk and sequences of one and a few tokens, of long and empty ones. (On the library's choice:
    both kernels, each with its own sequences.)"""
    ms = [1, 1050, 1, 0, 2, 1, 1, 17, 1, 3, 1, 1]
    lens = [700, 1100, 1, 30, 65, 0, 1300, 17, 64, 2, 129, 512]
    Case(cuda_lib, ms, lens, n_q, n_kv, d, 16, seed=d).check()
    Case(cuda_lib, ms, lens, n_q, n_kv, d, 32, seed=d + 1).check(window=100)


def test_kernel_hook_rejects_unknown_kind(cuda_lib):
    with pytest.raises(cuda_lib.PqeError):
        cuda_lib.pqe_test_set_attention_kernel(3)
