"""sample_tokens against the definition in 64 bits.

Tokens have to be the definition's: weights carry 2^-30 relative, so a number u within 2^-30 of a border between two tokens
could go either way; the reference gives u's distance to the border, and none of the seeds below comes that near (asserted).
logprob: its parts (t's quotient, the sum's logarithm) are 64-bit or carry 2^-24 of values up to 2^7: within 2^-22 * (8 + |lp|)."""
import numpy as np
import pytest
import torch

import sampling_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, I32 = torch.float32, torch.int32


def run(pqe, logits, u, want_status=0, **kw):
    B = logits.shape[0]
    tokens = torch.full((B,), -7, dtype=I32, device=DEV)
    lps = torch.full((B,), 5.0, device=DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    dev = {n: torch.tensor(v, dtype=I32 if n == "top_k" else F32, device=DEV) for n, v in kw.items()}
    pqe.sample_tokens(logits, torch.as_tensor(u, dtype=F32, device=DEV), tokens, status, logprobs=lps, **dev)
    assert status.item() == want_status
    return tokens.cpu().numpy(), lps.cpu().numpy()


def check(pqe, logits, u, **kw):
    tokens, lps = run(pqe, logits, u, **kw)
    l = logits.float().cpu().double().numpy()
    u = np.asarray(torch.as_tensor(u, dtype=F32).cpu(), dtype=np.float64)
    short = {"temperature": "t", "top_k": "k", "top_p": "p", "min_p": "mp"}
    for b in range(len(tokens)):
        s = {short[n]: (int(v[b]) if n == "top_k" else float(np.float32(v[b]))) for n, v in kw.items()}
        t, lp, near = ref.draw(l[b], u[b], **s)
        assert near > 2.0 ** -30, "the seed puts u on a border: choose another"
        assert tokens[b] == t, (b, s, u[b], tokens[b], t)
        assert abs(lps[b] - lp) <= 2.0 ** -22 * (8 + abs(lp)), (b, s, lps[b], lp)


def rows(B, V, seed, dtype=F32, peak=True, stride=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = 2.5 * torch.randn((B, V), generator=g, device=DEV)
    if peak:
        l += 9 * torch.rand((B, V), generator=g, device=DEV) * (torch.rand((B, V), generator=g, device=DEV) < 0.01)
    l = l.to(dtype)
    if stride:
        wide = torch.full((B, stride), float("nan"), dtype=dtype, device=DEV)
        wide[:, 1:V + 1] = l
        l = wide[:, 1:V + 1]
    return l, torch.rand(B, generator=g, device=DEV)


def settings(B, seed):
    r = np.random.default_rng(seed)
    return {"temperature": r.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.5], B), "top_k": r.choice([0, 0, 1, 5, 50, 1000, -3, 10 ** 6], B),
            "top_p": r.choice([1.0, 0.9, 0.95, 0.5, 0.1, 0.0, 1.5], B), "min_p": r.choice([0.0, 0.0, 0.02, 0.3, 1e-4, -1.0], B)}


@pytest.mark.parametrize("V", [1, 2, 3, 31, 33, 100, 1000, 4097, 32000, 50001, 131072, 200003])
@pytest.mark.parametrize("dtype", [F32, torch.bfloat16])
def test_mixed_settings(cuda_lib, V, dtype):
    B = 40
    l, u = rows(B, V, V, dtype)
    check(cuda_lib, l, u, **settings(B, V + 1))


@pytest.mark.parametrize("B,V", [(1, 50), (1, 131072), (2, 70001), (3, 368640), (300, 3000), (700, 999)])
@pytest.mark.parametrize("peak", [False, True])
def test_batches(cuda_lib, B, V, peak):
    l, u = rows(B, V, B + V, peak=peak)
    check(cuda_lib, l, u, **settings(B, B))


@pytest.mark.parametrize("name,values", [("temperature", [0.1, 0.5, 1, 2, 30]), ("top_k", [1, 2, 3, 40, 999, 5000]), ("top_p", [0.01, 0.3, 0.8, 0.99, 0.9999]),
                                         ("min_p", [1e-6, 0.01, 0.1, 0.9, 1.0, 1.5])])
@pytest.mark.parametrize("dtype,peak", [(F32, True), (F32, False), (torch.bfloat16, False)])
def test_each_setting_alone(cuda_lib, name, values, dtype, peak):
    B = 8 * len(values)
    l, u = rows(B, 40007, len(values), dtype, peak)
    check(cuda_lib, l, u, **{name: np.repeat(values, 8)})


def test_no_settings_and_rows_that_lie_apart(cuda_lib):
    """Without settings: the whole softmax. Rows start at any element; what lies between them (NaN) is not read."""
    for dtype in (F32, torch.bfloat16):
        for V, stride in ((1001, 1007), (4096, 4099), (131, 200), (60000, 60008)):
            l, u = rows(6, V, V, dtype, stride=stride)
            check(cuda_lib, l, u)
            check(cuda_lib, l, u, **settings(6, V))


def test_every_u_of_a_small_row(cuda_lib):
    """4096 numbers over one row of 37 logits: each kept token in its turn, none that is not kept, whatever the cut."""
    r = np.random.default_rng(3)
    l = torch.tensor(r.normal(0, 2, 37), dtype=F32).repeat(4096, 1).to(DEV)
    u = (np.arange(4096) + 0.37) / 4096
    for kw in ({}, {"top_k": 7}, {"top_p": 0.7}, {"min_p": 0.1}, {"top_k": 12, "top_p": 0.8, "min_p": 0.01, "temperature": 1.4}):
        kw = {n: np.full(4096, v) for n, v in kw.items()}
        check(cuda_lib, l, u, **kw)


def test_ends_of_u(cuda_lib):
    """u = 0 draws the first kept token of any weight, the largest u below 1 the last."""
    l, _ = rows(4, 5000, 8)
    l[:, 0] = l[:, -1] = -200.0  # far too small to be drawn
    for u, at in ((0.0, 0), (1 - 2.0 ** -24, -1)):
        for k in (0, 3, 100):
            tokens, _ = run(cuda_lib, l, [u] * 4, top_k=[k] * 4)
            for b in range(4):
                i, w = ref.kept(l[b].cpu().double().numpy(), k=k)
                i = i[w > 2.0 ** -40]
                if at == 0:
                    assert tokens[b] == i[0]
                else:
                    cum = np.cumsum(w[w > 2.0 ** -40])
                    assert tokens[b] == i[np.searchsorted(cum, (1 - 2.0 ** -24) * cum[-1], side="right")]


def test_equal_logits(cuda_lib):
    """Equal logits are ordered by index: top_k and top_p keep the first of them, across the whole row."""
    for V in (10, 1000, 70000):
        B = 16
        l = torch.zeros((B, V), device=DEV)
        l[:, 1::2] = -0.0  # equal to 0
        u = (np.arange(B) + 0.5) / B
        check(cuda_lib, l, u, top_k=[7] * B)
        check(cuda_lib, l, u, top_p=[0.33] * B)
        check(cuda_lib, l, u, top_k=[V // 2 + 1] * B, top_p=[0.5] * B)
        check(cuda_lib, l, u, temperature=[0.0] * B)
        check(cuda_lib, l, u, min_p=[1.0] * B)
        l[:, V // 3:] = 1.5
        l[:, V - 2:] = 3.0
        check(cuda_lib, l, u, top_k=[V // 4 + 3] * B)
        check(cuda_lib, l, u, top_p=[0.9] * B, top_k=[V // 2] * B)


def test_few_values(cuda_lib):
    """A dozen distinct values over a long row, the cuts inside runs of equal ones."""
    r = np.random.default_rng(5)
    B, V = 24, 60000
    l = torch.tensor(r.choice(np.linspace(-8, 4, 12), (B, V)), dtype=F32, device=DEV)
    check(cuda_lib, l, r.random(B).astype(np.float32), top_k=r.integers(1, V, B), top_p=r.choice([0.2, 0.6, 0.9, 0.99], B))


def test_masked_rows(cuda_lib):
    """-infinity is never drawn; one token left; rows with nothing left, NaN or +infinity give -1 and the others their token."""
    B, V = 9, 9000
    l, u = rows(B, V, 21)
    l[0, :] = -float("inf")
    l[1, :] = -float("inf")
    l[1, 8999] = -3.0
    l[2, 100:] = -float("inf")
    l[3, 4567] = float("nan")
    l[4, 0] = float("inf")
    l[5, 8998] = -float("nan")
    l[6, :8000] = -float("inf")
    l[7, 17] = 3.4e38
    l[8, :] = -3.4e38
    tokens, lps = run(cuda_lib, l, u, want_status=cuda_lib.PQE_STATUS_NO_TOKEN, top_k=[0, 5, 0, 0, 0, 0, 2000, 0, 0], top_p=[1, 0.5, 0.9, 1, 1, 1, 1, 0.9, 1])
    assert [int(x) for x in tokens[[0, 3, 4, 5]]] == [-1] * 4 and np.isnan(lps[[0, 3, 4, 5]]).all()
    assert tokens[1] == 8999 and lps[1] == 0 and tokens[7] == 17 and lps[7] == 0
    good = l[[1, 2, 6, 7, 8]]
    check(cuda_lib, good, u[[1, 2, 6, 7, 8]], top_k=[5, 0, 2000, 0, 0], top_p=[0.5, 0.9, 1, 0.9, 1])
    check(cuda_lib, good, u[[1, 2, 6, 7, 8]], top_k=[5, 0, 2000, 0, 0], min_p=[0.1] * 5, temperature=[0.0, 1, 1, 1, 1])


def test_settings_out_of_range(cuda_lib):
    nan, inf = float("nan"), float("inf")
    l, _ = rows(10, 700, 2)
    u = [0.5] * 6 + [1.0, -0.1, nan, 0.5]
    tokens, lps = run(cuda_lib, l, u, want_status=cuda_lib.PQE_STATUS_NO_TOKEN, temperature=[-1.0, nan, inf, 1, 1, 1, 1, 1, 1, 1],
                      top_p=[1, 1, 1, nan, 1, -0.5, 1, 1, 1, 1], min_p=[0, 0, 0, 0, nan, 0, 0, 0, 0, 0])
    assert list(tokens[[0, 1, 2, 3, 4, 6, 7, 8]]) == [-1] * 8
    assert tokens[5] == l[5].argmax().item() and tokens[9] >= 0
    check(cuda_lib, l[9:], [0.5])


def test_temperatures_far_from_one(cuda_lib):
    B = 8
    l, u = rows(B, 3000, 4)
    for t in (1e-45, 1e-38, 1e-30, 1e-10, 1e-4):  # the largest alone
        tokens, lps = run(cuda_lib, l, u, temperature=[t] * B)
        assert (tokens == l.argmax(1).cpu().numpy()).all() and (lps == 0).all()
    check(cuda_lib, l, u, temperature=[1e4] * B)
    check(cuda_lib, l, u, temperature=[3e38] * B)
    big = l * 1e37
    check(cuda_lib, big, u, temperature=[1e37] * B, top_p=[0.9] * B)
    check(cuda_lib, big, u, temperature=[3e38] * B)
    check(cuda_lib, l * 1e-30, u, temperature=[1e-30] * B, min_p=[0.01] * B)
    check(cuda_lib, l + 1000, u, top_p=[0.9] * B)  # fp32 holds only steps of 2^-14 there


def test_far_tail(cuda_lib):
    """Cuts among tokens that weigh next to nothing: counts go on below what sums can see."""
    B, V = 6, 20000
    l = torch.linspace(0, -150, V, device=DEV).repeat(B, 1)
    l = l[:, torch.randperm(V, generator=torch.Generator().manual_seed(1)).to(DEV)].contiguous()
    u = np.linspace(0.05, 0.95, B)
    check(cuda_lib, l, u, top_k=[19000] * B)
    check(cuda_lib, l, u, top_k=[5000] * B, top_p=[0.99999] * B)
    check(cuda_lib, l, u, min_p=[1e-20] * B)
    check(cuda_lib, l, u, min_p=[1e-38] * B, top_k=[15000] * B, top_p=[0.5] * B)


def test_a_row_is_the_same_everywhere(cuda_lib):
    """One row's token and logprob, wherever it stands, however many rows there are, run after run."""
    l, u = rows(1, 90001, 6)
    s = {"temperature": [0.9], "top_p": [0.97], "top_k": [3000]}
    one = run(cuda_lib, l, u, **s)
    for B in (1, 2, 37, 400):
        got = run(cuda_lib, l.repeat(B, 1), u.repeat(B), **{n: v * B for n, v in s.items()})
        assert (got[0] == one[0][0]).all() and (got[1] == one[1][0]).all()


def test_many_rows(cuda_lib):
    B = 70000  # more rows than a grid's second axis holds
    l, u = rows(B, 12, 1)
    tokens, _ = run(cuda_lib, l, u)
    cum = torch.softmax(l.double(), 1).cumsum(1)
    want = (cum <= u.double()[:, None]).sum(1).clamp(max=11)
    near = (cum - u.double()[:, None]).abs().min(1).values < 2.0 ** -28
    assert (torch.tensor(tokens, device=DEV).long() == want)[~near].all() and near.sum() < 10


def test_rows_behind_the_last_stay(cuda_lib):
    l, u = rows(5, 100, 3)
    tokens, lps = torch.full((9,), -7, dtype=I32, device=DEV), torch.full((9,), 5.0, device=DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    cuda_lib.sample_tokens(l, u, tokens, status, logprobs=lps)
    assert (tokens[5:] == -7).all() and (lps[5:] == 5).all() and (tokens[:5] >= 0).all()
    again = torch.empty(5, dtype=I32, device=DEV)
    cuda_lib.sample_tokens(l, u, again, status)  # without logprobs
    assert torch.equal(again, tokens[:5])
    n = cuda_lib.lib().pqe_kernel_launches()
    cuda_lib.sample_tokens(l[:0], u[:0], again[:0], status)
    assert cuda_lib.lib().pqe_kernel_launches() == n


def test_in_a_graph_and_on_two_streams(cuda_lib):
    B, V = 20, 40000
    data = [rows(B, V, s) for s in (1, 2, 3)]
    st = settings(B, 1)
    dev = {n: torch.tensor(v, dtype=I32 if n == "top_k" else F32, device=DEV) for n, v in st.items()}
    status = torch.zeros(1, dtype=I32, device=DEV)
    outs = [torch.empty(B, dtype=I32, device=DEV) for _ in range(2)]
    ins = [[t.clone() for t in data[i]] for i in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i, s in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            cuda_lib.sample_tokens(*ins[i], outs[i], status, **dev)
        graphs.append(g)
    for a, b in zip(ins[0], data[2]):
        a.copy_(b)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, d in zip(outs, (data[2], data[1])):
        want, _ = run(cuda_lib, *d, **st)
        assert (o.cpu().numpy() == want).all()


def test_long_strides(cuda_lib):
    """Rows whose offsets pass 32 bits."""
    V, stride = 5000, 1 << 30
    buf = torch.empty(2 * stride + V, dtype=torch.bfloat16, device=DEV)
    l = torch.as_strided(buf, (3, V), (stride, 1))
    src, u = rows(3, V, 9, torch.bfloat16)
    l.copy_(src)
    check(cuda_lib, l, u, **settings(3, 4))
