"""The decoder layer of examples/decoder_layer.py with block-scaled projections, and the step from its last hidden state to the
next token: each part against the 64-bit statement on what the part before it gave."""
import os
import sys

import pytest
import torch

import attention_ref as ref
import sampling_ref
import test_gpu_fp8_block as products

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _layer(**kw):
    import decoder_layer
    layer = decoder_layer.DecoderLayer(H=512, n_q=10, n_kv=2, d=64, E=8, I=128, k=2, n_pages=40, page_size=16, max_tokens=512, block_fp8=True, **kw)
    return layer, decoder_layer.Sequences(2, 40, 16, 300)


def _inputs(n, H=512):
    g = torch.Generator(device="cuda").manual_seed(5)
    return [torch.randn((n, H), generator=g, device="cuda").bfloat16() for _ in range(2)]


def test_attention_half_part_by_part(cuda_lib):
    lens = [90, 33]
    T = sum(lens)
    delta, residual = _inputs(T)
    layer, seqs = _layer()
    step = seqs.extend(lens)
    r = residual.clone()
    got = layer.attention(delta, r, step)
    # the norm's codes and the projection
    codes, scale = torch.empty((T, 512), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((T, 4), device="cuda")
    cuda_lib.add_rms_norm(delta, residual, layer.norm1, 1e-6, None, None, codes, scale, cuda_lib.PQE_Q8_B128)
    heads = layer.qkv(codes, scale, layer.status)
    products.check(heads, codes, scale, layer.qkv.q, layer.qkv.scale)
    heads = heads.view(T, 14, 64)
    kv = [ref.get(layer.cache_mem, s, 16, 2, 64) for s in step["slots"].split(lens)]
    for (k, v), rows in zip(kv, heads.split(lens)):
        assert torch.equal(k, ref.values(*ref.mxfp4(rows[:, 10:12]))) and torch.equal(v, ref.values(*ref.mxfp4(rows[:, 12:])))
    # attention over what the cache holds, within its own bound
    out = torch.empty((T, 10, 64), dtype=torch.bfloat16, device="cuda")
    cuda_lib.kv_paged_attention(layer.cache, heads[:, :10], step["q_offsets"], step["kv_lens"], step["block_table"], step["max_q"], layer.scale,
                                out, layer.ws, layer.status)
    o, a, _ = ref.attend(heads[:, :10], lens, lens, kv, layer.scale)
    assert not ((out.double() - o).abs() > 2.0 ** -8 * 1.01 * o.abs() + 2.0 ** -9 * a).any()
    # its codes, bit for bit, and the output projection
    codes, scale = torch.empty((T, 640), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((T, 5), device="cuda")
    cuda_lib.fp8_block_quantize(out.flatten(1), codes, scale)
    want_codes, want_scale = products.tiles(out.flatten(1), 1)
    assert torch.equal(codes.cpu().view(torch.uint8), want_codes.view(torch.uint8)) and torch.equal(scale.cpu(), want_scale)
    products.check(got, codes, scale, layer.out.q, layer.out.scale)
    assert layer.status.item() == 0
    moe = layer.experts(got, r)
    assert torch.isfinite(moe).all() and moe.abs().sum() > 0
    layer.moe.close()


def test_prompt_at_once_and_token_by_token(cuda_lib):
    """Tokens see the same cache either way; products of other numbers of rows round differently in their last bit, which can move a
    code of K, V or an activation by one step now and then: results are held to 2^-4 of their size (E4M3's half step)."""
    lens, tail = [120, 75], 6
    n = sum(lens)
    delta, residual = _inputs(n)
    first = [0, lens[0]]
    layer, seqs = _layer()
    res = residual.clone()
    whole = layer.attention(delta, res, seqs.extend(lens))
    layer2, seqs2 = _layer()
    rows = torch.cat([torch.arange(f, f + m - tail) for f, m in zip(first, lens)]).cuda()
    got = torch.empty_like(whole)
    got[rows] = layer2.attention(delta[rows].contiguous(), residual[rows].contiguous(), seqs2.extend([m - tail for m in lens]))
    for i in range(tail):
        rows = torch.tensor([f + m - tail + i for f, m in zip(first, lens)]).cuda()
        got[rows] = layer2.attention(delta[rows].contiguous(), residual[rows].contiguous(), seqs2.extend([1, 1]))
    off = (got.double() - whole.double()).norm(dim=1) / whole.double().norm(dim=1)
    assert off.max().item() < 2.0 ** -4 and layer.status.item() == 0 and layer2.status.item() == 0
    layer.moe.close()
    layer2.moe.close()


@pytest.mark.parametrize("T,V", [(1, 1000), (9, 5003), (64, 32000)])
def test_from_the_last_state_to_the_next_token(cuda_lib, T, V):
    import decoder_layer
    last = decoder_layer.Vocabulary(512, V, seed=3)
    delta, residual = _inputs(T)
    g = torch.Generator(device="cuda").manual_seed(T)
    u = torch.rand(T, generator=g, device="cuda")
    t = torch.rand(T, generator=g, device="cuda").round() * 0.7
    top_k = torch.randint(0, 60, (T,), generator=g, device="cuda", dtype=torch.int32)
    top_p = 0.5 + 0.5 * torch.rand(T, generator=g, device="cuda")
    min_p = 0.01 * torch.rand(T, generator=g, device="cuda")
    tokens, lps = last(delta, residual, u, temperature=t, top_k=top_k, top_p=top_p, min_p=min_p)
    codes, scale = torch.empty((T, 512), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((T, 4), device="cuda")
    cuda_lib.add_rms_norm(delta, residual, last.norm, 1e-6, None, None, codes, scale, cuda_lib.PQE_Q8_B128)
    logits = last.logits(delta, residual)
    products.check(logits, codes, scale, last.head.q, last.head.scale)
    l = logits.cpu().double().numpy()
    for b in range(T):
        token, lp, near = sampling_ref.draw(l[b], float(u[b]), t=float(t[b]), k=int(top_k[b]), p=float(top_p[b]), mp=float(min_p[b]))
        assert near > 2.0 ** -30 and tokens[b].item() == token and abs(lps[b].item() - lp) <= 2.0 ** -22 * (8 + abs(lp))
    assert last.status.item() == 0


def test_the_step_in_a_graph(cuda_lib):
    """Norm, product and sampling captured once and replayed on new states: the tokens of the same calls made one by one."""
    import decoder_layer
    last = decoder_layer.Vocabulary(512, 7001, seed=4)
    T = 12
    delta, residual = _inputs(T)
    u = torch.rand(T, device="cuda")
    k = torch.full((T,), 20, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = last(delta, residual, u, top_k=k)
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        delta.copy_(torch.randn(delta.shape, generator=g, device="cuda"))
        u.copy_(torch.rand(T, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = last(delta, residual, u, top_k=k)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_example_tokens(cuda_lib):
    """The loop twice: the same tokens, all of the vocabulary."""
    import decoder_layer
    a, b = (decoder_layer.main(["--sequences", "3", "--prompt", "70", "--steps", "4", "--vocabulary", "2003"]) for _ in range(2))
    assert a["ok"] and torch.equal(a["tokens"], b["tokens"]) and a["tokens"].shape == (3, 5) and int(a["tokens"].max()) < 2003
