"""The decoder layer of examples/decoder_layer.py: the same tokens as one prompt, and as a prompt
with single tokens after it, and the attention half against the 64-bit statement on what the cache
holds."""
import os
import sys

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _layer(**kw):
    import decoder_layer
    layer = decoder_layer.DecoderLayer(H=512, n_q=10, n_kv=2, d=64, E=8, I=128, k=2, n_pages=40, page_size=16, max_tokens=512, **kw)
    return layer, decoder_layer.Sequences(2, 40, 16, 300)


def _inputs(n):
    g = torch.Generator(device="cuda").manual_seed(5)
    return [torch.randn((n, 512), generator=g, device="cuda").bfloat16() for _ in range(2)]


@pytest.mark.parametrize("window", [0, 40])
def test_prompt_at_once_and_token_by_token(cuda_lib, window):
    """Tokens see the same cache either way. The products' sums may run in another order for another number of rows, which can
    move a K or V code by one step now and then: the attention's results are held to 2^-5 of their size, not to their last
    bits."""
    lens, tail = [120, 75], 6
    n = sum(lens)
    delta, residual = _inputs(n)
    first = [0, lens[0]]
    layer, seqs = _layer(window=window)
    res = residual.clone()
    whole = layer.attention(delta, res, seqs.extend(lens))
    layer2, seqs2 = _layer(window=window)
    rows = torch.cat([torch.arange(f, f + m - tail) for f, m in zip(first, lens)]).cuda()
    r = residual[rows].contiguous()
    part = layer2.attention(delta[rows].contiguous(), r, seqs2.extend([m - tail for m in lens]))
    got = torch.empty_like(whole)
    got[rows] = part
    for i in range(tail):
        rows = torch.tensor([f + m - tail + i for f, m in zip(first, lens)]).cuda()
        r = residual[rows].contiguous()
        got[rows] = layer2.attention(delta[rows].contiguous(), r, seqs2.extend([1, 1]))
        assert torch.equal(r, res[rows])
    off = (got.double() - whole.double()).norm(dim=1) / whole.double().norm(dim=1)
    assert off.max().item() < 2.0 ** -5
    assert layer.status.item() == 0 and layer2.status.item() == 0
    # the expert half takes it from there
    out = layer.experts(whole, res)
    assert torch.isfinite(out).all() and out.abs().sum() > 0
    layer.moe.close()
    layer2.moe.close()


def test_attention_half_against_the_statement(cuda_lib):
    lens = [90, 33]
    delta, residual = _inputs(sum(lens))
    layer, seqs = _layer()
    step = seqs.extend(lens)
    r = residual.clone()
    out = layer.attention(delta, r, step)
    # the same norm and projection, then attention in 64 bits over the cache's values
    codes = torch.empty((sum(lens), 512), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(sum(lens), device="cuda")
    cuda_lib.add_rms_norm(delta, residual, layer.norm1, 1e-6, None, None, codes, scale)
    heads = layer.project(codes, scale).view(-1, 14, 64)
    slots = step["slots"].split(lens)
    kv = [ref.get(layer.cache_mem, s, 16, 2, 64) for s in slots]
    for s, (k, v), rows in zip(slots, kv, heads.split(lens)):
        assert torch.equal(k, ref.values(*ref.mxfp4(rows[:, 10:12])))
        assert torch.equal(v, ref.values(*ref.mxfp4(rows[:, 12:])))
    o, a, _ = ref.attend(heads[:, :10], lens, lens, kv, layer.scale)
    want = o.flatten(1) @ layer.wo.double().T
    # attention's own bound (u |o| + 2^-9 A, u = 2^-8) through the product's rows, and the product's bf16 result
    bound = (2.0 ** -8 * 1.01 * o.abs() + 2.0 ** -9 * a).flatten(1) @ layer.wo.double().abs().T + 2.0 ** -8 * 1.01 * want.abs()
    assert not ((out.double() - want).abs() > bound).any()
    layer.moe.close()


def test_pages_go_back(cuda_lib):
    layer, seqs = _layer()
    step = seqs.extend([100, 20])
    assert len(seqs.free) == 40 - 7 - 2 and len(step["slots"].unique()) == 120
    seqs.release(0)
    assert len(seqs.free) == 38 and seqs.lens == [0, 20]
    layer.moe.close()


def test_example_runs(cuda_lib, capsys):
    import decoder_layer
    assert decoder_layer.main(["--sequences", "3", "--prompt", "70", "--steps", "4"])["ok"]
