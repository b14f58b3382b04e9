"""One decoder layer in a serving loop: attention over a 4-bit paged KV cache, then the paged MoE expert layer.

A step takes the tokens that are new (prompts, or one token a sequence) through

    add_rms_norm        residual addition and norm, E4M3 codes with a scale a row
    q|k|v projection    on those codes (a plain product; the library has none of its own)
    kv_cache_write      K and V rows, quantised into the sequences' pages
    kv_paged_attention  over everything cached so far
    output projection
    add_rms_norm        residual addition and norm, bf16 for the expert layer
    PagedMoELayer.step  route, permute, refill, expert FFN, combine

    python examples/decoder_layer.py [--sequences 8] [--prompt 300] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import paged_quantized_expert_gb300 as pqe  # noqa: E402


class Sequences:
    """The page tables of a set of sequences over one cache's pages, and what a step of new tokens needs of them."""

    def __init__(self, n: int, n_pages: int, page_size: int, max_tokens: int, device="cuda"):
        self.page_size, self.device = page_size, device
        self.free = list(range(n_pages - 1, -1, -1))
        self.tables: list[list[int]] = [[] for _ in range(n)]
        self.lens = [0] * n
        self.block_table = torch.zeros((n, -(-max_tokens // page_size)), dtype=torch.int32)

    def extend(self, new: list[int]) -> dict:
        """Room for new[b] more tokens of each sequence: their slots, and the step's offsets, lengths and table."""
        slots = []
        for b, n in enumerate(new):
            while len(self.tables[b]) * self.page_size < self.lens[b] + n:
                self.tables[b].append(self.free.pop())
                self.block_table[b, len(self.tables[b]) - 1] = self.tables[b][-1]
            slots += [self.tables[b][i // self.page_size] * self.page_size + i % self.page_size
                      for i in range(self.lens[b], self.lens[b] + n)]
            self.lens[b] += n
        offsets = [sum(new[:b]) for b in range(len(new) + 1)]
        dev = self.device
        return {"slots": torch.tensor(slots, dtype=torch.int64, device=dev),
                "q_offsets": torch.tensor(offsets, dtype=torch.int32, device=dev),
                "kv_lens": torch.tensor(self.lens, dtype=torch.int32, device=dev),
                "block_table": self.block_table.to(dev), "max_q": max(new), "total": offsets[-1]}

    def release(self, b: int):
        """Give a sequence's pages back."""
        self.free += self.tables[b]
        self.tables[b], self.lens[b] = [], 0


class DecoderLayer:
    """Random weights of one decoder layer, its KV cache and its expert layer."""

    def __init__(self, H=2048, n_q=16, n_kv=4, d=128, E=16, I=512, k=4, n_pages=1024, page_size=64, max_tokens=4096, window=0,
                 seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.H, self.n_q, self.n_kv, self.d, self.window, self.device = H, n_q, n_kv, d, window, device
        self.scale = d ** -0.5
        self.norm1 = (1 + 0.1 * rand(H)).bfloat16()
        self.norm2 = (1 + 0.1 * rand(H)).bfloat16()
        w = rand((n_q + 2 * n_kv) * d, H) * H ** -0.5
        self.wqkv = torch.empty(w.shape, dtype=torch.uint8, device=device)
        self.wqkv_scale = torch.empty(w.shape[0], dtype=torch.float32, device=device)
        pqe.pqe_quantize_fp8_rows(w, self.wqkv, self.wqkv_scale)
        self.wo = (rand(H, n_q * d) * (n_q * d) ** -0.5).bfloat16()
        self.w_router = rand(E, H) * 0.02
        stride = pqe.slot_stride(H, I)
        host = torch.zeros((E, stride), dtype=torch.uint8).pin_memory()
        page = torch.zeros(stride, dtype=torch.uint8, device=device)
        for e in range(E):
            pqe.pqe_pack_fp8_page(rand(2 * I, H) * 0.02, rand(H, I) * 0.02, H, I, page)
            host[e].copy_(page)
        self.moe = pqe.PagedMoELayer(E, H, I, k, E, E, max_tokens, host, [pqe.page_bytes(pqe.PQE_FMT_FP8, H, I)] * E)
        self.cache_mem, self.cache = pqe.alloc_kv_cache(n_pages, page_size, n_kv, d, device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.ws = torch.empty(0, dtype=torch.uint8, device=device)

    def project(self, codes, scale):
        """x W^T of E4M3 codes with row scales on both sides. E4M3 values are exact in bf16; a library product that takes the
        codes and scales as they are does the same."""
        y = codes.bfloat16() @ self.wqkv.view(torch.float8_e4m3fn).bfloat16().T
        return (y.float() * scale[:, None] * self.wqkv_scale).bfloat16()

    def attention(self, delta, residual, step):
        """norm, projection, cache write, attention, output projection; residual += delta in place. Returns the new delta."""
        T = step["total"]
        codes = torch.empty((T, self.H), dtype=torch.float8_e4m3fn, device=self.device)
        scale = torch.empty(T, dtype=torch.float32, device=self.device)
        pqe.add_rms_norm(delta, residual, self.norm1, 1e-6, residual, None, codes, scale, pqe.PQE_Q8_ROW)
        heads = self.project(codes, scale).view(T, self.n_q + 2 * self.n_kv, self.d)
        q, k, v = heads.split([self.n_q, self.n_kv, self.n_kv], 1)  # views into the fused rows
        pqe.kv_cache_write(self.cache, k, v, step["slots"], self.status)
        need = pqe.kv_paged_attention_workspace_size(len(step["kv_lens"]), T, step["max_q"], self.n_q, self.n_kv, self.d)
        if self.ws.numel() < need:
            self.ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        out = torch.empty((T, self.n_q, self.d), dtype=torch.bfloat16, device=self.device)
        pqe.kv_paged_attention(self.cache, q, step["q_offsets"], step["kv_lens"], step["block_table"], step["max_q"], self.scale,
                               out, self.ws, self.status, window=self.window)
        return out.flatten(1) @ self.wo.T

    def experts(self, delta, residual):
        """norm and expert layer; residual += delta in place. Returns the new delta."""
        y = torch.empty_like(residual)
        pqe.add_rms_norm(delta, residual, self.norm2, 1e-6, residual, y)
        out = torch.empty_like(y)
        self.moe.step(y, out, y.shape[0], w_router=self.w_router)
        return out

    def __call__(self, delta, residual, step):
        delta = self.attention(delta, residual, step)
        return self.experts(delta, residual)


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    tokens = a.sequences * (a.prompt + a.steps)
    layer = DecoderLayer(n_pages=a.sequences * (-(-(a.prompt + a.steps) // 64)), max_tokens=max(a.sequences * a.prompt, 64))
    seqs = Sequences(a.sequences, layer.cache.n_pages, 64, a.prompt + a.steps)
    g = torch.Generator(device="cuda").manual_seed(1)

    def step(new):
        s = seqs.extend([new] * a.sequences)
        delta = torch.randn((s["total"], layer.H), generator=g, device="cuda").bfloat16()
        residual = torch.randn((s["total"], layer.H), generator=g, device="cuda").bfloat16()
        return layer(delta, residual, s)

    step(a.prompt)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        out = step(1)
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(a.steps, 1)
    ok = layer.status.item() == 0 and bool(torch.isfinite(out).all())
    print(f"{tokens} tokens through one layer; a step of {a.sequences} tokens takes {t * 1e6:.0f} us; "
          f"{'ok' if ok else 'FAILED'} (status {layer.status.item()})")
    layer.moe.close()
    return {"ok": ok, "step_s": t}


if __name__ == "__main__":
    sys.exit(0 if main()["ok"] else 1)
