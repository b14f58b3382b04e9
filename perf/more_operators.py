"""Cases of what stands between a decoder layer's parts and behind its last one: block-scaled FP8 products, and sampling.

Three operators, each in a plain form (torch, 32 bits; 64 for sampling) and as the library's calls (`own`):

  quant   bf16 rows to E4M3 codes with one scale for each 128 values, alone or out of the residual norm
  matmul  x W^T of E4M3 codes: x with a scale for each 128 values of a row, W with one for each 128 x 128 tile
  sample  the next token of each row of logits from a given uniform number: temperature, top-k, min-p, top-p
"""
import math

import torch

own = False

DEV = "cuda"


# ---- the cases -----------------------------------------------------------------------------------


def listed():
    return [
        # one user's next token through the q|k|v projection (20 + 2 * 4 heads of 128): latency is all
        {"name": "mm_one_qkv", "op": "matmul", "M": 1, "N": 3584, "K": 2048, "out": "bf16"},
        # a decode step's output projection
        {"name": "mm_step_64", "op": "matmul", "M": 64, "N": 2048, "K": 2560, "out": "bf16"},
        # a decode step's logits over the vocabulary: the weights' bytes are all
        {"name": "mm_vocab_64", "op": "matmul", "M": 64, "N": 131072, "K": 2048, "out": "fp32"},
        # odd sizes everywhere: a last block of 16 along K, columns that end inside a tile, rows that end inside one
        {"name": "mm_ragged_333", "op": "matmul", "M": 333, "N": 1003, "K": 1040, "out": "fp32"},
        # a prompt through the q|k|v projection
        {"name": "mm_prompt_4099", "op": "matmul", "M": 4099, "N": 3584, "K": 2048, "out": "bf16"},
        # a module batch of prompts
        {"name": "mm_batch_16384", "op": "matmul", "M": 16384, "N": 4096, "K": 2560, "out": "bf16"},
        # a decode step's attention output before its projection
        {"name": "quant_step_64", "op": "quant", "T": 64, "H": 2560, "norm": False},
        # a module batch's residual norm, with codes for the projection behind it
        {"name": "quant_norm_16384", "op": "quant", "T": 16384, "H": 2048, "norm": True},
        # one user's next token, nucleus sampling
        {"name": "sample_one", "op": "sample", "B": 1, "V": 131072, "type": "fp32", "mix": "top_p", "peak": 1.0},
        # a serving step: each user has settings of their own, some greedy
        {"name": "sample_64_mixed", "op": "sample", "B": 64, "V": 131072, "type": "fp32", "mix": "mixed", "peak": 1.0},
        # bf16 logits (many equal ones) of an odd vocabulary, the nearly flat rows of an early checkpoint
        {"name": "sample_33_ties", "op": "sample", "B": 33, "V": 100003, "type": "bf16", "mix": "mixed", "peak": 0.0},
        # many rows of a small vocabulary, the whole distribution
        {"name": "sample_512_all", "op": "sample", "B": 512, "V": 32000, "type": "fp32", "mix": "all", "peak": 0.5},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "quant", "sample", "sample"])
    if op == "quant":
        return {"op": "quant", "T": _log(rng, 1, 16384), "H": 32 * _log(rng, 4, 64), "norm": rng.random() < 0.5}
    if op == "sample":
        B = _log(rng, 1, 512)
        return {"op": "sample", "B": B, "V": _log(rng, 1000, min(200_000, 16_000_000 // B)), "type": rng.choice(["fp32", "fp32", "bf16"]),
                "mix": rng.choice(["mixed", "mixed", "all", "top_p", "top_k"]), "peak": rng.choice([0.0, 0.5, 1.0])}
    K = 16 * _log(rng, 16, 512)
    M = _log(rng, 1, 16384)
    most = min(131072, 268_435_456 // K, int(0.8 * 16384 * 4096 * 2560 / (M * K)), 67_000_000 // M)
    N = _log(rng, 64, most)
    return {"op": "matmul", "M": M, "N": N - N % rng.choice([1, 8, 64, 128]) or 64, "K": K, "out": rng.choice(["bf16", "bf16", "fp32"])}


def work(case):
    c = case
    if c["op"] == "quant":
        n, blocks = c["T"] * c["H"], -(-c["H"] // 128)
        # rows read, codes and scales written; the norm reads a residual and its weight too and writes the new residual
        return {"bytes": 3 * n + 4 * c["T"] * blocks + (4 * n + 2 * c["H"] if c["norm"] else 0), "flops": (8 if c["norm"] else 3) * n}
    if c["op"] == "sample":
        # logits read once; an exponential and two additions a value
        return {"bytes": c["B"] * c["V"] * (4 if c["type"] == "fp32" else 2) + 28 * c["B"], "flops": 3 * c["B"] * c["V"]}
    M, N, K = c["M"], c["N"], c["K"]
    kb = -(-K // 128)
    held = M * K + N * K + 4 * kb * (M + -(-N // 128))
    return {"bytes": held + M * N * (2 if c["out"] == "bf16" else 4), "flops": 2 * M * N * K}


# ---- inputs --------------------------------------------------------------------------------------


def _pad(x, rows, cols):
    """x with zeros behind it, up to whole multiples of `rows` and `cols`."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def _codes(x, rows):
    """fp32 [n, k] -> E4M3 codes [n, k], fp32 scales [ceil(n / rows), ceil(k / 128)]: one for each rows x 128 tile."""
    n, k = x.shape
    tiles = _pad(x, rows, 128).unflatten(0, (-1, rows)).unflatten(2, (-1, 128))
    amax = tiles.abs().amax((1, 3))
    scale = torch.where(amax == 0, 1.0, amax / 448)
    q = (tiles / scale[:, None, :, None]).clamp(-448, 448)
    return q.flatten(2).flatten(0, 1)[:n, :k].contiguous().to(torch.float8_e4m3fn), scale


def _settings(g, c):
    """Sampling settings of each row, as users send them."""
    B = c["B"]
    pick = lambda values, dtype=torch.float32: torch.tensor(values, dtype=dtype, device=DEV)[  # noqa: E731
        torch.randint(0, len(values), (B,), generator=g, device=DEV)]
    s = {"temperature": pick([0.6, 0.7, 1.0, 1.0, 1.3]), "top_k": pick([0], torch.int32), "top_p": pick([1.0]), "min_p": pick([0.0])}
    if c["mix"] in ("top_p", "mixed"):
        s["top_p"] = pick([0.9, 0.95, 0.5, 1.0] if c["mix"] == "mixed" else [0.8, 0.9, 0.95])
    if c["mix"] in ("top_k", "mixed"):
        s["top_k"] = pick([0, 0, 20, 50, 1000] if c["mix"] == "mixed" else [1, 20, 40, 100, 1000], torch.int32)
    if c["mix"] == "mixed":
        s["min_p"] = pick([0.0, 0.0, 0.05, 0.001])
        s["temperature"] = pick([0.0, 0.6, 0.7, 1.0, 1.0, 1.3])
    return s


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    if c["op"] == "quant":
        T, H = c["T"], c["H"]
        # activations with a few channels far larger than the rest
        s = {"case": c, "x": (randn(T, H) * (1 + 20 * (torch.rand(H, generator=g, device=DEV) < 0.01))).bfloat16()}
        return {**s, "r": (4 * randn(T, H)).bfloat16(), "w": (1 + 0.2 * randn(H)).bfloat16(), "eps": 1e-6} if c["norm"] else s
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if c["op"] == "sample":
        B, V = c["B"], c["V"]
        logits = 2.5 * randn(B, V)
        # a trained model's rows: a few tokens well above all others, most far below
        logits += c["peak"] * (12 - 4 * torch.rand((B, V), generator=g, device=DEV).log2().neg()).clamp(min=-8) * (
            torch.rand((B, V), generator=g, device=DEV) < 0.001)
        return {"case": c, "logits": logits if c["type"] == "fp32" else logits.bfloat16(), "u": torch.rand(B, generator=g, device=DEV),
                **_settings(g, c), "status": status}
    M, N, K = c["M"], c["N"], c["K"]
    xq, xs = _codes(randn(M, K) * (1 + 20 * (torch.rand(K, generator=g, device=DEV) < 0.01)), 1)
    wq, ws = _codes(randn(N, K) * K ** -0.5 * (0.5 + torch.rand((N, 1), generator=g, device=DEV)), 128)
    return {"case": c, "xq": xq, "xs": xs, "wq": wq, "ws": ws, "status": status}


# ---- one pass ------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return _plain_quant(state) if op == "quant" else _plain_matmul(state) if op == "matmul" else _plain_sample(state)


def _own(s, op):
    import paged_quantized_expert_gb300 as pqe

    c = s["case"]
    if op == "matmul":
        out = torch.empty((c["M"], c["N"]), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
        pqe.fp8_block_matmul(s["xq"], s["xs"], s["wq"], s["ws"], out, s["status"])
        return out
    if op == "sample":
        tokens = torch.empty(c["B"], dtype=torch.int32, device=DEV)
        logprobs = torch.empty(c["B"], dtype=torch.float32, device=DEV)
        pqe.sample_tokens(s["logits"], s["u"], tokens, s["status"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                          min_p=s["min_p"], logprobs=logprobs)
        return {"tokens": tokens, "logprobs": logprobs}
    T, H = c["T"], c["H"]
    q = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty((T, -(-H // 128)), dtype=torch.float32, device=DEV)
    if not c["norm"]:
        pqe.fp8_block_quantize(s["x"], q, scale)
        return {"q": q, "scale": scale}
    res = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    pqe.add_rms_norm(s["x"], s["r"], s["w"], s["eps"], res, None, q, scale, pqe.PQE_Q8_B128)
    return {"res": res, "q": q, "scale": scale}


def _plain_quant(s):
    y = s["x"].float()
    if not s["case"]["norm"]:
        q, scale = _codes(y, 1)
        return {"q": q, "scale": scale}
    h = y + s["r"].float()
    q, scale = _codes(h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["w"].float(), 1)
    return {"res": h.bfloat16(), "q": q, "scale": scale}


def _plain_matmul(s):
    K = s["case"]["K"]
    x = s["xq"].float() * s["xs"].repeat_interleave(128, 1)[:, :K]
    w = s["wq"].float() * s["ws"].repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 0)[: s["case"]["N"]]
    y = torch.matmul(x, w.T)
    return y.bfloat16() if s["case"]["out"] == "bf16" else y


def _plain_sample(s):
    # 64 bits: a token is drawn where a sum over the vocabulary passes a border
    B, V = s["case"]["B"], s["case"]["V"]
    column = lambda t: t.double()[:, None]  # noqa: E731
    l, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    t = column(s["temperature"])
    w = torch.exp((l - l[:, :1]) / torch.where(t == 0, 1, t))
    rank = torch.arange(V, device=DEV)
    k = s["top_k"][:, None]
    k = torch.where((k <= 0) | (k > V), V, k)
    keep = (rank < torch.where(t == 0, 1, k)) & (w >= column(s["min_p"]))
    w = torch.where(keep, w, 0)
    before = torch.cumsum(w, 1) - w
    p = column(s["top_p"])
    w = torch.where((before < p * w.sum(1, keepdim=True)) | (p >= 1) | (rank == 0), w, 0)
    w = torch.empty_like(w).scatter_(1, order, w)  # in the vocabulary's own order
    cum = torch.cumsum(w, 1)
    total = cum[:, -1:]
    token = (cum <= column(s["u"]) * total).sum(1, keepdim=True)
    return {"tokens": token[:, 0].int(), "logprobs": torch.log(w.gather(1, token) / total)[:, 0].float()}


# ---- the definitions in 64 bits ------------------------------------------------------------------


def _exact_sample(s):
    """Row by row, by the definition's own steps: the candidates as a list of indices that each setting shortens."""
    tokens, logprobs = [], []
    for b in range(s["case"]["B"]):
        l = s["logits"][b].double()
        top = l.max()
        t, k, p, m = (s[n][b].item() for n in ("temperature", "top_k", "top_p", "min_p"))
        if t == 0:
            tokens.append((l == top).nonzero()[0, 0])
            logprobs.append(torch.zeros((), dtype=torch.float64, device=DEV))
            continue
        index = torch.sort(-l, stable=True).indices
        if 0 < k < index.numel():
            index = index[:k]
        if m > 0:
            index = index[l[index] - top >= t * math.log(m)]
        w = ((l[index] - top) / t).exp()
        if p < 1:
            n = int((w.cumsum(0) < p * w.sum()).sum()) + 1
            index, w = index[:n], w[:n]
        index, by = torch.sort(index)
        w = w[by]
        cum = w.cumsum(0)
        at = int(torch.searchsorted(cum, s["u"][b].double() * cum[-1], right=True))
        tokens.append(index[at])
        logprobs.append((l[index[at]] - top) / t - cum[-1].log())
    return {"tokens": torch.stack(tokens).int(), "logprobs": torch.stack(logprobs)}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "sample":
        return _exact_sample(s)
    if c["op"] == "quant":
        y = h = s["x"].double()
        if c["norm"]:
            h = y + s["r"].double()
            y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / c["H"] + s["eps"]) * s["w"].double()
        # the codes are what E4M3 can hold of y over the scale: not a value in 64 bits
        scale = torch.stack([b.abs().amax(1) / 448 for b in y.split(128, 1)], 1)
        return {**({"res": h} if c["norm"] else {}), "q": None, "scale": scale}
    if 2 * c["M"] * c["N"] * c["K"] > 2e12:
        return None
    out = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device=DEV)
    for b in range(-(-c["K"] // 128)):
        at = slice(128 * b, 128 * b + 128)
        by_row = s["ws"][:, b].double()[torch.arange(c["N"], device=DEV) // 128]
        out += (s["xq"][:, at].double() @ s["wq"][:, at].double().T) * s["xs"][:, b, None].double() * by_row
    return out
