"""Plain 64-bit statements of the attention-side operators, from pqe.h: the MXFP4
quantiser, the cache's byte layout, attention and the residual norm. torch on any
device, float64; nothing of the library is used."""
from __future__ import annotations

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def mxfp4(x: torch.Tensor):
    """x [..., d] -> codes [..., d] and E8M0 bytes [..., d/32] (int64): X = 2^(floor(log2 amax) - 2), nearest code, ties to the
    even one, 255 and zero codes for a block with a value that is not finite."""
    b = x.double().unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1)
    a = torch.where(bad.unsqueeze(-1), 0.0, b.abs())
    amax = a.amax(-1)
    e = torch.where(amax == 0, 0, torch.frexp(amax).exponent.long() - 1 - 2 + 127).clamp(0, 254)
    r = a * pow2(127 - e).unsqueeze(-1)
    order = [0, 2, 4, 6, 1, 3, 5, 7]  # argmin takes the first: even codes win ties
    grid = torch.tensor([E2M1[i] for i in order], dtype=torch.float64, device=x.device)
    code = torch.tensor(order, device=x.device)[(r.unsqueeze(-1) - grid).abs().argmin(-1)]
    code = torch.where(bad.unsqueeze(-1), 0, code + 8 * torch.signbit(b))
    return code.flatten(-2), torch.where(bad, 255, e)


def pow2(n: torch.Tensor) -> torch.Tensor:
    return ((n.long() + 1023) << 52).view(torch.float64)


def values(code: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    tab = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=code.device)
    s = torch.where(scale == 255, float("nan"), pow2(scale.long() - 127))
    return (tab[code.long()].unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def addresses(slots, h, page_size, n_kv, d):
    """Byte addresses, in a cache without gaps between pages, of head h's parts of the tokens at slots [n]:
    K code bytes [n, d], K scales [n, d/32], V code bytes, V scales; element e of a row uses the low nibble if even."""
    slots = slots.long()
    at = slots % page_size
    base = ((slots // page_size * n_kv + h) * (page_size // 16) + at // 16) * 17 * d
    e = torch.arange(d, device=slots.device)
    g = torch.arange(d // 32, device=slots.device)
    tok = (at % 16)[:, None]
    G, el = e // 32, e % 32
    t, j = tok % 8 // 2, tok % 2 + tok // 8 * 2
    base = base[:, None]
    return (base + tok * (d // 2) + el // 8 * (d // 8) + 4 * G + el % 8 // 2,
            base + 16 * d + tok * (d // 32) + g,
            base + 8 * d + G // 2 * 512 + (4 * (el // 4) + t) * 16 + 4 * j + G % 2 * 2 + el % 4 // 2,
            base + 16 * d + d // 2 + t * (d // 8) + g * 4 + j)


def put(flat, slots, k, v, page_size):
    """Write quantised rows k, v [n, n_kv, d] into the bytes `flat` (uint8) at distinct slots."""
    n, n_kv, d = k.shape
    for h in range(n_kv):
        adr = addresses(slots, h, page_size, n_kv, d)
        for x, ca, sa in ((k, adr[0], adr[1]), (v, adr[2], adr[3])):
            code, scale = mxfp4(x[:, h])
            flat[ca[:, ::2]] = (code[:, ::2] | code[:, 1::2] << 4).to(torch.uint8)
            flat[sa] = scale.to(torch.uint8)


def get(flat, slots, page_size, n_kv, d):
    """Values (float64) of the tokens at slots: k, v [n, n_kv, d]."""
    out = []
    nib = 4 * (torch.arange(d, device=flat.device) % 2)
    for h in range(n_kv):
        ka, ks, va, vs = addresses(slots, h, page_size, n_kv, d)
        out.append([values((flat[c].long() >> nib) & 15, flat[s].long()) for c, s in ((ka, ks), (va, vs))])
    return torch.stack([o[0] for o in out], 1), torch.stack([o[1] for o in out], 1)


def attend(q, ms, lens, kv, scale, causal=True, window=0):
    """q [total, n_q, d]; kv[b] = (k, v) [len_b, n_kv, d] float64. Returns out, A = sum_j p_j |v_j| and lse, in float64.
    A masked token's K and V reach nothing; a query that sees nothing gives zeros and -inf."""
    outs, absolute, lses, start = [], [], [], 0
    for m, n, (k, v) in zip(ms, lens, kv):
        qq = q[start:start + m].double()
        start += m
        n_q, d = qq.shape[1:]
        n_kv = k.shape[1]
        pos = n - m + torch.arange(m, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        see = (j <= pos) if causal else (j < n).expand(m, n)
        if window:
            see = see & (j > pos - window)
        z = torch.einsum("mhgd,jhd->hgmj", qq.view(m, n_kv, n_q // n_kv, d), k) * scale
        z = torch.where(see, z, float("-inf"))
        top = z.amax(-1, keepdim=True) if n else torch.full_like(z[..., :1].sum(-1, keepdim=True), float("-inf"))
        top = torch.where(top == float("-inf"), 0.0, top)
        p = torch.where(see, torch.exp(z - top), 0.0)
        l = p.sum(-1, keepdim=True)
        p = torch.where(l == 0, 0.0, p / l)
        # a masked token contributes nothing, not 0 * NaN
        o = torch.zeros((n_kv, n_q // n_kv, m, d), dtype=torch.float64, device=q.device)
        a = torch.zeros_like(o)
        bad = ~torch.isfinite(v)
        vf = torch.where(bad, 0.0, v)
        o += torch.einsum("hgmj,jhd->hgmd", p, vf)
        a += torch.einsum("hgmj,jhd->hgmd", p, vf.abs())
        for t in bad.flatten(1).any(1).nonzero()[:, 0].tolist():
            o = torch.where(see[:, t][None, None, :, None] & bad[t][:, None, None], float("nan"), o)
        outs.append(o.permute(2, 0, 1, 3).reshape(m, n_q, d))
        absolute.append(a.permute(2, 0, 1, 3).reshape(m, n_q, d))
        lses.append(torch.where(l == 0, float("-inf"), top + torch.log(l))[..., 0].permute(2, 0, 1).reshape(m, n_q))
    return torch.cat(outs), torch.cat(absolute), torch.cat(lses)


def norm(x, r, w, eps):
    """h and y of add_rms_norm in float64."""
    h = x.double() + (0 if r is None else r.double())
    return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()
