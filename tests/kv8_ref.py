"""The 8-bit cache operators and the sampler from their definitions, in 64 bits
(torch on whichever device the inputs are on; no code of the library)."""

import math

import numpy as np
import torch

E4M3, INT8 = 0, 1
CODE_MAX = {E4M3: 448.0, INT8: 127.0}


def decode(codes, fmt):
    """uint8 codes -> float64 values, from the formats' definitions."""
    c = codes.to(torch.int64)
    if fmt == INT8:
        return torch.where(c >= 128, c - 256, c).double()
    sign = 1.0 - 2.0 * (c >> 7).double()
    e, m = (c >> 3) & 15, (c & 7).double()
    return sign * torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))


def random_cache(fmt, slots, cap, kvh, d, seed, spread=0.4):
    """A filled cache: dict of the descriptor's fields."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = {"format": fmt, "slots": slots, "ctx_cap": cap, "kv_heads": kvh, "head_dim": d}
    for n in ("K", "V"):
        x = torch.randn(slots, kvh, cap, d, generator=g, device="cuda")
        x *= torch.exp(spread * torch.randn(slots, kvh, cap, 1, generator=g, device="cuda"))
        s = x.abs().amax(-1, keepdim=True) / CODE_MAX[fmt]
        y = x / s
        out[n] = (y.to(torch.float8_e4m3fn) if fmt == E4M3 else y.round().to(torch.int8)).view(torch.uint8)
        out[n + "s"] = s.squeeze(-1).contiguous()
    return out


def append_rows(qkv, qh, kvh, d, pos, norm, wq, wk, eps, inv_freq):
    """(q, k, v, slack): rows [T][heads][d] before rounding, and per (row, head, element) |a| + |b| of
    the rotated pair, which bounds the fp32 error."""
    T = qkv.shape[0]
    x = qkv[:, :(qh + 2 * kvh) * d].double().view(T, qh + 2 * kvh, d)
    q, k, v = x[:, :qh], x[:, qh:qh + kvh], x[:, qh + kvh:]
    if norm:
        r = lambda y, w: y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * (1.0 if w is None else w.double())  # noqa: E731
        q, k = r(q, wq), r(k, wk)
    both = torch.cat([q, k], 1)
    slack = both.abs()
    if inv_freq is not None:
        a, b = both.chunk(2, -1)
        ang = pos.double()[:, None, None] * inv_freq.double()
        both = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
        slack = (a.abs() + b.abs()).repeat(1, 1, 2)
    return both[:, :qh], both[:, qh:], v, slack


def attend(cache, Q, slots, lens, scale, prefix=None):
    """(o, bound): the output in 64 bits, and per element sum_j p_j |v_j| * (relative error a weight may have).

    A weight's own error: it is rounded to 16 bits (2^-11) on the way to the tensor cores, and its score,
    a sum of d products in fp32, may be off by (d + 8) * 2^-24 * scale * sum|q||k| absolute, which moves
    the weight, and in the same way the normalising sum, by that factor; e^x and the sums add 2^-18.
    What is rounded to 16 bits is p_j * (V's scale) in units of at most its largest value of the row.  fp16's
    smallest step is 2^-24, so a weight far below the largest is also off by up to 2^-25 of that largest one:
    2^-25 * max_j (p_j vs_j) * sum_j |code_j| of the output.
    Rows of slot < 0 are None."""
    B, qh, d = Q.shape
    kvh = cache["kv_heads"]
    G = qh // kvh
    out, bound = [], []
    for b in range(B):
        slot, n = int(slots[b]), int(lens[b])
        if slot < 0 or slot >= cache["slots"] or n < 0 or n > cache["ctx_cap"]:
            out.append(None)
            bound.append(None)
            continue
        parts = [(cache, slot, n)]
        if prefix is not None:
            parts.insert(0, prefix)
        codes = torch.cat([decode(c["V"][s, :, :j], c["format"]) for c, s, j in parts], 1).abs().sum(1)
        vs = torch.cat([c["Vs"][s, :, :j].double() for c, s, j in parts], 1)
        k, v = (torch.cat([decode(c[m][s, :, :j], c["format"]) * c[m + "s"][s, :, :j].double().unsqueeze(-1)
                           for c, s, j in parts], 1) for m in ("K", "V"))
        q = Q[b].double().view(kvh, G, d)
        if k.shape[1] == 0:
            out.append(torch.zeros(qh, d, dtype=torch.float64, device=Q.device))
            bound.append(torch.zeros(qh, d, dtype=torch.float64, device=Q.device))
            continue
        p = torch.softmax(torch.einsum("hgd,hnd->hgn", q, k) * scale, -1)
        off = torch.einsum("hgd,hnd->hgn", q.abs(), k.abs()).amax(-1, keepdim=True) * scale * (d + 8) * 2.0 ** -24
        out.append(torch.einsum("hgn,hnd->hgd", p, v).reshape(qh, d))
        small = 2.0 ** -25 * (p * vs[:, None]).amax(-1, keepdim=True) * codes[:, None]
        bound.append((torch.einsum("hgn,hnd->hgd", p, v.abs()) * (2.0 ** -11 + 2.0 ** -18 + 2 * off) + small).reshape(qh, d))
    return out, bound


def sample(x, temp, top_k, top_p, min_p, u):
    """(ids, logprobs, margin): margin is how far, relative to the weight it is compared with, the nearest
    comparison of the row is from going the other way (top-p's cut, min-p's cut, the draw)."""
    x = x.double().cpu().numpy()
    B, V = x.shape
    ids, logp, margin = np.full(B, -1), np.full(B, -np.inf), np.full(B, np.inf)
    for b in range(B):
        row = np.where(np.isnan(x[b]), -np.inf, x[b])
        top = row.max()
        if top == -np.inf:
            continue
        if not temp[b] > 0:
            ids[b], logp[b] = int(np.argmax(row)), 0.0
            continue
        order = np.argsort(-row, kind="stable")
        with np.errstate(invalid="ignore"):
            w = np.where(row == top, 1.0, np.where(row == -np.inf, 0.0, np.exp((row - top) / float(temp[b]))))
        s = w[order]
        n = V if top_k[b] <= 0 else min(V, int(top_k[b]))
        s = s[:n]
        p = float(top_p[b])
        if p < 1:
            cum, need = np.cumsum(s), p * s.sum()
            m = 1 + int((cum[:-1] < need).sum())
            if need > 0:
                margin[b] = min(margin[b], np.abs(cum[:-1] - need).min() / s.sum() if n > 1 else np.inf)
            s = s[:m]
        least = min(float(min_p[b]), 1.0)
        if least > 0:
            keep = s >= least
            near = np.abs(s - least)[s != 1.0]
            margin[b] = min(margin[b], near.min() if near.size else np.inf)
            s = s[:max(1, int(keep.sum()))]
        s = s[s > 0]
        kept = np.sort(order[:len(s)])
        cum = np.cumsum(w[kept])
        target = max(float(u[b]), 0.0) * cum[-1]
        if len(kept) > 1:
            margin[b] = min(margin[b], np.abs(cum[:-1] - target).min() / cum[-1])
        at = min(int(np.searchsorted(cum, target, side="right")), len(kept) - 1)
        ids[b], logp[b] = kept[at], math.log(w[kept[at]] / cum[-1])
    return ids, logp, margin
