"""The ragged step of the 8-bit cache from its definitions (Python integers and
64-bit torch; no code of the library)."""

import torch

import kv8_ref as ref

DRAFTS = 64


def depth_of(parents, j):
    """Number of ancestors of row j, None if the walk up leaves the rows before it."""
    n = 0
    while parents[j] != -1:
        if not 0 <= parents[j] < j:
            return None
        n, j = n + 1, parents[j]
    return n


def plan(slots, lens, counts, T, num_slots, cap, parents=None):
    """What kv8_plan writes, and per stream (start, n, tree) with n = 0 where it sits out or is refused."""
    B, t = len(slots), 0
    out = {"row_start": [], "after": [], "row_slot": [-1] * T, "row_index": [0] * T, "row_pos": [0] * T}
    streams = []
    for b in range(B):
        n, base = max(counts[b], 0), lens[b]
        fits = 0 <= slots[b] < num_slots and base >= 0 and counts[b] >= 0 and base + n <= cap and (n == 0 or t + n <= T)
        tree = fits and n > 0 and parents is not None and parents[t] != -2
        depth = list(range(n)) if fits else []
        if tree:
            depth = [depth_of(parents[t:t + n], j) for j in range(n)] if n <= DRAFTS else [None]
            fits = None not in depth
        out["row_start"].append(min(t, T))
        out["after"].append(base + n if fits else -1)
        if fits:
            for j in range(n):
                out["row_slot"][t + j], out["row_index"][t + j], out["row_pos"][t + j] = slots[b], base + j, base + depth[j]
        streams.append((min(t, T), n if fits else 0, bool(fits and tree)))
        t += n
    out["row_start"].append(min(t, T))
    return out, streams


def see(n, parents=None):
    """[n][n] bool: row j attends to row i of its own step."""
    m = torch.zeros(n, n, dtype=torch.bool)
    for j in range(n):
        if parents is None:
            m[j, :j + 1] = True
        else:
            at = j
            while at != -1:
                m[j, at] = True
                at = parents[at]
    return m


def attend(cache, Q, slots, lens, streams, scale, parents=None):
    """(o, bound, live): outputs in 64 bits [T][qh][d], what a kernel may be off before the last rounding, and which rows
    the step has.

    The bound per element is that of decode attention over this cache (kv8_ref.attend): weights rounded to 16 bits
    (2^-11), scores of d fp32 products (each weight and the normalising sum off by (d + 8) 2^-24 scale sum|q||k|),
    2^-18 for e^x and the sums, and fp16's smallest step against the row's largest term.  V scales below 2^-100 count
    as that there (the calls' stated range): weights are held against the maximum of x + max(log2 vs, -100), so a scale of
    2^-107 leaves the largest weight at 2^-7, and half of fp16's smallest step, 2^-25, is 2^-18 of it."""
    T, qh, d = Q.shape
    kvh = cache["kv_heads"]
    G = qh // kvh
    o = torch.zeros(T, qh, d, dtype=torch.float64, device=Q.device)
    bound, live = torch.zeros_like(o), torch.zeros(T, dtype=torch.bool, device=Q.device)
    for b, (t, n, tree) in enumerate(streams):
        if n == 0:
            continue
        live[t:t + n] = True
        s, base = slots[b], lens[b]
        L = base + n
        hidden = ~see(n, parents[t:t + n] if tree else None).to(Q.device)
        for h in range(kvh):
            vc, vs, ks = ref.decode(cache["V"][s, h, :L], cache["format"]), cache["Vs"][s, h, :L].double(), cache["Ks"][s, h, :L].double()
            k, v = ref.decode(cache["K"][s, h, :L], cache["format"]) * ks[:, None], vc * vs[:, None]
            q = Q[t:t + n, h * G:(h + 1) * G].double()
            x = torch.einsum("tgd,pd->tgp", q, k) * scale
            x[:, :, base:] = x[:, :, base:].masked_fill(hidden[:, None], -torch.inf)
            p = torch.softmax(x, -1)
            big = torch.einsum("tgd,pd->tgp", q.abs(), k.abs())
            big[:, :, base:] = big[:, :, base:].masked_fill(hidden[:, None], 0)
            off = big.amax(-1, keepdim=True) * scale * (d + 8) * 2.0 ** -24
            seen = torch.ones(n, L, dtype=torch.float64, device=Q.device)
            seen[:, base:] = (~hidden).double()
            # what a row does not attend to is no part of it, NaN or not
            clean = lambda y: torch.where(y.isfinite(), y, 0)  # noqa: E731
            part = slice(t, t + n), slice(h * G, (h + 1) * G)
            o[part] = torch.einsum("tgp,pd->tgd", p, clean(v))
            small = 2.0 ** -25 * (p * clean(vs).clamp(min=2.0 ** -100)).amax(-1, keepdim=True) * (seen @ clean(vc.abs()))[:, None]
            bound[part] = torch.einsum("tgp,pd->tgd", p, clean(v.abs())) * (2.0 ** -11 + 2.0 ** -18 + 2 * off) + small
    return o, bound, live


def accept(streams, lens, parents, tokens, ids, refused, before):
    """What kv8_tree_accept writes; `before` the lens of refused streams."""
    B = len(streams)
    out = {"path": [[-1] * DRAFTS for _ in range(B)], "fresh": [[-1] * DRAFTS for _ in range(B)], "kept": [0] * B, "n_fresh": [0] * B,
           "lens": list(before)}
    for b, (t, n, tree) in enumerate(streams):
        if refused[b]:
            continue
        if n and not tree:
            out["kept"][b], out["n_fresh"][b], out["fresh"][b][0] = n, 1, ids[t + n - 1]
        at = 0 if n and tree else None
        while at is not None:
            k = out["kept"][b]
            out["path"][b][k], out["fresh"][b][k] = at, ids[t + at]
            out["kept"][b] = out["n_fresh"][b] = k + 1
            at = next((j for j in range(n) if parents[t + j] == at and tokens[t + j] == ids[t + at] >= 0), None)
        out["lens"][b] = lens[b] + out["kept"][b]
    return out
