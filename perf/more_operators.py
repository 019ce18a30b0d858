"""Measured cases of the ragged-step operators of the 8-bit cache.

A serving step in which every stream brings its own number of rows: a prompt or
a part of one, one decode token, or a tree of drafted tokens.  The step is
planned once (``kv8_plan``: where each row goes, and how the attention splits),
every layer attends with that plan (``kv8_attend_rows``), and a step of drafts
ends with the walk down the trees (``kv8_tree_accept``) and, layer by layer, the
accepted rows closing up (``kv8_tree_keep``).  ``run`` makes the framework's
calls where ``own`` is true and computes the same values with elementary torch
operations otherwise; ``exact`` restates the definitions.
"""

import math

import numpy as np
import torch

own = False

E4M3, INT8 = 0, 1
CODE_MAX = {E4M3: 448.0, INT8: 127.0}
DRAFTS = 64   # rows a tree may have
FULL = {"qh": 32, "kvh": 4, "d": 128}
TINY = {"qh": 8, "kvh": 2, "d": 64}


def listed():
    return [
        # one decode step of a few streams with their drafts: the latency of planning it
        {"name": "plan_trees_8x17", "op": "plan", "B": 8, "n": 17, "base": 4000, "ragged": False, "tree": True, "pad": 3, **FULL},
        # a step of a large server: 512 streams of 1 to 128 rows
        {"name": "plan_512_prompts", "op": "plan", "B": 512, "n": 128, "base": 3000, "ragged": True, "tree": False, "pad": 64, **FULL},
        # two short prompts of the tiny layer: the latency of a call
        {"name": "rows_tiny_2x40", "op": "rows", "fmt": E4M3, "B": 2, "n": 40, "base": 0, "ragged": True, "tree": False, "pad": 3, **TINY},
        # prompts of different lengths that arrived together, packed into one step
        {"name": "rows_packed_16x1000", "op": "rows", "fmt": E4M3, "B": 16, "n": 1000, "base": 0, "ragged": True, "tree": False, "pad": 0,
         **FULL},
        # one long prompt
        {"name": "rows_prompt_8192", "op": "rows", "fmt": E4M3, "B": 1, "n": 8192, "base": 0, "ragged": False, "tree": False, "pad": 0, **FULL},
        # the next part of a long document, 8-bit integers
        {"name": "rows_chunk_1000x65536", "op": "rows", "fmt": INT8, "B": 1, "n": 1000, "base": 65536, "ragged": False, "tree": False, "pad": 0,
         **FULL},
        # one stream that drafts a small tree
        {"name": "tree_solo_13x4096", "op": "rows", "fmt": E4M3, "B": 1, "n": 13, "base": 4096, "ragged": False, "tree": True, "pad": 0, **FULL},
        # a batch of chat-length streams, each with a tree
        {"name": "tree_32x16x4096", "op": "rows", "fmt": E4M3, "B": 32, "n": 16, "base": 4096, "ragged": True, "tree": True, "pad": 5, **FULL},
        # a small batch's walk down its trees
        {"name": "accept_4x13", "op": "accept", "B": 4, "n": 13, "base": 500, "ragged": False, "tree": True, "pad": 0, **TINY},
        # the same for a large batch of the widest trees
        {"name": "accept_512x64", "op": "accept", "B": 512, "n": 64, "base": 500, "ragged": True, "tree": True, "pad": 0, **FULL},
        # one layer's cache after a small batch's step
        {"name": "keep_4x13", "op": "keep", "fmt": INT8, "B": 4, "n": 13, "base": 500, "ragged": False, "tree": True, "pad": 0, **TINY},
        # the same for a large batch of the widest trees
        {"name": "keep_256x64", "op": "keep", "fmt": E4M3, "B": 256, "n": 64, "base": 500, "ragged": True, "tree": True, "pad": 0, **FULL},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "prompt", "prompt", "chunk", "chunk", "tree", "tree", "accept", "keep"])
    qh, kvh = rng.choice([(32, 4), (8, 2), (16, 8), (12, 4), (4, 4), (16, 2), (10, 2)])
    c = {"op": "rows", "fmt": rng.choice([E4M3, INT8]), "ragged": rng.random() < 0.7, "tree": False, "pad": rng.choice([0, 0, 1, 5]),
         "qh": qh, "kvh": kvh, "d": rng.choice([64, 128])}
    if kind in ("prompt", "chunk"):
        c["B"] = _log_int(rng, 1, 16)
        c["n"] = _log_int(rng, 1, 8000 // c["B"])
        c["base"] = 0 if kind == "prompt" else _log_int(rng, 1, max(1, min(30000, 50_000_000 // c["n"]) // c["B"]))
        return c
    c.update(tree=True, B=_log_int(rng, 1, 32), n=_log_int(rng, 1, DRAFTS), base=_log_int(rng, 1, 4000))
    if kind == "tree":
        return c
    if kind != "keep":
        del c["fmt"]
    c.update(op=kind, B=_log_int(rng, 1, 256))
    if kind == "plan" and rng.random() < 0.5:
        c.update(tree=False, n=_log_int(rng, 1, 256))
    return c


def _counts(c):
    """The streams' rows of this step: spread over 1..n, or all n."""
    B, n = c["B"], c["n"]
    return np.array([1 + int((i + 0.5) / B * n) if c["ragged"] and B > 1 else n for i in range(B)], np.int64)


def _bases(c):
    """Positions that the streams hold before the step, in another order than their rows."""
    B, base = c["B"], c["base"]
    return np.array([int(((7 * i + 3) % B + 0.5) / B * base) if c["ragged"] and B > 1 else base for i in range(B)], np.int64)


def _moves(c):
    """Per stream: rows kept, and those of them, from the front, that are in place already."""
    kept = 1 + (_counts(c) - 1) // 3
    return kept, np.maximum(1, kept // 3)


def work(case):
    op, n, base = case["op"], _counts(case), _bases(case)
    qh, kvh, d, T, B = case["qh"], case["kvh"], case["d"], int(_counts(case).sum()) + case["pad"], case["B"]
    if op == "plan":
        return {"bytes": 12 * B + 8 * B + (16 if case["tree"] else 12) * T, "flops": 8 * T}
    if op == "accept":
        return {"bytes": 16 * T + B * (2 * 4 * DRAFTS + 12), "flops": 4 * T}
    if op == "keep":
        kept, first = _moves(case)
        return {"bytes": int((kept - first).sum()) * 4 * kvh * (d + 4) + 4 * int(kept.sum()) + 16 * B, "flops": int((kept - first).sum()) * kvh * d}
    pairs = int((n * base + n * (n + 1) // 2).sum())
    return {"bytes": int((base + n).sum()) * kvh * (2 * d + 8) + 4 * T * qh * d, "flops": 4 * pairs * qh * d}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return g


def _normal(g, *shape, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g).to(dtype)


def _cache(g, fmt, slots, cap, kvh, d):
    """A cache that earlier calls have filled; the magnitudes differ from head to head and from position to position."""
    out = {"format": fmt, "slots": slots, "ctx_cap": cap, "kv_heads": kvh, "head_dim": d}
    for n in ("K", "V"):
        x = _normal(g, slots, kvh, cap, d)
        x *= torch.exp(0.4 * _normal(g, slots, kvh, cap, 1))
        scale = x.abs().amax(-1, keepdim=True) / CODE_MAX[fmt]
        y = x / scale
        out[n] = (y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn) if fmt == E4M3 else y.round().to(torch.int8)).view(torch.uint8)
        out[n + "s"] = scale.squeeze(-1).contiguous()
    return out


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == E4M3 else torch.int8)


def _parents(counts, rs):
    """Trees in the order in which drafts are made: a row's parent is one of the few before it."""
    out = []
    for n in counts:
        j = np.arange(n)
        out.append(np.where(j == 0, -1, np.maximum(0, j - 1 - rs.randint(0, 6, n))))
    return np.concatenate(out).astype(np.int32)


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    rs = np.random.RandomState((seed * 31 + 5) % (1 << 31))
    dev = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, t)).cuda()  # noqa: E731
    B, qh, kvh, d = case["B"], case["qh"], case["kvh"], case["d"]
    n, base = _counts(case), _bases(case)
    T, cap = int(n.sum()) + case["pad"], int((n + base).max()) + 5
    slots = B + 1
    s = {"case": case, "cap": cap, "slots": slots, "T": T, "slot": dev(rs.permutation(slots)[:B]), "lens": dev(base), "counts": dev(n),
         "host": (n, base)}
    if op in ("rows", "keep"):
        s["cache"] = _cache(g, case["fmt"], slots, cap, kvh, d)
    else:   # the plan needs a cache's sizes only
        s["sizes"] = {"format": E4M3, "slots": slots, "ctx_cap": cap, "kv_heads": kvh, "head_dim": d}
    if case["tree"]:
        s["host_parents"] = np.concatenate([_parents(n, rs), np.full(case["pad"], -1, np.int32)])
        s["parents"] = dev(s["host_parents"])
    if op == "rows":
        s["Q"] = _normal(g, T, qh, d, dtype=torch.bfloat16)
        s["O"] = torch.zeros(T, qh, d, dtype=torch.bfloat16, device="cuda")
    if op == "plan":
        z = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")  # noqa: E731
        s["out"] = {"row_start": z(B + 1), "after": z(B), "row_slot": z(T), "row_index": z(T), "row_pos": z(T)}
    if op == "accept":
        # the model agrees with a draft more often than not
        start = np.concatenate([[0], np.cumsum(n)])
        tokens, ids = rs.randint(0, 32000, T).astype(np.int32), rs.randint(0, 32000, T).astype(np.int32)
        child = rs.permutation(np.nonzero(s["host_parents"] >= 0)[0])
        at = np.repeat(start[:-1], n)[child] + s["host_parents"][child]
        ids[at] = np.where(rs.rand(len(child)) < 0.8, tokens[child], ids[at])
        s["tokens"], s["ids"] = dev(tokens), dev(ids)
        i32 = lambda *k: torch.zeros(k, dtype=torch.int32, device="cuda")  # noqa: E731
        s["out"] = {"path": i32(B, DRAFTS), "kept": i32(B), "fresh": i32(B, DRAFTS), "n_fresh": i32(B), "lens": i32(B)}
    if op == "keep":
        kept, first = _moves(case)
        path = np.full((B, DRAFTS), -1, np.int32)
        for b in range(B):
            path[b, :first[b]] = np.arange(first[b])
            path[b, first[b]:kept[b]] = kept[b] + np.sort(rs.permutation(n[b] - kept[b])[:kept[b] - first[b]])
        s["path"], s["kept"] = dev(path), dev(kept)
    return s


# ---------------------------------------------------------------- the framework's calls

def _handle(s):
    """What a serving loop has: the cache descriptor and workspaces, made once, and this step's plan, made once for all layers."""
    import bit_moe_decode_w4a16_gb300 as bm
    h = s.get("handle")
    if h is None:
        c = s["case"]
        h = s["handle"] = {"bm": bm}
        cache = s.get("cache")
        if cache is None:
            z = s["sizes"]
            rows = (z["slots"], z["kv_heads"], z["ctx_cap"])
            cache = dict(z, **{n: torch.zeros(rows + (z["head_dim"],), dtype=torch.uint8, device="cuda") for n in ("K", "V")},
                         **{n: torch.zeros(rows, dtype=torch.float32, device="cuda") for n in ("Ks", "Vs")})
        h["cache"] = bm.kv8_cache(**cache)
        B, T, i32 = c["B"], s["T"], torch.int32
        h["plan"] = torch.empty(bm.kv8_plan_bytes(B, T, c["qh"], c["kvh"]), dtype=torch.uint8, device="cuda")
        if c["op"] != "plan":
            out = [torch.empty(k, dtype=i32, device="cuda") for k in (B + 1, B, T, T, T)]
            bm.kv8_plan(h["cache"], c["qh"], s["slot"], s["lens"], s["counts"], *out, h["plan"], parents=s.get("parents"))
        if c["op"] == "rows":
            n = bm.kv8_rows_workspace_bytes(B, T, c["qh"], c["kvh"], c["d"], s["cap"])
            h["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return h


def _run_own(s):
    h, op = _handle(s), s["case"]["op"]
    bm, plan = h["bm"], h["plan"]
    if op == "plan":
        o = s["out"]
        bm.kv8_plan(h["cache"], s["case"]["qh"], s["slot"], s["lens"], s["counts"], o["row_start"], o["after"], o["row_slot"], o["row_index"],
                    o["row_pos"], plan, parents=s.get("parents"))
        return o
    if op == "rows":
        bm.kv8_attend_rows(h["cache"], plan, s["Q"], s["O"], s["case"]["B"], h["ws"])
        return s["O"]
    if op == "accept":
        o = s["out"]
        bm.kv8_tree_accept(plan, s["tokens"], s["ids"], o["path"], o["kept"], o["fresh"], o["n_fresh"], o["lens"])
        return o
    bm.kv8_tree_keep(h["cache"], plan, s["path"], s["kept"])
    return _kept(s)


def _kept(s):
    c, fmt = s["cache"], s["case"]["fmt"]
    return {"K": _values(c["K"], fmt), "Ks": c["Ks"], "V": _values(c["V"], fmt), "Vs": c["Vs"]}


# ---------------------------------------------------------------- the plain form

def _rows_of(s):
    """Stream of each row (B for padding) and its place in the stream."""
    start = torch.cat([s["counts"].new_zeros(1, dtype=torch.int64), s["counts"].long().cumsum(0)])
    row = torch.arange(s["T"], device="cuda")
    stream = torch.searchsorted(start, row, right=True) - 1
    return start, row, stream


def _plain_plan(s):
    B, o = s["case"]["B"], s["out"]
    start, row, stream = _rows_of(s)
    pad = stream >= B
    stream = stream.clamp(max=B - 1)
    j = row - start[stream]
    base = s["lens"].long()[stream]
    depth = j
    if "parents" in s:
        at, depth = torch.where(pad, -1, s["parents"].long()), torch.zeros_like(j)
        first = start[stream]
        for _ in range(DRAFTS):
            depth = depth + (at >= 0)
            at = torch.where(at >= 0, s["parents"].long()[(first + at).clamp(min=0)], at)
    o["row_start"].copy_(start)
    o["after"].copy_(s["lens"] + s["counts"])
    for n, v, other in (("row_slot", s["slot"].long()[stream], -1), ("row_index", base + j, 0), ("row_pos", base + depth, 0)):
        o[n].copy_(torch.where(pad, other, v))
    return o


def _ancestors(par):
    """[n][n]: row j attends to row i of its own step."""
    n = par.shape[0]
    see = torch.eye(n, dtype=torch.bool, device=par.device)
    at = par.long()
    rows = torch.arange(n, device=par.device)
    for _ in range(n):
        live = at >= 0
        see[rows, at.clamp(min=0)] |= live
        at = torch.where(live, par.long()[at.clamp(min=0)], at)
    return see


def _plain_rows(s):
    c, cache = s["case"], s["cache"]
    qh, kvh, d = c["qh"], c["kvh"], c["d"]
    counts, bases = s["host"]
    at = 0
    for b in range(c["B"]):
        n, base = int(counts[b]), int(bases[b])
        L = base + n
        slot = s["slot"][b].long()
        see = torch.arange(L, device="cuda") <= base + torch.arange(n, device="cuda")[:, None]
        if c["tree"]:
            see = torch.cat([torch.ones(n, base, dtype=torch.bool, device="cuda"), _ancestors(s["parents"][at:at + n])], 1)
        q = s["Q"][at:at + n].float().view(n, kvh, qh // kvh, d)
        for h in range(kvh):
            k, v = (_values(cache[m], c["fmt"])[slot, h, :L].float() * cache[m + "s"][slot, h, :L, None] for m in ("K", "V"))
            score = (q[:, h].transpose(0, 1) @ k.T / math.sqrt(d)).masked_fill(~see, -math.inf)
            p = torch.exp(score - score.amax(-1, keepdim=True))
            o = (p / p.sum(-1, keepdim=True)) @ v
            s["O"][at:at + n].view(n, kvh, qh // kvh, d)[:, h].copy_(o.transpose(0, 1))
        at += n
    return s["O"]


def _plain_accept(s):
    B, o = s["case"]["B"], s["out"]
    start, row, stream = _rows_of(s)
    stream = stream.clamp(max=B - 1)
    T = s["T"]
    parent = torch.where(s["parents"] >= 0, start[stream] + s["parents"], -1)
    wanted = s["ids"].long()[parent.clamp(min=0)]
    fits = (parent >= 0) & (s["tokens"].long() == wanted) & (wanted >= 0)
    # the first fitting child of each row
    child = torch.full((T + 1,), T, dtype=torch.int64, device="cuda")
    child.scatter_reduce_(0, torch.where(fits, parent, T), torch.where(fits, row, T), "amin")
    child[T] = T
    first = start[:B]
    at = first.clone()
    path, fresh = [], []
    ids = torch.cat([s["ids"].long(), s["ids"].new_full((1,), -1, dtype=torch.int64)])
    for _ in range(DRAFTS):
        path.append(torch.where(at < T, at - first, -1))
        fresh.append(ids[at])
        at = child[at]
    path, fresh = torch.stack(path, 1), torch.stack(fresh, 1)
    kept = (path >= 0).sum(1)
    for n, v in (("path", path), ("fresh", fresh), ("kept", kept), ("n_fresh", kept), ("lens", s["lens"].long() + kept)):
        o[n].copy_(v)
    return o


def _plain_keep(s):
    cache = s["cache"]
    i = torch.arange(DRAFTS, device="cuda")
    b, to = ((i < s["kept"][:, None]) & (s["path"] != i)).nonzero(as_tuple=True)
    slot, base = s["slot"].long()[b], s["lens"].long()[b]
    for n in ("K", "V", "Ks", "Vs"):
        cache[n][slot, :, base + to] = cache[n][slot, :, base + s["path"].long()[b, to]]
    return _kept(s)


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "rows": _plain_rows, "accept": _plain_accept, "keep": _plain_keep}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions, on the host or in 64 bits

_E4M3 = np.array([(-1.0 if c & 128 else 1.0) * ((c & 7) / 8 * 2.0 ** -6 if not c & 120 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                  for c in range(256)])
_INT8 = np.arange(256, dtype=np.uint8).view(np.int8).astype(np.float64)


def _decode(codes, fmt):
    return torch.from_numpy(_E4M3 if fmt == E4M3 else _INT8).to(codes.device)[codes.long()]


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rows": _exact_rows, "accept": _exact_accept, "keep": _exact_keep}[case["op"]](s)


def _exact_plan(s):
    n, base = s["host"]
    slot, T = s["slot"].cpu().numpy(), s["T"]
    out = {"row_start": np.zeros(len(n) + 1, np.int64), "after": base + n, "row_slot": np.full(T, -1), "row_index": np.zeros(T, np.int64),
           "row_pos": np.zeros(T, np.int64)}
    t = 0
    for b in range(len(n)):
        for j in range(n[b]):
            depth, up = 0, j
            while s["case"]["tree"] and s["host_parents"][t + up] >= 0:
                depth, up = depth + 1, s["host_parents"][t + up]
            out["row_slot"][t + j], out["row_index"][t + j] = slot[b], base[b] + j
            out["row_pos"][t + j] = base[b] + (depth if s["case"]["tree"] else j)
        t += n[b]
        out["row_start"][b + 1] = t
    return out


def _exact_rows(s):
    c = s["case"]
    qh, kvh, d, (counts, bases) = c["qh"], c["kvh"], c["d"], s["host"]
    G, t, out = qh // kvh, 0, torch.zeros(s["T"], qh, d, dtype=torch.float64, device="cuda")
    for b, slot in enumerate(s["slot"].tolist()):
        n, base = int(counts[b]), int(bases[b])
        hidden = np.triu(np.ones((n, n), bool), 1)
        if c["tree"]:
            hidden = np.ones((n, n), bool)
            for j in range(n):
                up = j
                while up >= 0:
                    hidden[j, up] = False
                    up = s["host_parents"][t + up]
        hidden = torch.from_numpy(hidden).cuda()
        for h in range(kvh):
            k, v = (_decode(s["cache"][m][slot, h, :base + n], c["fmt"]) * s["cache"][m + "s"][slot, h, :base + n].double().unsqueeze(-1)
                    for m in ("K", "V"))
            for g in range(h * G, h * G + G):
                x = torch.einsum("td,pd->tp", s["Q"][t:t + n, g].double(), k) * d ** -0.5
                x[:, base:].masked_fill_(hidden, -math.inf)
                out[t:t + n, g] = torch.softmax(x, 1) @ v
        t += n
    return out


def _exact_accept(s):
    n, base = s["host"]
    B, tokens, ids, par = len(n), s["tokens"].cpu().numpy(), s["ids"].cpu().numpy(), s["host_parents"]
    out = {"path": np.full((B, DRAFTS), -1), "fresh": np.full((B, DRAFTS), -1), "kept": np.zeros(B, np.int64)}
    t = 0
    for b in range(B):
        at, k = 0, 0
        while at is not None:
            out["path"][b, k], out["fresh"][b, k] = at, ids[t + at]
            k += 1
            at = next((j for j in range(at + 1, n[b]) if par[t + j] == at and tokens[t + j] == ids[t + at]), None)
        out["kept"][b] = k
        t += n[b]
    return dict(out, n_fresh=out["kept"], lens=base + out["kept"])


def _exact_keep(s):
    cache, fmt = s["cache"], s["case"]["fmt"]
    out = {n: _decode(cache[n], fmt) if n in ("K", "V") else cache[n].double() for n in ("K", "V", "Ks", "Vs")}
    before = {n: x.clone() for n, x in out.items()}
    path, kept = s["path"].cpu().numpy(), s["kept"].cpu().numpy()
    for b, slot in enumerate(s["slot"].tolist()):
        base = int(s["host"][1][b])
        for i in range(kept[b]):
            for n in out:
                out[n][slot, :, base + i] = before[n][slot, :, base + int(path[b, i])]
    return out
