"""Measured cases of the 8-bit cache operators and of the sampler.

Each case is one call as a serving loop makes it between the projections of a
decode step: rows of q, k, v written to the cache, the cache read back,
attended (alone, or behind a prefix that the batch shares), and a token drawn
from the logits.  ``run`` makes the framework's calls where ``own`` is true and
computes the same values with elementary torch operations otherwise;
``exact`` restates the definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

E4M3, INT8 = 0, 1
CODE_MAX = {E4M3: 448.0, INT8: 127.0}
TINY = 2.0 ** -110   # a head whose largest value is below this is stored as zeros
EPS = 1e-6


def listed():
    return [
        # two streams of the tiny layer and some padding: the latency of a call
        {"name": "append_tiny", "op": "append", "T": 5, "qh": 8, "kvh": 2, "d": 64, "norm": True, "base": 1e4},
        # one decode step of 32 streams, full-width heads
        {"name": "append_decode_32", "op": "append", "T": 32, "qh": 32, "kvh": 4, "d": 128, "norm": True, "base": 1e4},
        # a prompt of 4000 tokens written at once
        {"name": "append_prompt_4000", "op": "append", "T": 4000, "qh": 32, "kvh": 4, "d": 128, "norm": True,
         "base": 1e6},
        # a few positions from the middle of a slot, for a test or a trace
        {"name": "read_odd_1001", "op": "read", "fmt": INT8, "kvh": 2, "d": 64, "first": 37, "count": 1001},
        # a whole long slot, for a checkpoint or a move to a 16-bit arena
        {"name": "read_65536", "op": "read", "fmt": E4M3, "kvh": 4, "d": 128, "first": 0, "count": 65536},
        # one stream alone
        {"name": "attend_solo_4096", "op": "attend", "fmt": E4M3, "B": 1, "L": 4096, "qh": 32, "kvh": 4, "d": 128,
         "ragged": False},
        # the ragged 16-stream batch of the long-context arena
        {"name": "attend_ragged_16x8192", "op": "attend", "fmt": E4M3, "B": 16, "L": 8192, "qh": 32, "kvh": 4, "d": 128,
         "ragged": True},
        # a full batch of chat-length streams, 8-bit integers
        {"name": "attend_int8_32x1500", "op": "attend", "fmt": INT8, "B": 32, "L": 1500, "qh": 32, "kvh": 4, "d": 128,
         "ragged": True},
        # three streams of the tiny layer's heads on a short shared prompt
        {"name": "prefix_tiny_3x1000", "op": "prefix", "fmt": INT8, "B": 3, "P": 1000, "L": 90, "qh": 8, "kvh": 2, "d": 64},
        # a full batch on one long shared document, each with its own turn behind it
        {"name": "prefix_32x32768", "op": "prefix", "fmt": E4M3, "B": 32, "P": 32768, "L": 512, "qh": 32, "kvh": 4,
         "d": 128},
        # one stream, the whole vocabulary, nucleus sampling
        {"name": "sample_1_nucleus", "op": "sample", "B": 1, "V": 151936, "half": False, "filters": "nucleus"},
        # a full batch in which every request has settings of its own
        {"name": "sample_32_mixed", "op": "sample", "B": 32, "V": 151936, "half": False, "filters": "mixed"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "prefix", "prefix", "sample", "sample"])
    qh, kvh = rng.choice([(32, 4), (8, 2), (16, 8), (12, 4), (4, 4), (16, 2)])
    d = rng.choice([64, 128])
    fmt = rng.choice([E4M3, INT8])
    if op == "append":
        return {"op": op, "T": _log_int(rng, 1, 4000), "qh": qh, "kvh": kvh, "d": d, "norm": rng.random() < 0.7,
                "base": rng.choice([1e4, 1e6])}
    if op == "read":
        return {"op": op, "fmt": fmt, "kvh": kvh, "d": d, "first": rng.randrange(0, 1000), "count": _log_int(rng, 1, 30000)}
    if op == "attend":
        B = _log_int(rng, 1, 32)
        return {"op": op, "fmt": fmt, "B": B, "L": _log_int(rng, 1, 60000 // B), "qh": qh, "kvh": kvh, "d": d,
                "ragged": rng.random() < 0.7}
    if op == "prefix":
        B = _log_int(rng, 1, 32)
        return {"op": op, "fmt": fmt, "B": B, "P": _log_int(rng, 100, 30000), "L": _log_int(rng, 1, 512), "qh": qh,
                "kvh": kvh, "d": d}
    return {"op": op, "B": _log_int(rng, 1, 32), "V": _log_int(rng, 100, 151936), "half": rng.random() < 0.3,
            "filters": rng.choice(["none", "topk", "nucleus", "mixed"])}


def _lengths(B, L, ragged):
    """The streams' lengths: spread over 1..L, or all L."""
    return [1 + int((i + 0.5) / B * L) if ragged and B > 1 else L for i in range(B)]


def work(case):
    op = case["op"]
    if op == "append":
        T, qh, kvh, d = case["T"], case["qh"], case["kvh"], case["d"]
        return {"bytes": T * ((2 * qh + 2 * kvh) * d * 2 + 2 * kvh * (d + 4) + 12), "flops": T * (qh + 2 * kvh) * d * 10}
    if op == "read":
        n = 2 * case["kvh"] * case["count"]
        return {"bytes": n * (3 * case["d"] + 4), "flops": n * case["d"]}
    if op in ("attend", "prefix"):
        B, qh, kvh, d = case["B"], case["qh"], case["kvh"], case["d"]
        P = case.get("P", 0)
        own_len = sum(_lengths(B, case["L"], case.get("ragged", True)))
        return {"bytes": (own_len + P) * kvh * (2 * d + 8) + 4 * B * qh * d, "flops": 4 * (own_len + B * P) * qh * d}
    return {"bytes": case["B"] * case["V"] * (2 if case["half"] else 4), "flops": 4 * case["B"] * case["V"]}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 11)
    return g


def _normal(g, *shape, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g).to(dtype)


def _quantise(x, fmt):
    """Codes (uint8 bit patterns) and scales of x [..., d]."""
    amax = x.abs().amax(-1, keepdim=True)
    live = amax >= TINY
    inv = torch.where(live, CODE_MAX[fmt] / amax, torch.zeros_like(amax))
    scale = torch.where(live, amax / CODE_MAX[fmt], torch.zeros_like(amax))
    if fmt == E4M3:
        codes = (x * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes = (x * inv).round().clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)
    return codes, scale.squeeze(-1)


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == E4M3 else torch.int8)


def _cache(g, fmt, slots, cap, kvh, d):
    """A cache that earlier calls have filled; the magnitudes differ from head to head and from position to position."""
    out = {"format": fmt, "slots": slots, "ctx_cap": cap, "kv_heads": kvh, "head_dim": d}
    for n in ("K", "V"):
        x = _normal(g, slots, kvh, cap, d)
        x *= torch.exp(0.4 * _normal(g, slots, kvh, cap, 1))
        out[n], out[n + "s"] = _quantise(x, fmt)
    return out


def _order(B, slots, seed):
    return np.random.RandomState(seed % (1 << 31)).permutation(slots)[:B].astype(np.int32)


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    rs = np.random.RandomState((seed * 31 + 5) % (1 << 31))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    if op == "append":
        T, qh, kvh, d = case["T"], case["qh"], case["kvh"], case["d"]
        if T > 64:   # a prompt: consecutive positions of one slot, behind what it holds
            slots, first = 2, 77
            slot, index = np.full(T, 1, np.int32), np.arange(first, first + T, dtype=np.int32)
            cap = first + T + 3
        else:        # a decode step: one row to a slot, some rows padding
            slots, cap = T + 1, 300
            slot = rs.permutation(slots)[:T].astype(np.int32)
            index = rs.randint(0, cap, T).astype(np.int32)
            slot[T - T // 5:] = -1
        f = case["base"] ** (-2.0 * np.arange(d // 2) / d)
        return {"case": case, "cache": _cache(g, E4M3, slots, cap, kvh, d), "slot": dev(slot), "index": dev(index),
                "pos": dev(index + 1000), "qkv": _normal(g, T, (qh + 2 * kvh) * d, dtype=torch.bfloat16),
                "inv_freq": dev(f.astype(np.float32)), "Q": torch.zeros(T, qh, d, dtype=torch.bfloat16, device="cuda"),
                "wq": (1 + 0.2 * _normal(g, d)).to(torch.bfloat16), "wk": (1 + 0.2 * _normal(g, d)).to(torch.bfloat16)}
    if op == "read":
        n, kvh, d = case["count"], case["kvh"], case["d"]
        out = [torch.empty(kvh, n, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        return {"case": case, "cache": _cache(g, case["fmt"], 2, case["first"] + n + 1, kvh, d), "K": out[0], "V": out[1]}
    if op in ("attend", "prefix"):
        B, qh, kvh, d = case["B"], case["qh"], case["kvh"], case["d"]
        lens = np.array(_lengths(B, case["L"], case.get("ragged", True)), np.int32)
        rs.shuffle(lens)
        s = {"case": case, "cache": _cache(g, case["fmt"], B + 1, case["L"] + 5, kvh, d), "slot": dev(_order(B, B + 1, seed)),
             "lens": dev(lens), "Q": _normal(g, B, qh, d, dtype=torch.bfloat16),
             "O": torch.zeros(B, qh, d, dtype=torch.bfloat16, device="cuda")}
        if op == "prefix":
            s["prefix"] = _cache(g, case["fmt"], 1, case["P"] + 1, kvh, d)
        return s
    B, V = case["B"], case["V"]
    # logits of a language model: a bell, some likely tokens, masked ones
    x = 2.0 * _normal(g, B, V)
    x += torch.where(_normal(g, B, V) > 3.3, 6.0, 0.0)
    temp, top_k, top_p, min_p = (np.ones(B), np.zeros(B, np.int32), np.ones(B), np.zeros(B))
    for b in range(B):
        temp[b] = rs.uniform(0.6, 1.3)
        kind = case["filters"]
        if kind in ("nucleus", "mixed") and rs.rand() < (1.0 if kind == "nucleus" else 0.6):
            top_p[b] = rs.uniform(0.8, 0.98)
        if kind in ("topk", "mixed") and rs.rand() < (1.0 if kind == "topk" else 0.5):
            top_k[b] = rs.randint(1, 200)
        if kind == "mixed" and rs.rand() < 0.3:
            min_p[b] = rs.uniform(0.01, 0.2)
    if case["filters"] == "mixed" and B >= 4:
        temp[0] = 0.0                       # a greedy request
        x[1, V // 3:] = -math.inf           # a grammar that allows a third of the vocabulary
        x[2] = -math.inf                    # a grammar that allows nothing
    f32 = lambda a: dev(np.asarray(a, np.float32))  # noqa: E731
    return {"case": case, "logits": x.to(torch.bfloat16) if case["half"] else x, "temp": f32(temp), "top_k": dev(top_k.astype(np.int32)),
            "top_p": f32(top_p), "min_p": f32(min_p), "u": f32(rs.randint(0, 1 << 24, B) / float(1 << 24)),
            "ids": torch.zeros(B, dtype=torch.int32, device="cuda"), "logp": torch.zeros(B, dtype=torch.float32, device="cuda")}


# ---------------------------------------------------------------- the framework's calls

def _handle(s):
    """What a serving loop makes once: the cache descriptors and the workspace."""
    import bit_moe_decode_w4a16_gb300 as bm
    h = s.get("handle")
    if h is None:
        h = s["handle"] = {"bm": bm}
        for n in ("cache", "prefix"):
            if n in s:
                h[n] = bm.kv8_cache(**s[n])
        c = s["case"]
        if c["op"] in ("attend", "prefix"):
            n = bm.kv8_workspace_bytes(c["B"], c["qh"], c["kvh"], c["d"], s["cache"]["ctx_cap"], c.get("P", 0))
            h["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        if c["op"] == "append":
            h["rope"] = bm.kv8_rope(norm=c["norm"], q_norm=s["wq"], k_norm=s["wk"], eps=EPS, inv_freq=s["inv_freq"])
    return h


def _run_own(s):
    h, op = _handle(s), s["case"]["op"]
    bm = h["bm"]
    if op == "append":
        bm.kv8_append(h["cache"], s["qkv"], h["rope"], s["slot"], s["index"], s["Q"], rope_pos=s["pos"])
        return _appended(s)
    if op == "read":
        c = s["case"]
        bm.kv8_read(h["cache"], 1, c["first"], c["count"], s["K"], s["V"])
        return [s["K"], s["V"]]
    if op == "attend":
        bm.kv8_attend(h["cache"], s["Q"], s["slot"], s["lens"], s["O"], h["ws"])
        return s["O"]
    if op == "prefix":
        bm.kv8_attend_prefix(h["cache"], h["prefix"], 0, s["case"]["P"], s["Q"], s["slot"], s["lens"], s["O"], h["ws"])
        return s["O"]
    bm.bm_sample(s["logits"], s["temp"], s["top_k"], s["top_p"], s["min_p"], s["u"], s["ids"], s["logp"])
    return [s["ids"], s["logp"]]


def _appended(s):
    c = s["cache"]
    return {"Q": s["Q"], "K": _values(c["K"], E4M3), "Ks": c["Ks"], "V": _values(c["V"], E4M3), "Vs": c["Vs"]}


# ---------------------------------------------------------------- the plain form

def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _rotate(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c, cache = s["case"], s["cache"]
    T, qh, kvh, d = c["T"], c["qh"], c["kvh"], c["d"]
    x = s["qkv"].view(T, qh + 2 * kvh, d).float()
    q, k, v = x.split([qh, kvh, kvh], 1)
    if c["norm"]:
        q, k = _norm(q, s["wq"].float()), _norm(k, s["wk"].float())
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    q, k = _rotate(q, cos, sin), _rotate(k, cos, sin)
    live = (s["slot"] >= 0).nonzero()[:, 0]
    slot, index = s["slot"][live].long(), s["index"][live].long()
    s["Q"][live] = q[live].to(torch.bfloat16)
    for n, y in (("K", k), ("V", v)):
        codes, scale = _quantise(y[live], E4M3)
        cache[n][slot, :, index] = codes
        cache[n + "s"][slot, :, index] = scale
    return _appended(s)


def _plain_read(s):
    c, cache = s["case"], s["cache"]
    at = slice(c["first"], c["first"] + c["count"])
    for n in ("K", "V"):
        s[n].copy_(_values(cache[n], c["fmt"])[1, :, at].float() * cache[n + "s"][1, :, at, None])
    return [s["K"], s["V"]]


def _plain_attend(s):
    c, cache = s["case"], s["cache"]
    B, qh, kvh, d, L = c["B"], c["qh"], c["kvh"], c["d"], c["L"]
    slot = s["slot"].long()
    own_kv = [_values(cache[n], c["fmt"])[slot, :, :L].float() * cache[n + "s"][slot, :, :L, None] for n in ("K", "V")]
    q = s["Q"].float().view(B, kvh, qh // kvh, d)
    score = q @ own_kv[0].transpose(2, 3) / math.sqrt(d)
    score = score.masked_fill(torch.arange(L, device="cuda") >= s["lens"][:, None, None, None], -math.inf)
    if "prefix" in s:
        P = c["P"]
        pre = [_values(s["prefix"][n], c["fmt"])[0, :, :P].float() * s["prefix"][n + "s"][0, :, :P, None] for n in ("K", "V")]
        score = torch.cat([q @ pre[0].transpose(1, 2) / math.sqrt(d), score], -1)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    if "prefix" in s:
        o = p[..., :P] @ pre[1] + p[..., P:] @ own_kv[1]
    else:
        o = p @ own_kv[1]
    s["O"].copy_(o.view(B, qh, d))
    return s["O"]


def _plain_sample(s):
    x = s["logits"].double()
    V = x.shape[1]
    x = x.masked_fill(x.isnan(), -math.inf)
    top, best = x.max(1, keepdim=True)
    nothing = top == -math.inf
    greedy = s["temp"][:, None] <= 0
    temp = torch.where(greedy, 1.0, s["temp"].double()[:, None])
    w = torch.exp((x - torch.where(nothing, 0.0, top)) / temp)
    ranked, order = torch.sort(w, dim=1, descending=True, stable=True)
    rank = torch.arange(V, device="cuda")
    k = s["top_k"][:, None].long()
    ranked = ranked.masked_fill((k > 0) & (rank >= k), 0.0)
    before = ranked.cumsum(1) - ranked
    total = ranked.sum(1, keepdim=True)
    p, least = s["top_p"].double()[:, None], s["min_p"].double()[:, None]
    keep = (ranked > 0) & ((p >= 1) | (before < p * total)) & (ranked >= least * ranked[:, :1])
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ranked, 0.0))
    cum = kept.cumsum(1)
    total = kept.sum(1, keepdim=True)
    pick = (cum <= s["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    logp = torch.log(kept.gather(1, pick) / total)
    best = (x == top).to(torch.uint8).argmax(1, keepdim=True)   # the first of equal ones
    pick, logp = torch.where(greedy, best, pick), torch.where(greedy, 0.0, logp)
    s["ids"].copy_(torch.where(nothing, -1, pick)[:, 0])
    s["logp"].copy_(torch.where(nothing, -math.inf, logp)[:, 0])
    return [s["ids"], s["logp"]]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "append":
        return _plain_append(state)
    if op == "read":
        return _plain_read(state)
    return _plain_sample(state) if op == "sample" else _plain_attend(state)


# ---------------------------------------------------------------- the definition in 64 bits

_E4M3 = np.array([(-1.0 if c & 128 else 1.0) * ((c & 7) / 8 * 2.0 ** -6 if not c & 120 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                  for c in range(256)])
_INT8 = np.arange(256, dtype=np.uint8).view(np.int8).astype(np.float64)


def _decode(codes, fmt):
    table = torch.from_numpy(_E4M3 if fmt == E4M3 else _INT8).to(codes.device)
    return table[codes.long()]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(s)
    if op == "read":
        c, at = s["cache"], slice(case["first"], case["first"] + case["count"])
        return [_decode(c[n][1, :, at], case["fmt"]) * c[n + "s"][1, :, at].double().unsqueeze(-1) for n in ("K", "V")]
    if op == "sample":
        return _exact_sample(s)
    B, qh, kvh, d = case["B"], case["qh"], case["kvh"], case["d"]
    G, out = qh // kvh, torch.zeros(case["B"], case["qh"], case["d"], dtype=torch.float64, device="cuda")
    for b in range(B):
        slot, n = int(s["slot"][b]), int(s["lens"][b])
        for h in range(kvh):
            rows = [(s["cache"], slot, n)] + ([(s["prefix"], 0, case["P"])] if op == "prefix" else [])
            k, v = (torch.cat([_decode(c[m][i, h, :j], case["fmt"]) * c[m + "s"][i, h, :j].double()[:, None] for c, i, j in rows])
                    for m in ("K", "V"))
            a = torch.softmax(torch.einsum("gd,nd->gn", s["Q"][b, h * G:(h + 1) * G].double(), k) * d ** -0.5, 1)
            out[b, h * G:(h + 1) * G] = torch.einsum("gn,nd->gd", a, v)
    return out


def _exact_append(s):
    """Q and the scales from the definition; in the place of a code, the quotient that it rounds."""
    case = s["case"]
    T, qh, kvh, d = case["T"], case["qh"], case["kvh"], case["d"]
    h = d // 2
    x = s["qkv"].cpu().double().numpy().reshape(T, qh + 2 * kvh, d)
    slot, index, pos = (s[n].cpu().numpy() for n in ("slot", "index", "pos"))
    f = s["inv_freq"].cpu().numpy().astype(np.float64)
    if case["norm"]:
        size = np.sqrt((x * x).sum(-1, keepdims=True) / d + EPS)
        wq, wk = (s[n].cpu().double().numpy() for n in ("wq", "wk"))
        x = np.concatenate([x[:, :qh] / size[:, :qh] * wq, x[:, qh:qh + kvh] / size[:, qh:qh + kvh] * wk, x[:, qh + kvh:]], 1)
    z = (x[:, :qh + kvh, :h] + 1j * x[:, :qh + kvh, h:]) * np.exp(1j * pos[:, None, None].astype(np.float64) * f)
    y = np.concatenate([np.concatenate([z.real, z.imag], -1), x[:, qh + kvh:]], 1)
    cache = s["cache"]
    out = {"K": _decode(cache["K"], E4M3).cpu().numpy(), "V": _decode(cache["V"], E4M3).cpu().numpy(),
           "Ks": cache["Ks"].cpu().double().numpy(), "Vs": cache["Vs"].cpu().double().numpy(),
           "Q": s["Q"].cpu().double().numpy()}
    live = slot >= 0
    out["Q"][live] = y[live, :qh]
    for n, part in (("K", y[live, qh:qh + kvh]), ("V", y[live, qh + kvh:])):
        size = np.abs(part).max(-1)
        out[n + "s"][slot[live], :, index[live]] = size / 448.0
        out[n][slot[live], :, index[live]] = part / size[..., None] * 448.0
    return out


def _exact_sample(s):
    x = s["logits"].double().cpu().numpy()
    temp, top_k, top_p, min_p, u = (s[n].cpu().numpy().astype(np.float64) for n in ("temp", "top_k", "top_p", "min_p", "u"))
    ids, logp = np.full(len(x), -1, np.int64), np.full(len(x), -np.inf)
    for b, row in enumerate(x):
        if not (row > -np.inf).any():
            continue
        if temp[b] <= 0:
            ids[b], logp[b] = int(np.argmax(row)), 0.0
            continue
        order = np.argsort(-row, kind="stable")
        w = np.exp((row[order] - row[order[0]]) / temp[b])
        if top_k[b] > 0:
            w, order = w[:int(top_k[b])], order[:int(top_k[b])]
        n = len(w)
        if top_p[b] < 1:
            n = 1 + int(np.searchsorted(np.cumsum(w)[:-1], top_p[b] * w.sum(), side="left"))
        n = min(n, int((w >= min_p[b]).sum()), int((w > 0).sum()))
        by_id = np.sort(order[:n])
        v = np.exp((row[by_id] - row.max()) / temp[b])
        at = int(np.searchsorted(np.cumsum(v), u[b] * v.sum(), side="right"))
        ids[b], logp[b] = by_id[min(at, n - 1)], math.log(v[min(at, n - 1)] / v.sum())
    return [ids, logp]
