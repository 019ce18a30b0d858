"""Ragged steps over the 8-bit cache: the plan, attention of packed rows and of
trees, the walk down the trees and the closing up, against their definitions;
and a serving loop of all of them against one that decodes token by token."""

import random

import numpy as np
import pytest
import torch

import kv8_ref as ref
import kv8_step_ref as step
from kv8_ref import E4M3, INT8

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0 ** -8    # a bf16 rounding, relative to the value
FORMATS = [pytest.param(E4M3, id="e4m3"), pytest.param(INT8, id="int8")]
FILL = 5.0


@pytest.fixture(scope="module")
def bm():
    import bit_moe_decode_w4a16_gb300 as m
    m.build()
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """A step's device vectors and what the plan made of them."""

    def __init__(self, bm, cache, qh, slots, lens, counts, T, parents=None, plan=True):
        self.bm, self.cache, self.qh, self.B, self.T = bm, cache, qh, len(slots), T
        self.host = (list(slots), list(lens), list(counts))
        self.slots, self.lens, self.counts = _i32(slots), _i32(lens), _i32(counts)
        self.host_parents = parents
        self.parents = None if parents is None else _i32(parents)
        new = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
        self.out = {"row_start": new(self.B + 1), "after": new(self.B), "row_slot": new(T), "row_index": new(T), "row_pos": new(T)}
        self.handle = bm.kv8_cache(**cache)
        n = bm.kv8_plan_bytes(self.B, T, qh, cache["kv_heads"])
        self.plan = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")
        ws = bm.kv8_rows_workspace_bytes(self.B, T, qh, cache["kv_heads"], cache["head_dim"], cache["ctx_cap"])
        self.ws = torch.full((ws,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN records
        if plan:
            self.make()

    def make(self, stream=None):
        o = self.out
        self.bm.kv8_plan(self.handle, self.qh, self.slots, self.lens, self.counts, o["row_start"], o["after"], o["row_slot"], o["row_index"],
                         o["row_pos"], self.plan, parents=self.parents, stream=stream)

    def attend(self, Q, O=None, scale=None, stream=None):
        O = torch.full_like(Q, FILL) if O is None else O
        self.bm.kv8_attend_rows(self.handle, self.plan, Q, O, self.B, self.ws, scale=scale, stream=stream)
        return O

    def want(self):
        c = self.cache
        return step.plan(*self.host, self.T, c["slots"], c["ctx_cap"], self.host_parents)

    def check(self, Q, O, scale=None):
        _, streams = self.want()
        d = Q.shape[2]
        o, bound, live = step.attend(self.cache, Q, self.host[0], self.host[1], streams, d ** -0.5 if scale is None else scale, self.host_parents)
        assert (O[~live] == FILL).all()
        err = (O[live].double() - o[live]).abs()
        tol = BF16_HALF * o[live].abs() + bound[live] * (1 + BF16_HALF)
        assert O[live].isfinite().all()
        assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


def _rows(T, qh, d, seed=3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(T, qh, d, generator=g, device="cuda").bfloat16()


def _tree(n, rs, wide=6):
    return [-1 if j == 0 else max(0, j - 1 - rs.randrange(wide)) for j in range(n)]


def _filled(fmt, lens, counts, kvh, d, seed, extra=3, slots=None):
    """A cache whose slot b holds what stream b attends to, and spoilt positions behind it."""
    n = len(lens)
    cap = max(a + max(b, 0) for a, b in zip(lens, counts)) + extra
    cache = ref.random_cache(fmt, n, cap, kvh, d, seed)
    for b, s in enumerate(range(n) if slots is None else slots):
        _spoil(cache, s, lens[b] + max(counts[b], 0))
    return cache


def _spoil(cache, slot, n):
    """What is behind a stream's last position must not matter."""
    for m in ("K", "V"):
        cache[m][slot, :, n:] = 0xFF
        cache[m + "s"][slot, :, n:] = float("nan")


# ---------------------------------------------------------------- plan

HEAD = np.dtype([(n, np.int32) for n in ("magic", "B", "T", "qh", "kvh", "slots", "cap", "items", "units")] + [("pad", np.int32, 7)])
ITEM = np.dtype([("who", np.uint32), ("what", np.uint32), ("t0", np.int32), ("t1", np.int32)])


def _check_pieces(s, streams):
    """Every tile of every block exactly once, the longest pieces first."""
    raw = s.plan.cpu().numpy()
    head = raw[:64].view(HEAD)[0]
    kvh = s.cache["kv_heads"]
    G = s.qh // kvh
    items = raw[64 + 64 * s.B + (s.T + 1) // 2 * 16:].view(ITEM)[:head["items"]]
    seen = {}
    size = []
    for it in items:
        b, kh, block = it["who"] & 1023, it["who"] >> 10, it["what"] & 65535
        seen.setdefault((int(b), int(kh), int(block)), []).append((int(it["t0"]), int(it["t1"]), int(it["what"] >> 16)))
        size.append((it["t1"] - it["t0"]) * (1 + (streams[b][1] * G - block * 256 > 128)))
    keys = set()
    for b, (_, n, tree) in enumerate(streams):
        for block in range((n * G + 255) // 256):
            rows = min(n, (min(n * G, 256 * block + 256) - 1) // G + 1)
            ext = -(-(s.host[1][b] + (n if tree else rows)) // 128)
            for kh in range(kvh):
                keys.add((b, kh, block))
                at = 0
                parts = sorted(seen[(b, kh, block)])
                for c, (t0, t1, what) in enumerate(parts):
                    assert t0 == at and t1 > t0 and what == (65535 if len(parts) == 1 else c)
                    at = t1
                assert at == ext
    assert keys == set(seen)
    shift = 0
    while (2 * -(-s.cache["ctx_cap"] // 128) + 8) >> shift >= 1024:
        shift += 1
    cost = [int(x + 6) >> shift for x in size]
    assert cost == sorted(cost, reverse=True)


def _check_plan(s):
    want, streams = s.want()
    for n, v in want.items():
        assert s.out[n].tolist() == v, n
    _check_pieces(s, streams)


def _planned(bm, slots, lens, counts, T, num_slots, cap, qh, kvh, parents=None):
    z = lambda *s, t=torch.uint8: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    cache = {"format": E4M3, "slots": num_slots, "ctx_cap": cap, "kv_heads": kvh, "head_dim": 64, "K": z(num_slots, kvh, cap, 64),
             "V": z(num_slots, kvh, cap, 64), "Ks": z(num_slots, kvh, cap, t=torch.float32), "Vs": z(num_slots, kvh, cap, t=torch.float32)}
    return Step(bm, cache, qh, slots, lens, counts, T, parents)


@pytest.mark.parametrize("B,T,n,cap,qh,kvh", [(1, 1, 1, 10, 2, 1), (3, 60, 20, 300, 8, 2), (1, 700, 700, 5000, 16, 2), (40, 900, 33, 400, 4, 4),
                                              (200, 5000, 40, 200, 12, 4), (1024, 3000, 5, 40, 8, 1), (7, 9000, 1500, 9000, 64, 8),
                                              (2, 40, 20, 40000, 2, 2)])
def test_plan_runs(bm, B, T, n, cap, qh, kvh):
    rs = random.Random(B * T)
    slots = [rs.randrange(B + 2) for _ in range(B)]
    counts = [rs.choice([0, 1, rs.randrange(n + 1)]) for _ in range(B)]
    lens = [rs.randrange(cap - c + 1) for c in counts]
    _check_plan(_planned(bm, slots, lens, counts, T, B + 2, cap, qh, kvh))


@pytest.mark.parametrize("B,n,wide", [(1, 1, 1), (2, 64, 1), (5, 64, 64), (33, 17, 3), (300, 40, 6), (1024, 4, 2)])
def test_plan_trees(bm, B, n, wide):
    """Chains (64 deep), stars, and trees between; runs among them."""
    rs = random.Random(n)
    counts = [rs.randrange(n + 1) if b else n for b in range(B)]
    lens = [rs.randrange(0, 200) for _ in range(B)]
    parents = []
    for b, c in enumerate(counts):
        p = _tree(c, rs, wide)
        if c and b % 5 == 4:
            p[0] = -2
            p[1:] = [99] * (c - 1)         # not read
        if c > 3 and b % 7 == 3:
            p[2] = -1                      # a second root
        parents += p
    T = len(parents) + 3
    _check_plan(_planned(bm, list(range(B)), lens, counts, T, B, 300, 8, 2, parents + [5, -1, 7]))


def test_plan_refuses_streams_by_themselves(bm):
    cap, T = 100, 90
    #          fits  slot  slot  len  count  cap  fits  sits out  fits  cap exactly  behind T  behind T  empty behind T
    slots = [3, -1, 9, 4, 5, 6, 7, 8, 0, 1, 2, 2, 2]
    lens = [10, 0, 0, -1, 5, 95, 0, 40, 100, 90, 0, 0, 7]
    counts = [5, 3, 4, 2, -6, 6, 20, 0, 0, 10, 45, 1, 0]
    s = _planned(bm, slots, lens, counts, T, 9, cap, 8, 2)
    _check_plan(s)
    assert s.out["after"].tolist() == [15, -1, -1, -1, -1, -1, 20, 40, 100, 100, -1, -1, 7]
    big = 2 ** 31 - 1
    s = _planned(bm, [0, 1, 2, big], [0, big, 3, 0], [big, big, big, 1], 10, 4, cap, 8, 2)
    _check_plan(s)
    assert s.out["after"].tolist() == [-1, -1, -1, -1] and s.out["row_start"].tolist() == [0, 10, 10, 10, 10]


def test_plan_refuses_what_is_no_tree(bm):
    trees = [[-1, 0, 1], [-1, 1, 0], [0, 0], [-1, 0, 5], [-3], [-1, -2], [-1] + [0] * 64, [-2] + [0] * 64, [2 ** 31 - 1], [-1, 0, 0]]
    parents = [p for t in trees for p in t]
    s = _planned(bm, list(range(10)), [4] * 10, [len(t) for t in trees], len(parents), 10, 200, 8, 2, parents)
    _check_plan(s)
    assert [a >= 0 for a in s.out["after"].tolist()] == [True, False, False, False, False, False, False, True, False, True]


def test_plan_without_rotary_positions(bm):
    s = _planned(bm, [0, 1], [3, 4], [2, 2], 5, 2, 20, 8, 2)
    pos = s.out["row_pos"].clone()
    s.out["row_pos"].fill_(-9)
    o = s.out
    bm.kv8_plan(s.handle, 8, s.slots, s.lens, s.counts, o["row_start"], o["after"], o["row_slot"], o["row_index"], None, s.plan)
    assert (o["row_pos"] == -9).all() and torch.equal(o["row_index"], pos)


# ---------------------------------------------------------------- attention of runs

LENGTHS = [1, 2, 7, 8, 15, 16, 17, 31, 33, 64, 127, 128, 129, 200, 255, 256, 257, 300]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("qh,kvh,d", [(32, 4, 128), (8, 2, 64), (12, 4, 128), (4, 4, 64), (16, 2, 64), (7, 1, 128), (2, 1, 64), (10, 2, 128)])
def test_prompts(bm, fmt, qh, kvh, d):
    """Whole prompts of many lengths, packed, with padding behind them."""
    counts, lens = LENGTHS + [0, 5], [0] * (len(LENGTHS) + 2)
    slots = list(torch.randperm(len(counts), generator=torch.Generator().manual_seed(qh)).tolist())
    cache = _filled(fmt, lens, counts, kvh, d, 21, slots=slots)
    T = sum(counts) + 3
    s = Step(bm, cache, qh, slots, lens, counts, T)
    Q = _rows(T, qh, d)
    s.check(Q, s.attend(Q))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("qh,kvh,d", [(32, 4, 128), (8, 2, 64), (12, 4, 64), (4, 4, 128), (8, 1, 128), (1, 1, 64)])
def test_chunks_behind_positions(bm, fmt, qh, kvh, d):
    """Parts of prompts and single tokens behind what their streams hold; refused and empty streams among them."""
    counts = [1, 1, 1, 16, 17, 40, 128, 200, 3, 0, 4, 4, 33]
    lens = [0, 1, 4000, 127, 128, 1000, 2048, 5, 511, 40, -1, 9, 2049]
    slots = list(range(13))
    cache = _filled(fmt, lens, counts, kvh, d, 22)
    slots[11] = 13
    T = sum(counts)
    s = Step(bm, cache, qh, slots, lens, counts, T)
    Q = _rows(T, qh, d)
    s.check(Q, s.attend(Q))


# pieces: one to a block, evenly cut, cut along the line of blocks
@pytest.mark.parametrize("fmt,qh,kvh,d,n,base", [(E4M3, 8, 1, 128, 1, 40001), (INT8, 32, 4, 128, 16, 33000), (E4M3, 8, 2, 64, 70, 20000),
                                                 (E4M3, 32, 4, 128, 700, 9000), (INT8, 16, 2, 64, 1300, 8191), (E4M3, 4, 4, 128, 3000, 6500),
                                                 (E4M3, 32, 4, 128, 2100, 0), (INT8, 8, 8, 64, 999, 30000)])
def test_long_streams(bm, fmt, qh, kvh, d, n, base):
    cache = ref.random_cache(fmt, 2, base + n + 2, kvh, d, 23)
    _spoil(cache, 1, base + n)
    s = Step(bm, cache, qh, [1], [base], [n], n)
    Q = _rows(n, qh, d)
    s.check(Q, s.attend(Q))


def test_single_rows_agree_with_decode_attention(bm):
    """A step of one row each: what kv8_attend computes, within both calls' bounds."""
    lens = [0, 1, 126, 127, 128, 500, 1023, 3000]
    cache = _filled(E4M3, lens, [1] * 8, 4, 128, 24)
    s = Step(bm, cache, 32, list(range(8)), lens, [1] * 8, 8)
    Q = _rows(8, 32, 128)
    O = s.attend(Q)
    s.check(Q, O)
    P = torch.empty_like(Q)
    ws = torch.empty(bm.kv8_workspace_bytes(8, 32, 4, 128, cache["ctx_cap"]), dtype=torch.uint8, device="cuda")
    bm.kv8_attend(s.handle, Q, s.slots, s.out["after"], P, ws)
    s.check(Q, P)


# ---------------------------------------------------------------- attention of trees

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("qh,kvh,d", [(32, 4, 128), (8, 2, 64), (12, 4, 128), (4, 4, 64), (5, 1, 128)])
def test_trees(bm, fmt, qh, kvh, d):
    rs = random.Random(qh)
    counts = [1, 2, 13, 16, 17, 31, 32, 33, 63, 64, 64, 0, 5, 20, 200]
    lens = [0, 127, 0, 100, 4000, 128, 65, 90, 1000, 64, 3, 7, 50, 250, 333]
    parents = []
    for b, n in enumerate(counts):
        p = _tree(n, rs, [1, 3, 64][b % 3])
        if b == 12:
            p[3] = -1                      # a second root
        if b == 13:
            p[4] = 9                       # no tree: refused
        if b == 14:
            p[0] = -2                      # a run in a step of trees
        parents += p
    cache = _filled(fmt, lens, counts, kvh, d, 25)
    T = len(parents) + 2
    s = Step(bm, cache, qh, list(range(len(counts))), lens, counts, T, parents + [0, 0])
    _check_plan(s)
    Q = _rows(T, qh, d)
    s.check(Q, s.attend(Q))


@pytest.mark.parametrize("fmt,d,code", [(E4M3, 128, 0x7F), (E4M3, 64, 0xFF), (INT8, 128, 0x80)])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_what_a_row_does_not_attend_to_does_not_touch_it(bm, fmt, d, code, scale):
    """NaN codes and any scale at a sibling's position, and in a run at later rows' positions."""
    for base in (0, 100, 127, 300):
        n = 40
        cache = _filled(fmt, [base, base], [n, n], 2, d, 26)
        for at in (5, 28):                 # row 5 and row 28 of either stream
            for m in ("K", "V"):
                cache[m][:, :, base + at] = code
                cache[m + "s"][:, :, base + at] = scale
        parents = [-1] + [0] * 5 + [max(j - 7, 1) for j in range(6, n)]   # 5 has descendants: 12, 19, ...
        s = Step(bm, cache, 8, [0, 1], [base, base], [n, n], 2 * n, parents + [-2] + [0] * (n - 1))
        Q = _rows(2 * n, 8, d)
        O = s.attend(Q)
        _, streams = s.want()
        hidden = torch.cat([~step.see(n, parents)[:, [5, 28]].any(1), torch.arange(n) < 5]).cuda()
        o, bound, _ = step.attend(cache, Q, [0, 1], [base, base], streams, d ** -0.5, s.host_parents)
        tol = BF16_HALF * o.abs() + bound * (1 + BF16_HALF)
        assert hidden.sum() > 20
        assert O[hidden].isfinite().all() and ((O.double() - o).abs() <= tol)[hidden].all()


def test_nan_stays_with_the_rows_that_attend_to_it(bm):
    cache = _filled(E4M3, [200, 200], [20, 20], 2, 128, 27)
    cache["Ks"][1, 0, 100] = float("nan")
    s = Step(bm, cache, 16, [0, 1], [200, 200], [20, 20], 40)
    Q = _rows(40, 16, 128)
    Q[3, 2, 7] = float("nan")
    Q[4, 3, 1] = float("inf")
    O = s.attend(Q)
    bad = torch.zeros(40, 16, dtype=torch.bool, device="cuda")
    bad[20:, :8] = bad[3, 2] = bad[4, 3] = True
    assert O[bad].isnan().all() and O[~bad].isfinite().all()


@pytest.mark.parametrize("fmt,qh,kvh,d,n,base", [(E4M3, 16, 2, 128, 40, 700), (INT8, 8, 1, 64, 33, 0), (E4M3, 32, 4, 128, 700, 100)])
def test_spoilt_query_rows_leave_their_neighbours(bm, fmt, qh, kvh, d, n, base):
    """NaN and infinities in a few heads of a few rows: the same warps' other rows are as near as ever."""
    cache = _filled(fmt, [base], [n], kvh, d, 28)
    s = Step(bm, cache, qh, [0], [base], [n], n)
    Q = _rows(n, qh, d)
    bad = torch.zeros(n, qh, dtype=torch.bool, device="cuda")
    for j, h, x in ((3, 2, "nan"), (4, 3, "inf"), (5, 0, "-inf"), (n - 1, qh - 1, "inf"), (n // 2, 1, "nan")):
        bad[j, h] = True
        Q[j, h, (5 * j + h) % d] = float(x)
    O = s.attend(Q)
    assert O[bad].isnan().all()
    Q[bad] = 0
    O[bad] = s.attend(Q)[bad]
    s.check(Q, O)


def test_streams_of_one_slot(bm):
    """A slot that several streams of a step read, their rows at positions of their own; one stream's rows lie among another's past."""
    lens, counts = [0, 300, 100, 300, 700], [100, 40, 200, 1, 64]
    cache = ref.random_cache(E4M3, 1, 800, 2, 128, 30)
    s = Step(bm, cache, 16, [0] * 5, lens, counts, sum(counts))
    Q = _rows(sum(counts), 16, 128)
    s.check(Q, s.attend(Q))


# ---------------------------------------------------------------- magnitudes

@pytest.mark.parametrize("seed", [0, 1, 47, 51, 89, 99, 114, 148, 179, 181, 205, 241, 259, 297])
def test_peaked_and_uneven_values(bm, seed):
    """Scores far apart, V scales over 12 binary orders, heads of zeros."""
    torch.manual_seed(seed)
    fmt = seed & 1
    lens, counts = [600, 300, 0], [5, 64, 200]
    cache = ref.random_cache(fmt, 3, 700, 2, 128, 28 + seed, spread=0.0)
    cache["Vs"] *= torch.exp2(torch.randint(-6, 7, cache["Vs"].shape, device="cuda").float())
    cache["Ks"] *= torch.exp2(torch.randint(-4, 5, cache["Ks"].shape, device="cuda").float())
    cache["K"][0, 0, 10:50] = 0
    cache["Ks"][0, 0, 10:50] = 0
    cache["V"][1] = 0
    cache["Vs"][1] = 0
    s = Step(bm, cache, 16, [0, 1, 2], lens, counts, 269)
    Q = (4 * _rows(269, 16, 128, seed).float()).bfloat16()
    O = s.attend(Q)
    s.check(Q, O)
    assert (O[5:69] == 0).all()


@pytest.mark.parametrize("exp", [-100, -40, 40, 95])
def test_extreme_scales(bm, exp):
    """Values far from 1: the output has V's magnitude, whatever it is."""
    cache = ref.random_cache(E4M3, 1, 300, 1, 64, 29)
    cache["Vs"] *= 2.0 ** exp
    cache["Ks"] *= 2.0 ** 20
    Q = (_rows(40, 8, 64).float() * 2.0 ** -20).bfloat16()
    s = Step(bm, cache, 8, [0], [260], [40], 40)
    s.check(Q, s.attend(Q))


@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("fmt,d", [(E4M3, 128), (INT8, 64)])
def test_rising_and_falling_scores(bm, fmt, d, up):
    """Scores that rise by 2 a tile move the reference again and again; falling ones never do."""
    n = 2500
    cache = ref.random_cache(fmt, 1, n, 1, d, 30, spread=0.0)
    g = torch.linspace(0.02, 1.0, n, device="cuda")
    cache["K"][0, 0] = cache["K"][0, 0, 0]
    cache["Ks"][0, 0] = cache["Ks"][0, 0, 0] * (g if up else g.flip(0))
    k = ref.decode(cache["K"][0, 0, 0], fmt) * cache["Ks"][0, 0].max().double()
    q = (k * 40 * d ** 0.5 / k.square().sum()).bfloat16()            # scores from 1 to 40
    Q = q.expand(100, 8, d).contiguous()
    s = Step(bm, cache, 8, [0], [n - 100], [100], 100)
    s.check(Q, s.attend(Q))


# positions of a tile of 128 fall to different threads, tiles to different warps and pieces
@pytest.mark.parametrize("exp", [-90, 0, 27, 95])
@pytest.mark.parametrize("fmt,d", [(E4M3, 128), (INT8, 64)])
@pytest.mark.parametrize("n,live", [(129, [128]), (128, [127]), (301, [300]), (600, [0]), (1513, [40, 1100]), (2, [1])])
def test_heads_of_zeros_keep_their_share(bm, fmt, d, n, live, exp):
    """Positions whose V is zero weigh in the denominator, whatever the magnitude of the others."""
    cache = ref.random_cache(fmt, 1, n, 2, d, 31)
    dead = torch.ones(n, dtype=torch.bool, device="cuda")
    dead[live] = False
    cache["V"][0, :, dead] = 0
    cache["Vs"][0, :, dead] = 0
    cache["Vs"][0, :, ~dead] = 2.0 ** exp
    Q = torch.cat([torch.zeros(1, 8, d, device="cuda").bfloat16(), _rows(1, 8, d)])
    s = Step(bm, cache, 8, [0], [n - 2], [2], 2)
    s.check(Q, s.attend(Q))


@pytest.mark.parametrize("exp", [-127, -60, 60, 127])
def test_query_rows_of_any_magnitude(bm, exp):
    cache = ref.random_cache(E4M3, 1, 200, 2, 64, 32)
    cache["Ks"] *= 2.0 ** -min(max(exp, -100), 100)
    Q = (_rows(50, 8, 64).double().clamp(-1.5, 1.5) * 2.0 ** exp).bfloat16()
    s = Step(bm, cache, 8, [0], [150], [50], 50)
    s.check(Q, s.attend(Q))


def test_another_score_factor(bm):
    cache = _filled(INT8, [100], [50], 2, 64, 33)
    s = Step(bm, cache, 8, [0], [100], [50], 50)
    Q = _rows(50, 8, 64)
    s.check(Q, s.attend(Q, scale=0.3), scale=0.3)


# ---------------------------------------------------------------- the call

def test_rows_do_not_depend_on_the_rest_of_the_step(bm):
    rs = random.Random(5)
    counts = [1, 16, 40, 300, 64, 7, 500, 1] + [rs.randrange(1, 30) for _ in range(30)]
    lens = [3000, 2900, 0, 700, 2048, 100, 0, 5] + [rs.randrange(0, 3000) for _ in range(30)]
    parents = []
    for b, n in enumerate(counts):
        parents += _tree(n, rs) if n <= 64 and b % 2 else [-2] + [0] * (n - 1)
    cache = _filled(E4M3, lens, counts, 4, 128, 34)
    T = sum(counts)
    s = Step(bm, cache, 32, list(range(38)), lens, counts, T, parents)
    Q = _rows(T, 32, 128)
    whole = s.attend(Q)
    assert torch.equal(whole, s.attend(Q))
    start = s.out["row_start"].tolist()
    for b in (0, 1, 3, 4, 6, 12, 37):
        a, z = start[b], start[b + 1]
        solo = Step(bm, cache, 32, [b], [lens[b]], [counts[b]], z - a, parents[a:z])
        assert torch.equal(solo.attend(Q[a:z].clone()), whole[a:z])


def test_a_plan_of_other_sizes_leaves_everything(bm):
    cache = _filled(E4M3, [10, 20], [5, 6], 2, 64, 35)
    s = Step(bm, cache, 8, [0, 1], [10, 20], [5, 6], 11, [-1] * 5 + [-1, 0, 1, 2, 3, 4])
    Q = _rows(11, 8, 64)
    other = {n: (v[:1].contiguous() if torch.is_tensor(v) else v) for n, v in cache.items()}
    other["slots"] = 1
    O = torch.full_like(Q, FILL)
    bm.kv8_attend_rows(bm.kv8_cache(**other), s.plan, Q, O, 2, s.ws)                       # another cache
    bm.kv8_attend_rows(s.handle, s.plan, Q, O, 1, s.ws)                                    # another B
    bm.kv8_attend_rows(s.handle, s.plan, Q[:10].clone(), O[:10], 2, s.ws)                  # another T
    half = torch.full((11, 4, 64), FILL, dtype=torch.bfloat16, device="cuda")
    bm.kv8_attend_rows(s.handle, s.plan, half.clone(), half, 2, s.ws)                      # other heads
    blank = torch.zeros_like(s.plan)
    bm.kv8_attend_rows(s.handle, blank, Q, O, 2, s.ws)                                     # no plan
    assert (O == FILL).all() and (half == FILL).all()
    path, kept = torch.zeros(2, 64, dtype=torch.int32, device="cuda"), _i32([3, 3])
    path[:, :3] = _i32([0, 2, 4])
    before = {n: cache[n].clone() for n in ("K", "V", "Ks", "Vs")}
    bm.kv8_tree_keep(s.handle, blank, path, kept)
    bm.kv8_tree_keep(bm.kv8_cache(**other), s.plan, path, kept)
    bm.kv8_tree_keep(s.handle, s.plan, path[:1].clone(), kept[:1].clone())
    for n, v in before.items():
        assert torch.equal(v.view(torch.uint8), cache[n].view(torch.uint8))
    out = [torch.full(k, -7, dtype=torch.int32, device="cuda") for k in ((2, 64), (2,), (2, 64), (2,), (2,))]
    ids = torch.zeros(11, dtype=torch.int32, device="cuda")
    bm.kv8_tree_accept(blank, ids, ids, *out)
    bm.kv8_tree_accept(s.plan, ids[:10].clone(), ids[:10].clone(), *out)
    assert all((x == -7).all() for x in out)


def test_graph_replays_with_other_lengths(bm):
    """Plan and attention captured once, replayed with each step's own lengths; two graphs in turn, a workspace each."""
    lens, counts = [100, 3000, 40], [17, 5, 64]
    cache = _filled(E4M3, [3200] * 3, [64] * 3, 2, 64, 36)
    T, Q = 200, _rows(200, 8, 64)
    graphs = []
    for _ in range(2):
        s = Step(bm, cache, 8, [0, 1, 2], lens, counts, T)
        O = s.attend(Q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.make()
            s.attend(Q, O)
        graphs.append((s, O, g))
    for turn, (lens, counts) in enumerate([([5, 6, 7], [64, 64, 64]), ([3000, 0, 1], [1, 100, 0]), ([0, 0, 0], [0, 0, 0]), ([2900, 2000, 3], [1, 1, 9])]):
        s, O, g = graphs[turn % 2]
        O.fill_(FILL)
        for v, x in ((s.lens, lens), (s.counts, counts)):
            v.copy_(_i32(x))
        s.host = ([0, 1, 2], lens, counts)
        g.replay()
        torch.cuda.synchronize()
        _check_plan(s)
        s.check(Q, O)


def test_streams_that_overlap(bm):
    """Calls on two streams share a plan and run at once, with workspaces of their own."""
    lens, counts = [4000, 1000], [16, 100]
    cache = _filled(INT8, lens, counts, 4, 128, 37)
    s = Step(bm, cache, 32, [0, 1], lens, counts, 116)
    Q = _rows(116, 32, 128)
    want = s.attend(Q)
    torch.cuda.synchronize()
    ws = [s.ws.clone(), s.ws.clone()]
    streams, O = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.full_like(Q, FILL) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for k in range(2):
            bm.kv8_attend_rows(s.handle, s.plan, Q, O[k], 2, ws[k], stream=streams[k])
    torch.cuda.synchronize()
    assert torch.equal(O[0], want) and torch.equal(O[1], want)


def test_offsets_past_32_bits(bm):
    """A cache whose codes pass 2^31 bytes: attended and closed up behind that point."""
    kvh, d, cap, slots = 2, 128, 3_000_000, 3
    c = {"format": E4M3, "slots": slots, "ctx_cap": cap, "kv_heads": kvh, "head_dim": d}
    for n in ("K", "V"):
        c[n] = torch.zeros(slots, kvh, cap, d, dtype=torch.uint8, device="cuda")
        c[n + "s"] = torch.zeros(slots, kvh, cap, device="cuda")
    small = ref.random_cache(E4M3, 1, 40, kvh, d, 38)
    for n in ("K", "V", "Ks", "Vs"):
        c[n][2, :, cap - 40:] = small[n][0]
    c["K"][2, :, cap - 40:] = 0              # all scores are 0: every position has the same weight
    n = 20
    s = Step(bm, c, 4, [2], [cap - n], [n], n, _tree(n, random.Random(1)))
    Q = _rows(n, 4, d)
    O = s.attend(Q)
    v = ref.decode(c["V"][2, :, cap - 40:], E4M3) * c["Vs"][2, :, cap - 40:].double().unsqueeze(-1)
    see = step.see(n, s.host_parents).double().cuda()
    total = cap - n + see.sum(1)
    want = (v[:, :40 - n].sum(1, keepdim=True) + torch.einsum("ji,hid->hjd", see, v[:, 40 - n:])) / total[None, :, None]
    size = v.abs().sum(1)[:, None] / cap
    want, size = (x.transpose(0, 1).repeat_interleave(2, 1) for x in (want, size))
    assert ((O.double() - want).abs() <= BF16_HALF * want.abs() + size * 2.0 ** -10).all()
    path, kept = torch.full((1, 64), -1, dtype=torch.int32, device="cuda"), _i32([3])
    path[0, :3] = _i32([0, 7, 19])
    before = c["V"][2, :, cap - 40:].clone()
    bm.kv8_tree_keep(s.handle, s.plan, path, kept)
    got = c["V"][2, :, cap - 40:]
    assert torch.equal(got[:, 21], before[:, 27]) and torch.equal(got[:, 22], before[:, 39]) and torch.equal(got[:, 23:], before[:, 23:])


@pytest.mark.parametrize("fmt,qh,kvh,d,most", [(E4M3, 32, 8, 128, 128), (INT8, 8, 8, 64, 128), (E4M3, 16, 4, 64, 300)])
def test_many_short_streams(bm, fmt, qh, kvh, d, most):
    """More pieces of one tile than the GPU has SMs, many times over, some of two or three tiles among them: a CTA goes from one to the next."""
    rs = random.Random(most + d)
    lens = [rs.randrange(most) for _ in range(700)]
    counts = [min(rs.choice([1, 1, 2, 7, 16]), most - n) for n in lens]
    cache = _filled(fmt, lens, counts, kvh, d, 40)
    s = Step(bm, cache, qh, list(range(700)), lens, counts, sum(counts) + 3)
    Q = _rows(sum(counts) + 3, qh, d)
    O = s.attend(Q)
    s.check(Q, O)
    for _ in range(10):
        assert torch.equal(s.attend(Q), O)


def test_largest_step(bm):
    """1024 streams, some of them on one slot."""
    rs = random.Random(8)
    B = 1024
    counts, lens = [rs.randrange(0, 5) for _ in range(B)], [rs.randrange(0, 30) for _ in range(B)]
    slots = [rs.randrange(-1, 50) for _ in range(B)]
    cache = ref.random_cache(E4M3, 49, 40, 1, 64, 39)
    T = sum(counts)
    s = Step(bm, cache, 8, slots, lens, counts, T)
    Q = _rows(T, 8, 64)
    s.check(Q, s.attend(Q))


# ---------------------------------------------------------------- accept and keep

def _accepted(bm, s, tokens, ids, lens=None):
    B = s.B
    new = lambda *k: torch.full(k, -99, dtype=torch.int32, device="cuda")  # noqa: E731
    out = {"path": new(B, 64), "kept": new(B), "fresh": new(B, 64), "n_fresh": new(B), "lens": new(B) if lens is None else lens}
    bm.kv8_tree_accept(s.plan, _i32(tokens), _i32(ids), out["path"], out["kept"], out["fresh"], out["n_fresh"], out["lens"])
    return out


def _walk_case(rs, counts, vocab):
    parents, tokens, ids = [], [], []
    for n in counts:
        p = _tree(n, rs, rs.choice([1, 2, 6, 64]))
        if n and rs.random() < 0.15:
            p[0] = -2
        parents += p
        tokens += [rs.randrange(vocab) for _ in range(n)]
        ids += [rs.choice([-1, rs.randrange(vocab)]) if rs.random() < 0.1 else rs.randrange(vocab) for _ in range(n)]
    return parents, tokens, ids


@pytest.mark.parametrize("B,n,vocab", [(1, 1, 2), (1, 64, 1), (6, 13, 3), (300, 64, 2), (1024, 5, 2)])
def test_accept(bm, B, n, vocab):
    rs = random.Random(B + n)
    counts = [rs.randrange(n + 1) if b else n for b in range(B)]
    parents, tokens, ids = _walk_case(rs, counts, vocab)
    T = len(parents) + 4
    lens = [rs.randrange(0, 100) for _ in range(B)]
    slots = [b if rs.random() < 0.95 else -1 for b in range(B)]
    s = _planned(bm, slots, lens, counts, T, B, 200, 2, 1, parents + [-1] * 4)
    out = _accepted(bm, s, tokens + [1] * 4, ids + [1] * 4)
    _, streams = s.want()
    want = step.accept(streams, lens, parents, tokens, ids, [a < 0 for a in slots], [-99] * B)
    for k, v in want.items():
        assert out[k].tolist() == v, k
    if vocab == 1 and n == 64:
        assert want["kept"][0] > 1
    # the lengths may be those that the plan read
    again = _accepted(bm, s, tokens + [1] * 4, ids + [1] * 4, lens=s.lens)
    assert again["lens"].tolist() == step.accept(streams, lens, parents, tokens, ids, [a < 0 for a in slots], lens)["lens"]


def test_accept_deepest_chain(bm):
    n = 64
    s = _planned(bm, [0], [3], [n], n, 1, 100, 2, 1, list(range(-1, n - 1)))
    out = _accepted(bm, s, list(range(100, 100 + n)), list(range(101, 101 + n)))
    assert out["path"][0].tolist() == list(range(n)) and out["kept"].tolist() == [n] and out["lens"].tolist() == [3 + n]
    assert out["fresh"][0].tolist() == list(range(101, 101 + n))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kvh,d", [(4, 128), (2, 64), (1, 128)])
def test_keep(bm, fmt, kvh, d):
    rs = random.Random(kvh)
    counts = [64, 13, 1, 40, 20, 20, 20, 30, 0, 64]
    lens = [5, 0, 7, 100, 3, 3, 3, 9, 4, 0]
    parents = []
    for b, n in enumerate(counts):
        parents += _tree(n, rs) if b != 7 else [-2] + [0] * (n - 1)
    slots = list(range(10))
    slots[6] = -1
    path = [[-1] * 64 for _ in counts]
    kept = [64, 5, 1, 9, 21, 4, 3, 3, 2, 33]
    path[0] = list(range(63, -1, -1))                    # any rows in any order: all are read before any is written
    path[1][:5] = [0, 1, 4, 9, 12]
    path[2][0] = 0
    path[3][:9] = [0, 3, 3, 3, 8, 20, 21, 39, 2]
    path[4][:21] = list(range(20)) + [19]                # more than the stream has: left alone
    path[5][:4] = [0, 1, 20, 3]                          # a row it does not have: left alone
    path[6][:3] = [0, 2, 3]                              # refused
    path[7][:3] = [0, 2, 3]                              # a run
    path[8][:2] = [0, 0]                                 # no rows
    path[9][:33] = list(range(0, 64, 2)) + [63]
    cache = ref.random_cache(fmt, 10, 140, kvh, d, 40)
    before = {n: cache[n].clone() for n in ("K", "V", "Ks", "Vs")}
    s = Step(bm, cache, 2 * kvh, slots, lens, counts, len(parents), parents)
    bm.kv8_tree_keep(s.handle, s.plan, _i32(path), _i32(kept))
    for n, old in before.items():
        want = old.clone()
        for b in (0, 1, 3, 9):
            for i in range(kept[b]):
                want[b, :, lens[b] + i] = old[b, :, lens[b] + path[b][i]]
        assert torch.equal(want, cache[n]), n


def test_keep_of_nonsense_counts(bm):
    cache = ref.random_cache(E4M3, 3, 100, 2, 64, 41)
    before = {n: cache[n].clone() for n in ("K", "V", "Ks", "Vs")}
    s = Step(bm, cache, 8, [0, 1, 2], [0, 0, 0], [4, 4, 4], 12, [-1, 0, 1, 2] * 3)
    path = torch.full((3, 64), 2 ** 30, dtype=torch.int32, device="cuda")
    bm.kv8_tree_keep(s.handle, s.plan, path, _i32([2 ** 31 - 1, -2 ** 31, 3]))
    for n, old in before.items():
        assert torch.equal(old, cache[n])


# ---------------------------------------------------------------- a serving loop

@pytest.mark.parametrize("fmt,qh,kvh,d", [(E4M3, 8, 2, 64), (INT8, 32, 4, 128)])
def test_drafting_loop_gives_the_tokens_of_decoding_one_by_one(bm, fmt, qh, kvh, d):
    """A toy model (a table of qkv rows per token, and a product back to logits): prompts in parts, then trees of
    drafts, half of them right, against one token at a time through kv8_attend.

    Where two tokens are so close that the outputs' last rounding decides, the two may say different ones: a stream is
    compared up to there, and there both tokens' logits, from the output in 64 bits, have to lie within what
    the outputs may be off (2^-8 of each element and the attention's own bound, times the product's weights) of the largest."""
    V, B, cap = 50, 4, 400
    rs = random.Random(7)
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    table = torch.randn(V, (qh + 2 * kvh) * d, generator=g, device="cuda").bfloat16()
    out = torch.randn(qh * d, V, generator=g, device="cuda", dtype=torch.float64)
    rope = bm.kv8_rope(norm=True, inv_freq=(1e4 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)).float().cuda())
    prompts = [[rs.randrange(V) for _ in range(n)] for n in (3, 130, 61, 200)]
    empty = lambda: dict(ref.random_cache(fmt, B, cap, kvh, d, 1))  # noqa: E731

    def choose(O):
        logits = O.double().flatten(1) @ out
        ids = torch.empty(O.shape[0], dtype=torch.int32, device="cuda")
        z = torch.zeros(O.shape[0], device="cuda")
        bm.bm_sample(logits.float().contiguous(), z, None, None, None, z, ids)
        return ids

    # one by one
    plain = empty()
    h = bm.kv8_cache(**plain)
    ws = torch.empty(bm.kv8_workspace_bytes(B, qh, kvh, d, cap), dtype=torch.uint8, device="cuda")
    slots = _i32(range(B))
    said, asked = [[] for _ in range(B)], [[] for _ in range(B)]
    now, at = [p[0] for p in prompts], [0] * B
    while min(len(x) for x in said) < 30:
        Q, O = torch.empty(B, qh, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, qh, d, dtype=torch.bfloat16, device="cuda")
        bm.kv8_append(h, table[now], rope, slots, _i32(at), Q)
        at = [a + 1 for a in at]
        bm.kv8_attend(h, Q, slots, _i32(at), O, ws)
        ids = choose(O).tolist()
        for b in range(B):
            if at[b] < len(prompts[b]):
                now[b] = prompts[b][at[b]]
            else:
                said[b].append(ids[b])
                asked[b].append(Q[b].clone())
                now[b] = ids[b]
    # in ragged steps
    cache = empty()
    h = bm.kv8_cache(**cache)
    got, T = [[] for _ in range(B)], 256
    lens = _i32([0] * B)
    todo = [list(p) for p in prompts]
    new = lambda *k: torch.empty(k, dtype=torch.int32, device="cuda")  # noqa: E731
    start, after, rslot, rindex, rpos, counts = new(B + 1), new(B), new(T), new(T), new(T), new(B)
    path, kept, fresh, n_fresh = new(B, 64), new(B), new(B, 64), new(B)
    plan = torch.empty(bm.kv8_plan_bytes(B, T, qh, kvh), dtype=torch.uint8, device="cuda")
    ws = torch.empty(bm.kv8_rows_workspace_bytes(B, T, qh, kvh, d, cap), dtype=torch.uint8, device="cuda")
    longest = 0
    while min(len(x) for x in got) < 30:
        tokens, parents, n, part = [], [], [], []
        for b in range(B):
            if todo[b]:                    # a part of the prompt
                rows = todo[b][:70]
                todo[b] = todo[b][70:]
                tokens += rows
                parents += [-2] + [0] * (len(rows) - 1)
                part.append(bool(todo[b]))
            else:                          # the last token, and drafts: what will be said, mixed with what will not
                rows, p, tip, depth = [got[b][-1]], [-1], 0, {0: 0}
                for _ in range(rs.randrange(0, 12)):
                    right = rs.random() < 0.6
                    want = said[b][len(got[b]) + depth[tip]] if len(got[b]) + depth[tip] < len(said[b]) else 0
                    rows.append(want if right else (want + 1 + rs.randrange(V - 1)) % V)
                    p.append(tip)
                    depth[len(rows) - 1] = depth[tip] + 1
                    if right:
                        tip = len(rows) - 1
                tokens += rows
                parents += p
                part.append(False)
            n.append(len(rows))
        counts.copy_(_i32(n))
        pad = T - len(tokens)
        tok = _i32(tokens + [0] * pad)
        par = _i32(parents + [0] * pad)
        bm.kv8_plan(h, qh, slots, lens, counts, start, after, rslot, rindex, rpos, plan, parents=par)
        Q, O = torch.zeros(T, qh, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, qh, d, dtype=torch.bfloat16, device="cuda")
        bm.kv8_append(h, table[tok.long()], rope, rslot, rindex, Q, rope_pos=rpos)
        bm.kv8_attend_rows(h, plan, Q, O, B, ws)
        ids = choose(O)
        bm.kv8_tree_accept(plan, tok, ids, path, kept, fresh, n_fresh, lens)
        bm.kv8_tree_keep(h, plan, path, kept)
        for b in range(B):
            if not part[b]:
                new_ones = fresh[b, :int(n_fresh[b])].tolist()
                got[b] += new_ones
                longest = max(longest, len(new_ones))
    assert longest >= 4
    same = 0
    for b in range(B):
        k = next((i for i, (x, y) in enumerate(zip(got[b], said[b])) if x != y), min(len(got[b]), len(said[b])))
        same += k
        if k < min(len(got[b]), len(said[b])):
            o, bound = ref.attend(plain, asked[b][k][None], _i32([b]), _i32([len(prompts[b]) + k]), d ** -0.5)
            off = (BF16_HALF * o[0].abs() + bound[0] * (1 + BF16_HALF)).flatten() @ out.abs()
            logits = o[0].flatten() @ out
            for x in (got[b][k], said[b][k]):
                assert logits[x] + off[x] >= (logits - off).max()
        # up to there the cache holds the codes of decoding one by one
        held = min(int(lens[b]), at[b], len(prompts[b]) + k)
        for n in ("K", "V"):
            assert torch.equal(cache[n][b, :, :held], plain[n][b, :, :held])
            assert torch.equal(cache[n + "s"][b, :, :held], plain[n + "s"][b, :, :held])
    assert same >= 60
