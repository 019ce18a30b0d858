"""Attention of ragged steps at its largest: streams of so many blocks that none is
cut, many kv heads, and rows past 2^31 elements.  Rows are compared where
reading it all in 64 bits would take too long: the first and last, the borders of blocks and tiles, and some between."""

import random

import pytest
import torch

import kv8_ref as ref
from kv8_ref import E4M3, INT8
from test_gpu_kv8_step import BF16_HALF, FILL, FORMATS, Step, _filled, _rows, _spoil

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bm():
    import bit_moe_decode_w4a16_gb300 as m
    m.build()
    return m


def _check_rows(cache, slot, base, Q, O, rows, heads):
    """Rows `rows` (places in a stream of consecutive ones; Q and O are the stream's) of query heads `heads`, by the bound of kv8_step_ref."""
    d, kvh = Q.shape[2], cache["kv_heads"]
    G, at = Q.shape[1] // kvh, torch.tensor(rows, device="cuda")
    L = base + max(rows) + 1
    hidden = torch.arange(L, device="cuda") > base + at[:, None]
    scale = d ** -0.5
    for h in heads:
        kh = h // G
        vc, vs = ref.decode(cache["V"][slot, kh, :L], cache["format"]), cache["Vs"][slot, kh, :L].double()
        k = ref.decode(cache["K"][slot, kh, :L], cache["format"]) * cache["Ks"][slot, kh, :L].double()[:, None]
        q = Q[at, h].double()
        p = torch.softmax((q @ k.T * scale).masked_fill(hidden, -torch.inf), -1)
        off = (q.abs() @ k.abs().T).masked_fill(hidden, 0).amax(-1, keepdim=True) * scale * (d + 8) * 2.0 ** -24
        want = p @ (vc * vs[:, None])
        small = 2.0 ** -25 * (p * vs.clamp(min=2.0 ** -100)).amax(-1, keepdim=True) * ((~hidden).double() @ vc.abs())
        bound = (p @ (vc * vs[:, None]).abs()) * (2.0 ** -11 + 2.0 ** -18 + 2 * off) + small
        err, tol = (O[at, h].double() - want).abs(), BF16_HALF * want.abs() + bound * (1 + BF16_HALF)
        assert (err <= tol).all(), (h, float((err / tol).max()))


def _borders(n, base, G, seed):
    """Places around the borders of blocks of 256 query rows and of tiles of 128 positions, the ends, and others."""
    rs = random.Random(seed)
    at = {0, 1, n - 1, n - 2}
    for k in (1, 2, n * G // 512, n * G // 256):
        at |= {256 * k // G + e for e in (-1, 0, 1)}
    for k in (1, base // 128 + 1, (base + n) // 128):
        at |= {128 * k - base + e for e in (-1, 0, 1)}
    at |= {rs.randrange(n) for _ in range(40)}
    return sorted(j for j in at if 0 <= j < n)


# 608 blocks and more of a stream: whole, whatever its length
@pytest.mark.parametrize("fmt,qh,kvh,d,n,base", [(E4M3, 32, 4, 128, 8192, 0), (INT8, 32, 4, 128, 5000, 3000), (E4M3, 16, 2, 64, 10001, 40),
                                                 (INT8, 12, 4, 64, 13000, 9000), (E4M3, 8, 1, 128, 19457, 1)])
def test_streams_of_many_blocks(bm, fmt, qh, kvh, d, n, base):
    cache = ref.random_cache(fmt, 2, base + n + 3, kvh, d, 60)
    _spoil(cache, 1, base + n)
    s = Step(bm, cache, qh, [1], [base], [n], n + 1)
    Q = _rows(n + 1, qh, d)
    O = s.attend(Q)
    assert O[:n].isfinite().all() and (O[n] == FILL).all()
    _check_rows(cache, 1, base, Q, O, _borders(n, base, qh // kvh, n), {0, qh // kvh - 1, qh // 2, qh - 1})


# in long pieces references lie 2^4 and 2^8 below their maxima, weights accordingly higher
@pytest.mark.parametrize("exp,dead", [(-91, 0.0), (-91, 0.9), (0, 0.999), (0, 1.0), (100, 0.0), (100, 0.9)])
@pytest.mark.parametrize("fmt,n,base", [(E4M3, 2600, 70000), (INT8, 19500, 131072)])
def test_long_pieces_at_the_ends_of_the_scales(bm, fmt, n, base, exp, dead):
    """V scales from 2^-100 to 2^100, and positions without V, which weigh in the sum alone."""
    cache = ref.random_cache(fmt, 1, base + n, 1, 64, 63)
    cache["Vs"] *= 2.0 ** exp
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    off = torch.rand(base + n, generator=g, device="cuda") < dead
    cache["V"][0, 0, off] = 0
    cache["Vs"][0, 0, off] = 0
    s = Step(bm, cache, 8, [0], [base], [n], n)
    Q = _rows(n, 8, 64)
    O = s.attend(Q)
    assert O.isfinite().all()
    _check_rows(cache, 0, base, Q, O, [0, 1, 31, 32, 33, n // 2, n - 2, n - 1] + list(range(100, 116)), range(8))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("qh,kvh,d,counts,lens", [(16, 16, 128, [1, 40, 300, 1, 7], [5000, 0, 100, 127, 4096]), (32, 16, 64, [64, 1, 200], [2048, 9000, 0]),
                                                  (77, 77, 64, [1, 33, 260, 5], [4500, 10, 0, 4200]), (154, 77, 64, [3, 140], [6000, 128]),
                                                  (300, 300, 64, [1, 30, 270], [4100, 130, 5]), (1024, 1024, 64, [1, 20], [300, 4100]),
                                                  (1024, 128, 64, [2, 40], [4500, 0])])
def test_many_kv_heads(bm, fmt, qh, kvh, d, counts, lens):
    """One or more blocks for each of many heads: whole ones, evenly cut ones and ones cut along the line, by the heads alone."""
    cache = _filled(fmt, lens, counts, kvh, d, 61)
    T = sum(counts) + 2
    s = Step(bm, cache, qh, list(range(len(counts))), lens, counts, T)
    Q = _rows(T, qh, d)
    s.check(Q, s.attend(Q))


def test_rows_past_32_bits(bm):
    """2^20 rows of 17 heads of 128: Q and O pass 2^31 elements, the records 2^32 floats.  All streams read one slot."""
    qh, d, B, n, base = 17, 128, 1024, 1024, 20
    T = B * n
    cache = ref.random_cache(E4M3, 1, base + n + 30, qh, d, 62)
    _spoil(cache, 0, base + n)
    lens = [base - b % 3 for b in range(B)]
    s = Step(bm, cache, qh, [0] * B, lens, [n] * B, T)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    Q = torch.empty(T, qh, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    assert Q.numel() > 2 ** 31 and s.ws.numel() > 2 ** 34
    O = s.attend(Q)
    assert O[-n:].isfinite().all()
    for b in (0, 1, 511, B // 2, 963, 964, B - 2, B - 1):   # 963: the first whose rows pass 2^31 elements
        a = b * n
        _check_rows(cache, 0, lens[b], Q[a:a + n], O[a:a + n], _borders(n, lens[b], 1, b), {0, 8, qh - 1})
