"""Attention of ragged steps where the 16-bit operands could lose something:
weights far below the row's largest, and query elements far below theirs."""

import math

import pytest
import torch

import kv8_ref as ref
from kv8_ref import E4M3, INT8
from test_gpu_kv8_step import BF16_HALF, FORMATS, Step, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bm():
    import bit_moe_decode_w4a16_gb300 as m
    m.build()
    return m


# pieces of a stream's blocks: 8192 positions; up to 70 784; all of 2^19, as the blocks are too many to be cut
@pytest.mark.parametrize("fmt,d,n,base,piece", [(E4M3, 64, 1, 1 << 17, 1 << 13), (INT8, 128, 2600, 1 << 17, 70784), (E4M3, 64, 19500, 1 << 19, 543788),
                                                (INT8, 64, 19500, 1 << 19, 543788)])
@pytest.mark.parametrize("at", [0, 3000])
@pytest.mark.parametrize("depth", [20.0, 24.5, 25.1, 26.5, 30.0])
def test_light_weights_keep_their_share(bm, fmt, d, n, base, piece, at, depth):
    """One position far above all others, which weigh 2^-depth of it each and whose values have one sign: what is lost of them adds up.

    A weight is rounded to fp16, 2^-11 of itself or half a smallest step, 2^-25, against a reference that leaves the row's largest at 1 or
    more in pieces of up to 2^13 positions, at 2^4 up to 2^17, at 2^8 beyond: all of up to 2^21 positions lose at most 2^13 2^-25 =
    2^17 2^-29 = 2^21 2^-33 = 2^-12 of the largest weight, times the largest of their codes.  That does not grow with their number.
    Scores: (d + 8) 2^-24 of the largest, as in kv8_step_ref; 2^-18 for e^x and the normalising sum.

    The outputs' fp32 sums: beside a sum of 2^e the tensor cores keep of each product multiples of 2^(e - 25), and of 16 of them together
    multiples of 2^(e - 23), both cut off, not rounded (of products of 2^(e - 27) nothing is left).  16 2^-25 + 2^-23 for 16 positions,
    (2^-25 + 2^-27) of the output for each of the piece: much beside the large position's value, nothing beside none."""
    L = base + n
    c = {"format": fmt, "slots": 1, "ctx_cap": L, "kv_heads": 1, "head_dim": d}
    for m in ("K", "V"):
        c[m] = torch.zeros(1, 1, L, d, dtype=torch.uint8, device="cuda")
        c[m + "s"] = torch.ones(1, 1, L, device="cuda")
    one = 0x38 if fmt == E4M3 else 1
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    lo, hi = (0x30, 0x40) if fmt == E4M3 else (1, 4)
    c["V"][:] = torch.randint(lo, hi, c["V"].shape, generator=g, device="cuda", dtype=torch.uint8)
    c["V"][0, 0, at] = 0
    c["V"][0, 0, at, d // 2:] = one
    c["K"][0, 0, at, 0] = one
    Q = torch.zeros(n, 8, d, dtype=torch.bfloat16, device="cuda")
    Q[:, :, 0] = depth * math.log(2)
    s = Step(bm, c, 8, [0], [base], [n], n)
    O = s.attend(Q, scale=1.0)
    score = float(Q[0, 0, 0])
    w = math.exp(-score)
    v = ref.decode(c["V"][0, 0], fmt)
    large = v[at].clone()
    v[at] = 0
    total = 1 + w * torch.arange(base, base + n, dtype=torch.float64, device="cuda")[:, None]
    o = (large + w * v.cumsum(0)[base:]) / total
    off = score * (d + 8) * 2.0 ** -24
    bound = o * (2.0 ** -11 + 2.0 ** -18 + 2 * off + piece * (2.0 ** -25 + 2.0 ** -27)) + 2.0 ** -12 * v.max() / total
    err = (O.double() - o[:, None]).abs()
    tol = (BF16_HALF * o + bound * (1 + BF16_HALF))[:, None]
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("qh,kvh,d,n,base", [(8, 2, 64, 50, 150), (32, 4, 128, 300, 40)])
@pytest.mark.parametrize("exp", [10, 18, 24, 30, 90])
def test_query_elements_far_below_their_rows_largest(bm, fmt, qh, kvh, d, n, base, exp):
    """An element that all keys answer with zero says nothing about the others, however large it is."""
    cache = ref.random_cache(fmt, 1, base + n, kvh, d, 41)
    at = 5
    cache["K"][..., at] = 0
    Q = _rows(n, qh, d)
    Q[:, :, at] = 2.0 ** exp
    s = Step(bm, cache, qh, [0], [base], [n], n)
    s.check(Q, s.attend(Q))
