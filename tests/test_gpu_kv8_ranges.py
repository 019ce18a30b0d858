"""Attention over the 8-bit cache where magnitudes lie far apart: against 64 bits,
or bit for bit against the same problem in other units."""

import pytest
import torch

import kv8_ref as ref
from test_gpu_kv8 import BF16_HALF, E4M3, FORMATS, INT8, _attend, _check_rows, _i32, bm  # noqa: F401

pytestmark = pytest.mark.gpu


def _v_zero_but(cache, slot, live, exp):
    """V of a slot: heads of zeros, but at the positions `live`, whose scale becomes 2^exp."""
    dead = torch.ones(cache["ctx_cap"], dtype=torch.bool)
    dead[live] = False
    dead = dead.to(cache["V"].device)
    cache["V"][slot, :, dead] = 0
    cache["Vs"][slot, :, dead] = 0
    cache["Vs"][slot, :, ~dead] = 2.0 ** exp


# positions of a stage of 128 are dealt out 32 to a warp: the live ones come later in the same warp's walk, in another
# warp, in another chunk (256), before the zeros, and in their midst
@pytest.mark.parametrize("exp", [-90, 0, 20, 27, 60, 95])
@pytest.mark.parametrize("fmt,d", [(E4M3, 128), (INT8, 64)])
@pytest.mark.parametrize("n,live", [(129, [128]), (128, [127]), (301, [300]), (600, [0]), (513, [40, 512]), (2, [1])])
def test_heads_of_zeros_keep_their_share(bm, fmt, d, n, live, exp):
    """Positions whose V is zero weigh in the denominator, whatever the magnitude of the others."""
    cache = ref.random_cache(fmt, 1, n, 2, d, 71)
    _v_zero_but(cache, 0, live, exp)
    Q = torch.cat([torch.zeros(1, 8, d, device="cuda"), torch.randn(1, 8, d, device="cuda")]).bfloat16()
    slots, lens = _i32(0, 0), _i32(n, n)
    _check_rows(_attend(bm, cache, Q, slots, lens), *ref.attend(cache, Q, slots, lens, d ** -0.5))


# 32 kv heads: 4 chunks of 256 positions, two tiles each; 2 kv heads: one tile to a chunk
@pytest.mark.parametrize("exp", [0, 27, 95])
@pytest.mark.parametrize("fmt,kvh,d", [(E4M3, 32, 64), (INT8, 2, 128), (E4M3, 32, 128)])
@pytest.mark.parametrize("live", [[130], [1023], [0], None])
def test_prefix_heads_of_zeros_keep_their_share(bm, fmt, kvh, d, live, exp):
    P, qh = 1024, 2 * kvh
    prefix, cache = ref.random_cache(fmt, 1, P, kvh, d, 72), ref.random_cache(fmt, 3, 9, kvh, d, 73)
    if live is None:                       # what is not zero lies behind the prefix
        _v_zero_but(prefix, 0, [], 0)
        cache["Vs"][:] = 2.0 ** exp
    else:
        _v_zero_but(prefix, 0, live, exp)
    Q = torch.cat([torch.zeros(1, qh, d, device="cuda"), torch.randn(2, qh, d, device="cuda")]).bfloat16()
    slots, lens = _i32(0, 1, 2), _i32(9, 0 if live else 9, 5)
    O = _attend(bm, cache, Q, slots, lens, prefix=prefix, p_len=P)
    _check_rows(O, *ref.attend(cache, Q, slots, lens, d ** -0.5, prefix=(prefix, 0, P)))


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("P", [0, 200])
@pytest.mark.parametrize("n", [1, 5, 300])
def test_scores_of_the_largest_size(bm, n, P, sign):
    """Equal scores of +-1.6e7: some average of the values, whatever the steps of fp32 make of the weights."""
    d = 64
    cache, prefix = ref.random_cache(E4M3, 1, n, 1, d, 74), ref.random_cache(E4M3, 1, 200, 1, d, 75)
    for c in (cache, prefix):
        c["K"][:] = 0x7E if sign > 0 else 0xFE     # +-448
        c["Ks"][:] = 2.0 ** -8
    Q = torch.full((1, 4, d), 1.6e7 / (448 * 2.0 ** -8 * d * d ** -0.5), device="cuda").bfloat16()
    O = _attend(bm, cache, Q, _i32(0), _i32(n), prefix=prefix if P else None, p_len=P)
    v = torch.cat([ref.decode(c["V"][0, 0, :m], E4M3) * c["Vs"][0, 0, :m, None].double() for c, m in ((cache, n), (prefix, P))])
    slack = v.abs().amax(0) * 2.0 ** -7
    assert O.isfinite().all() and (O[0].double() <= v.amax(0) + slack).all() and (O[0].double() >= v.amin(0) - slack).all()
    if not P:                              # all scores come from the same instructions: equal weights
        want, size = v.mean(0), v.abs().mean(0)
        assert ((O[0].double() - want).abs() <= BF16_HALF * want.abs() + size * (2.0 ** -11 + 2.0 ** -18) * (1 + BF16_HALF)).all()


def _in_units(exp, P, seed=76):
    """(cache, prefix, Q) of one problem with query rows times 2^exp and keys divided by it."""
    d = 64
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cache, prefix = ref.random_cache(E4M3, 2, 300, 2, d, seed), ref.random_cache(E4M3, 1, P or 1, 2, d, seed + 1)
    for c in (cache, prefix):
        c["Ks"][:] = 2.0 ** (-7 - exp)
    Q = torch.randn(2, 8, d, generator=g, device="cuda").bfloat16() * 2.0 ** exp
    return cache, (prefix if P else None), Q.bfloat16()


@pytest.mark.parametrize("P", [0, 200])
@pytest.mark.parametrize("exp", [-110, -101, -60, 60, 100, 110, 124])
def test_query_rows_of_any_magnitude(bm, exp, P):
    """Query rows times 2^exp with keys of 2^-exp: the same bits."""
    slots, lens = _i32(0, 1), _i32(300, 77)
    out = []
    for e in (0, exp):
        cache, prefix, Q = _in_units(e, P)
        assert Q.isfinite().all()
        out.append(_attend(bm, cache, Q, slots, lens, prefix=prefix, p_len=P))
    assert out[1].isfinite().all() and torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))


@pytest.mark.parametrize("P", [0, 200])
def test_query_rows_at_the_ends_of_the_type(bm, P):
    """Rows of the type's largest and smallest numbers, keys to match, against 64 bits."""
    d = 64
    slots, lens = _i32(0, 1), _i32(300, 77)
    for value, ks in ((torch.finfo(torch.bfloat16).max, 2.0 ** -138), (2.0 ** -126, 2.0 ** 114), (2.0 ** -131, 2.0 ** 118)):
        cache, prefix, Q = _in_units(0, P)
        sign = torch.where(Q > 0, 1.0, -1.0)
        Q = (sign * value).bfloat16()
        for c in (cache, prefix):
            if c is not None:
                c["Ks"][:] = ks
        assert Q.isfinite().all() and (Q != 0).all()
        O = _attend(bm, cache, Q, slots, lens, prefix=prefix, p_len=P)
        _check_rows(O, *ref.attend(cache, Q, slots, lens, d ** -0.5, prefix=(prefix, 0, P) if P else None))


@pytest.mark.parametrize("kvh,d", [(4, 128), (8, 64)])
def test_one_workspace_for_every_prefix(bm, kvh, d):
    """A buffer made for the longest prefix, context and batch serves the shorter ones, which may have more chunks."""
    qh, longest = 2 * kvh, 8192
    prefix, cache = ref.random_cache(E4M3, 1, longest, kvh, d, 78), ref.random_cache(E4M3, 4, 60, kvh, d, 79)
    ws = torch.full((bm.kv8_workspace_bytes(4, qh, kvh, d, 60, longest),), 255, dtype=torch.uint8, device="cuda")
    Q = torch.randn(4, qh, d, device="cuda").bfloat16()
    slots, lens = _i32(0, 1, 2, 3), _i32(60, 0, 31, 1)
    for P in (longest, 2432, 4864, 4865, 2433, 4225, 1, 0):
        for B in (4, 1):
            q, s, n = Q[:B].clone(), slots[:B].clone(), lens[:B].clone()
            O = _attend(bm, cache, q, s, n, prefix=prefix, p_len=P, ws=ws)
            _check_rows(O, *ref.attend(cache, q, s, n, d ** -0.5, prefix=(prefix, 0, P)))


@pytest.mark.parametrize("B", [447, 448, 1024])
def test_large_batches_of_wide_heads(bm, B):
    """Around the batch from which an SM holds two CTAs instead of three: every row, and the bits of rows alone."""
    qh, kvh, d, cap = 6, 2, 128, 600
    cache = ref.random_cache(INT8, 40, cap, kvh, d, 80)
    slots, lens = torch.randint(-1, 41, (B,)).int().cuda(), torch.randint(0, cap + 2, (B,)).int().cuda()
    Q = torch.randn(B, qh, d, device="cuda").bfloat16()
    O = _attend(bm, cache, Q, slots, lens)
    _check_rows(O, *ref.attend(cache, Q, slots, lens, d ** -0.5))
    for b in (0, B // 2, B - 1):
        solo = _attend(bm, cache, Q[b:b + 1].clone(), slots[b:b + 1].clone(), lens[b:b + 1].clone())
        assert torch.equal(solo[0].view(torch.int16), O[b].view(torch.int16))
