"""The 8-bit K/V cache against its definition in 64 bits: what kv8_append
writes, what kv8_read gives back, decode attention over it alone and behind a
shared prefix, and a serving loop of all of them with the sampler."""

import pytest
import torch

import kv8_ref as ref
from kv8_ref import E4M3, INT8

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0 ** -8    # a bf16 rounding, relative to the value
FORMATS = [pytest.param(E4M3, id="e4m3"), pytest.param(INT8, id="int8")]


@pytest.fixture(scope="module")
def bm():
    import bit_moe_decode_w4a16_gb300 as m
    m.build()
    return m


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _freqs(d, base=1e4):
    return (base ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)).float().cuda()


# ---------------------------------------------------------------- append

def _check_append(bm, fmt, T, qh, kvh, d, norm, rotate, weights=True, ld_pad=0, slots=None, index=None, pos=None, cap=40,
                  qkv=None, n_slots=None, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if slots is None:
        n_slots = T + 2
        slots = torch.randperm(n_slots, generator=g, device="cuda")[:T].int()
        index = torch.randint(0, cap, (T,), generator=g, device="cuda").int()
        pos = torch.randint(0, 200000, (T,), generator=g, device="cuda").int()
    elif n_slots is None:
        n_slots = max(int(slots.max()) + 2, 2)
    cache = ref.random_cache(fmt, n_slots, cap, kvh, d, seed + 1)
    before = {n: cache[n].clone() for n in ("K", "V", "Ks", "Vs")}
    row = (qh + 2 * kvh) * d
    if qkv is None:
        qkv = rnd(T, row + ld_pad).bfloat16()
    wq, wk = ((1 + 0.3 * rnd(d)).bfloat16(), (1 + 0.3 * rnd(d)).bfloat16()) if weights else (None, None)
    f = _freqs(d) if rotate else None
    Q = torch.full((T, qh, d), 7.0, dtype=torch.bfloat16, device="cuda")
    rope = bm.kv8_rope(norm=norm, q_norm=wq, k_norm=wk, eps=1e-6, inv_freq=f)
    bm.kv8_append(bm.kv8_cache(**cache), qkv, rope, slots, index, Q, rope_pos=pos)
    torch.cuda.synchronize()
    q, k, v, slack = ref.append_rows(qkv, qh, kvh, d, index if pos is None else pos, norm, wq, wk, 1e-6, f)
    live = (slots >= 0) & (slots < n_slots) & (index >= 0) & (index < cap)
    # fp32 on the way: the mean's tree sum, sqrt, quotient and products are within 16 roundings (2^-20 of each
    # factor); cosine and sine are within 2^-21 (the angle in turns is rounded to fp32); both together 2^-19
    loose = slack * 2.0 ** -19
    assert (Q[~live] == 7.0).all()
    err = (Q.double() - q).abs()[live]
    assert (err <= (BF16_HALF * q.abs() + loose[:, :qh] + 2.0 ** -133)[live]).all(), float(err.max())
    for n, y, lo in (("K", k, loose[:, qh:]), ("V", v, torch.zeros_like(v))):
        want = before[n].clone()
        at = (slots[live].long(), slice(None), index[live].long())
        got, s = cache[n][at], cache[n + "s"][at].double()[..., None]
        yl, ll = y[live], lo[live]
        M = ref.CODE_MAX[fmt]
        amax = yl.abs().amax(-1, keepdim=True)
        assert ((s * M - amax).abs() <= ll.amax(-1, keepdim=True) + amax * 2.0 ** -23).all()
        value = ref.decode(got, fmt) * s
        # half a step of the format (e4m3: 2^-4 of the value, or half the smallest subnormal, 2^-10 codes), and the
        # fp32 error of the value and of the scale the code was divided by
        step = 0.5 * s if fmt == INT8 else torch.maximum(2.0 ** -4 * yl.abs(), 2.0 ** -10 * s)
        err = (value - yl).abs()
        assert (err <= step * (1 + 2.0 ** -18) + 2 * ll + amax * 2.0 ** -22).all(), float(err.max())
        # every other byte of the cache is as it was
        want[at] = got
        assert torch.equal(want, cache[n])
        swant = before[n + "s"].clone()
        swant[at] = cache[n + "s"][at]
        assert torch.equal(swant, cache[n + "s"])
    return cache, Q


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,qh,kvh,d", [(1, 8, 2, 64), (5, 32, 4, 128), (33, 12, 4, 128), (7, 4, 4, 64), (3, 128, 16, 128),
                                        (2, 1, 1, 64), (300, 8, 8, 128), (5000, 6, 2, 64), (2500, 32, 4, 128)])
def test_append(bm, fmt, T, qh, kvh, d):
    _check_append(bm, fmt, T, qh, kvh, d, norm=True, rotate=True)


@pytest.mark.parametrize("norm,rotate,weights", [(False, True, False), (True, False, True), (False, False, False), (True, True, False)])
def test_append_without_parts(bm, norm, rotate, weights):
    _check_append(bm, E4M3, 6, 8, 2, 64, norm, rotate, weights)
    _check_append(bm, INT8, 6, 16, 2, 128, norm, rotate, weights)


def test_append_strided_rows_padding_and_default_positions(bm):
    slots, index = _i32(2, -1, 0, 9, 1, 2, 3), _i32(3, 1, -1, 5, 40, 4, 0)   # padding: rows 1, 2 (index), 4 (index = cap)
    _check_append(bm, E4M3, 7, 8, 2, 128, True, True, ld_pad=24, slots=slots, index=index)
    _check_append(bm, INT8, 2, 8, 2, 64, True, True, slots=_i32(-1, 2 ** 30), index=_i32(0, 0), n_slots=3)


def test_append_far_positions(bm):
    pos = _i32(0, 1, 131071, 1000003, 2 ** 24 + 1, 2 ** 29)
    _check_append(bm, E4M3, 6, 8, 2, 128, True, True, slots=_i32(0, 1, 2, 3, 4, 5), index=_i32(0, 1, 2, 3, 4, 39), pos=pos)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_special_heads(bm, fmt):
    qh, kvh, d = 2, 4, 64
    x = torch.randn(1, (qh + 2 * kvh) * d, device="cuda").bfloat16().view(1, qh + 2 * kvh, d)
    x[0, qh + 0] = 0                       # a zero head
    x[0, qh + 1] = 2.0 ** -120             # below the smallest stored magnitude
    x[0, qh + 2, 5] = float("nan")
    x[0, qh + 3, 63] = float("-inf")
    x[0, qh + kvh, 3] = 3e38               # near the type's largest
    cache = ref.random_cache(fmt, 1, 4, kvh, d, 3)
    Q = torch.empty(1, qh, d, dtype=torch.bfloat16, device="cuda")
    bm.kv8_append(bm.kv8_cache(**cache), x.view(1, -1), bm.kv8_rope(), _i32(0), _i32(2), Q)
    K = torch.empty(kvh, 1, d, dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    bm.kv8_read(bm.kv8_cache(**cache), 0, 2, 1, K, V)
    torch.cuda.synchronize()
    assert torch.equal(Q[0], x[0, :qh])
    assert (K[0] == 0).all() and (K[1] == 0).all() and K[2].isnan().all() and K[3].isnan().all()
    assert cache["Ks"][0, 0, 2] == 0 and cache["Ks"][0, 1, 2] == 0
    big = x[0, qh + kvh].double()
    assert V[0].isfinite().all() and abs(float(V[0, 0, 3]) / float(big[3]) - 1) <= BF16_HALF + 2.0 ** -22


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kvh,d,first,count", [(2, 64, 0, 1), (4, 128, 37, 1001), (1, 128, 5, 0), (3, 64, 1099, 1)])
def test_read(bm, fmt, kvh, d, first, count):
    cache = ref.random_cache(fmt, 2, 1100, kvh, d, 11)
    K = torch.full((kvh, count, d), 9.0, dtype=torch.bfloat16, device="cuda")
    V = torch.full_like(K, 9.0)
    bm.kv8_read(bm.kv8_cache(**cache), 1, first, count, K, V)
    for n, out in (("K", K), ("V", V)):
        at = slice(first, first + count)
        want = ref.decode(cache[n][1, :, at], fmt) * cache[n + "s"][1, :, at].double().unsqueeze(-1)
        # the product is rounded to fp32 and then to bf16
        assert ((out.double() - want).abs() <= want.abs() * (BF16_HALF + 2.0 ** -23)).all()


def test_read_every_code(bm):
    for fmt in (E4M3, INT8):
        codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 1, 4, 64)
        if fmt == E4M3:
            codes = torch.where((codes & 127) == 127, torch.zeros_like(codes), codes)   # its two NaN codes are never written
        one = torch.ones(1, 1, 4, device="cuda")
        K = torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda")
        V = torch.empty_like(K)
        bm.kv8_read(bm.kv8_cache(fmt, 1, 4, 1, 64, codes, codes.clone(), one, one), 0, 0, 4, K, V)
        assert torch.equal(K.double(), ref.decode(codes[0], fmt)) and torch.equal(K, V)


# ---------------------------------------------------------------- attend

def _attend(bm, cache, Q, slots, lens, scale=None, prefix=None, p_slot=0, p_len=0, fill=5.0, ws=None, stream=None):
    B, qh, d = Q.shape
    O = torch.full((B, qh, d), fill, dtype=torch.bfloat16, device="cuda")
    n = bm.kv8_workspace_bytes(B, qh, cache["kv_heads"], d, cache["ctx_cap"], p_len)
    if ws is None:
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")     # NaN wherever it is read unwritten
    if prefix is None:
        bm.kv8_attend(bm.kv8_cache(**cache), Q, slots, lens, O, ws, scale=scale, stream=stream)
    else:
        bm.kv8_attend_prefix(bm.kv8_cache(**cache), bm.kv8_cache(**prefix), p_slot, p_len, Q, slots, lens, O, ws, scale=scale, stream=stream)
    return O


def _check_rows(O, want, bound, fill=5.0):
    for b in range(O.shape[0]):
        if want[b] is None:
            assert (O[b] == fill).all(), b
            continue
        err = (O[b].double() - want[b]).abs()
        tol = BF16_HALF * want[b].abs() + bound[b] * (1 + BF16_HALF)
        assert O[b].isfinite().all() and (err <= tol).all(), (b, float((err - tol).max()))


def _spoil(cache, slot, n):
    """What is behind a stream's last position must not matter."""
    for m in ("K", "V"):
        cache[m][slot, :, n:] = 0xFF
        cache[m + "s"][slot, :, n:] = float("nan")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("qh,kvh,d", [(32, 4, 128), (8, 2, 64), (12, 4, 128), (4, 4, 64), (16, 2, 64), (7, 1, 128), (2, 1, 64)])
def test_attend_ragged(bm, fmt, qh, kvh, d):
    lens = [0, 1, 2, 7, 8, 15, 16, 17, 31, 33, 64, 127, 128, 129, 255, 256, 257, 511, 513, 777]
    cap = 777
    slots = torch.randperm(len(lens)).int()
    cache = ref.random_cache(fmt, len(lens), cap, kvh, d, 21)
    for s, n in zip(slots.tolist(), lens):
        _spoil(cache, s, n)
    rows = [(int(s), n) for s, n in zip(slots, lens)] + [(-1, 5), (len(lens), 5), (3, -1), (3, cap + 1), (int(slots[-1]), 300)]
    slots, lens = _i32(*[r[0] for r in rows]), _i32(*[r[1] for r in rows])
    Q = torch.randn(len(rows), qh, d, device="cuda").bfloat16()
    O = _attend(bm, cache, Q, slots, lens)
    _check_rows(O, *ref.attend(cache, Q, slots, lens, d ** -0.5))


@pytest.mark.parametrize("fmt,n", [(E4M3, 16384), (INT8, 16385), (E4M3, 40001)])
def test_attend_long_streams(bm, fmt, n):
    cache = ref.random_cache(fmt, 2, 40001, 2, 128, 5)
    Q = torch.randn(2, 16, 128, device="cuda").bfloat16()
    slots, lens = _i32(1, 0), _i32(n, 1000)
    _check_rows(_attend(bm, cache, Q, slots, lens), *ref.attend(cache, Q, slots, lens, 128 ** -0.5))


@pytest.mark.parametrize("fmt", FORMATS)
def test_attend_peaked_and_uneven_values(bm, fmt):
    """Scores far apart, V scales over 12 binary orders, heads of zeros."""
    cache = ref.random_cache(fmt, 3, 600, 2, 128, 8, spread=0.0)
    cache["Vs"] *= torch.exp2(torch.randint(-6, 7, cache["Vs"].shape, device="cuda").float())
    cache["Ks"] *= torch.exp2(torch.randint(-4, 5, cache["Ks"].shape, device="cuda").float())
    cache["K"][0, 0, 10:50] = 0
    cache["Ks"][0, 0, 10:50] = 0
    cache["V"][1] = 0
    cache["Vs"][1] = 0
    Q = 4 * torch.randn(3, 16, 128, device="cuda").bfloat16()
    slots, lens = _i32(0, 1, 2), _i32(600, 600, 599)
    O = _attend(bm, cache, Q, slots, lens)
    _check_rows(O, *ref.attend(cache, Q, slots, lens, 128 ** -0.5))
    assert (O[1] == 0).all()


@pytest.mark.parametrize("exp", [-100, -40, 40])
def test_attend_extreme_scales(bm, exp):
    """Values far from 1: the output has V's magnitude, whatever it is."""
    cache = ref.random_cache(E4M3, 1, 300, 1, 64, 9)
    cache["Vs"] *= 2.0 ** exp
    cache["Ks"] *= 2.0 ** 20
    Q = (torch.randn(1, 8, 64, device="cuda") * 2.0 ** -20).bfloat16()
    slots, lens = _i32(0), _i32(300)
    _check_rows(_attend(bm, cache, Q, slots, lens), *ref.attend(cache, Q, slots, lens, 0.125))


def test_attend_nan_stays_in_its_row(bm):
    cache = ref.random_cache(E4M3, 3, 300, 2, 128, 10)
    cache["Ks"][1, 0, 100] = float("nan")
    Q = torch.randn(3, 16, 128, device="cuda").bfloat16()
    slots, lens = _i32(0, 1, 2), _i32(300, 300, 300)
    O = _attend(bm, cache, Q, slots, lens)
    assert O[1, :8].isnan().all() and O[1, 8:].isfinite().all() and O[0].isfinite().all() and O[2].isfinite().all()


def test_attend_rows_do_not_depend_on_the_batch(bm):
    cache = ref.random_cache(E4M3, 40, 3000, 4, 128, 12)
    lens = torch.randint(1, 3001, (40,)).int().cuda()
    slots = torch.randperm(40).int().cuda()
    Q = torch.randn(40, 32, 128, device="cuda").bfloat16()
    whole = _attend(bm, cache, Q, slots, lens)
    for b in (0, 7, 39):
        solo = _attend(bm, cache, Q[b:b + 1].clone(), slots[b:b + 1].clone(), lens[b:b + 1].clone())
        assert torch.equal(solo[0].view(torch.int16), whole[b].view(torch.int16))
    assert torch.equal(whole.view(torch.int16), _attend(bm, cache, Q, slots, lens).view(torch.int16))


def test_offsets_past_32_bits(bm):
    """A cache whose codes pass 2^31 bytes: written, read and attended behind that point."""
    kvh, d, cap, slots = 2, 128, 3_000_000, 3
    c = {"format": E4M3, "slots": slots, "ctx_cap": cap, "kv_heads": kvh, "head_dim": d}
    for n in ("K", "V"):
        c[n] = torch.zeros(slots, kvh, cap, d, dtype=torch.uint8, device="cuda")
        c[n + "s"] = torch.zeros(slots, kvh, cap, device="cuda")
    T = 20
    qkv = torch.randn(T, (4 + 2 * kvh) * d, device="cuda").bfloat16()
    Q = torch.empty(T, 4, d, dtype=torch.bfloat16, device="cuda")
    h = bm.kv8_cache(**c)
    idx = torch.arange(cap - T, cap, dtype=torch.int32, device="cuda")
    bm.kv8_append(h, qkv, bm.kv8_rope(), torch.full((T,), 2, dtype=torch.int32, device="cuda"), idx, Q)
    K = torch.empty(kvh, T, d, dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    bm.kv8_read(h, 2, cap - T, T, K, V)
    v = qkv[:, 6 * d:].double().view(T, kvh, d).transpose(0, 1)
    assert ((V.double() - v).abs() <= 2.0 ** -4 * v.abs() + v.abs().amax(-1, keepdim=True) * 2.0 ** -18 + BF16_HALF * v.abs()).all()
    # zero keys everywhere else: the T written positions and the cap - T zero ones share the weight
    O = _attend(bm, c, torch.zeros(1, 4, d, device="cuda").bfloat16(), _i32(2), _i32(cap))
    want = (ref.decode(c["V"][2, :, cap - T:], E4M3) * c["Vs"][2, :, cap - T:].double().unsqueeze(-1)).sum(1) / cap
    want = want.repeat_interleave(2, 0)
    size = v.abs().sum(1).repeat_interleave(2, 0) / cap
    assert ((O[0].double() - want).abs() <= BF16_HALF * want.abs() + size * 2.0 ** -10).all()


@pytest.mark.parametrize("P", [0, 130])
def test_largest_batch(bm, P):
    """1024 rows, some of them of one slot, with and without a prefix."""
    B, qh, kvh, d = 1024, 8, 1, 64
    cache = ref.random_cache(E4M3, 50, 40, kvh, d, 14)
    slots, lens = torch.randint(-1, 50, (B,)).int().cuda(), torch.randint(0, 41, (B,)).int().cuda()
    Q = torch.randn(B, qh, d, device="cuda").bfloat16()
    prefix = ref.random_cache(E4M3, 1, 130, kvh, d, 15) if P else None
    O = _attend(bm, cache, Q, slots, lens, prefix=prefix, p_len=P)
    _check_rows(O, *ref.attend(cache, Q, slots, lens, d ** -0.5, prefix=(prefix, 0, P) if P else None))


def test_nothing_to_attend_over(bm):
    """All rows empty or padding: zeros, or what was there."""
    cache = ref.random_cache(INT8, 3, 20, 2, 64, 16)
    Q = torch.randn(4, 4, 64, device="cuda").bfloat16()
    O = _attend(bm, cache, Q, _i32(0, -1, 2, 7), _i32(0, 5, 0, 5))
    assert (O[0] == 0).all() and (O[1] == 5).all() and (O[2] == 0).all() and (O[3] == 5).all()


# ---------------------------------------------------------------- shared prefix

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,P,qh,kvh,d", [(1, 1, 8, 2, 64), (3, 1000, 8, 2, 64), (5, 129, 32, 4, 128), (17, 2049, 32, 4, 128),
                                          (40, 300, 12, 4, 128), (33, 128, 4, 4, 64), (9, 5000, 16, 2, 128), (2, 640, 7, 1, 64),
                                          (130, 5000, 32, 4, 128), (97, 20000, 8, 1, 64), (100, 40, 8, 1, 128)])
def test_prefix(bm, fmt, B, P, qh, kvh, d):
    prefix = ref.random_cache(fmt, 2, P + 3, kvh, d, 31)
    _spoil(prefix, 1, P)
    cache = ref.random_cache(fmt, B, 70, kvh, d, 32)
    lens = torch.randint(0, 71, (B,)).int()
    slots = torch.randperm(B).int()
    lens[0] = 0
    if B > 4:
        slots[3] = -1
        lens[4] = 71
    for s, n in zip(slots.tolist(), lens.tolist()):
        if s >= 0 and n <= 70:
            _spoil(cache, s, n)
    slots, lens = slots.cuda(), lens.cuda()
    Q = torch.randn(B, qh, d, device="cuda").bfloat16()
    O = _attend(bm, cache, Q, slots, lens, prefix=prefix, p_slot=1, p_len=P)
    _check_rows(O, *ref.attend(cache, Q, slots, lens, d ** -0.5, prefix=(prefix, 1, P)))


def test_prefix_of_the_same_cache_and_of_length_zero(bm):
    cache = ref.random_cache(INT8, 6, 400, 2, 128, 33)
    Q = torch.randn(4, 16, 128, device="cuda").bfloat16()
    slots, lens = _i32(1, 2, 3, 1), _i32(10, 0, 400, 3)
    O = _attend(bm, cache, Q, slots, lens, prefix=cache, p_slot=5, p_len=333)
    _check_rows(O, *ref.attend(cache, Q, slots, lens, 128 ** -0.5, prefix=(cache, 5, 333)))
    none = _attend(bm, cache, Q, slots, lens, prefix=cache, p_slot=5, p_len=0)
    assert torch.equal(none.view(torch.int16), _attend(bm, cache, Q, slots, lens).view(torch.int16))
    assert (none[1] == 0).all()


def test_prefix_rows_do_not_depend_on_the_batch(bm):
    prefix = ref.random_cache(E4M3, 1, 3000, 4, 128, 41)
    cache = ref.random_cache(E4M3, 37, 300, 4, 128, 42)
    lens = torch.randint(0, 301, (37,)).int().cuda()
    slots = torch.randperm(37).int().cuda()
    Q = torch.randn(37, 32, 128, device="cuda").bfloat16()
    whole = _attend(bm, cache, Q, slots, lens, prefix=prefix, p_len=2777)
    for b in (0, 16, 36):
        solo = _attend(bm, cache, Q[b:b + 1].clone(), slots[b:b + 1].clone(), lens[b:b + 1].clone(), prefix=prefix, p_len=2777)
        assert torch.equal(solo[0].view(torch.int16), whole[b].view(torch.int16))


@pytest.mark.parametrize("fmt, B, P, qh, kvh, d", [(E4M3, 40, 20001, 16, 2, 128), (INT8, 300, 9999, 8, 1, 64), (E4M3, 130, 5000, 32, 4, 128)])
def test_prefix_of_several_chunks_to_a_cta(bm, fmt, B, P, qh, kvh, d):
    """More tiles of query rows than fit at once: a CTA takes several chunks of one and of three tiles, the last one short;
    scores grow along the prefix, so references move in every chunk."""
    prefix = ref.random_cache(fmt, 1, P, kvh, d, 45)
    prefix["Ks"] *= torch.linspace(0.2, 3, P, device="cuda")
    cache = ref.random_cache(fmt, B, 20, kvh, d, 46)
    slots, lens = torch.arange(B, dtype=torch.int32, device="cuda"), torch.arange(B, dtype=torch.int32, device="cuda") % 21
    Q = torch.randn(B, qh, d, device="cuda").bfloat16()
    O = _attend(bm, cache, Q, slots, lens, prefix=prefix, p_len=P)
    _check_rows(O, *ref.attend(cache, Q, slots, lens, d ** -0.5, prefix=(prefix, 0, P)))
    for b in (0, B // 2, B - 1):
        solo = _attend(bm, cache, Q[b:b + 1].clone(), slots[b:b + 1].clone(), lens[b:b + 1].clone(), prefix=prefix, p_len=P)
        assert torch.equal(solo[0].view(torch.int16), O[b].view(torch.int16))


def test_prefix_uneven_values(bm):
    """V scales over 12 binary orders and large scores in the shared part."""
    for fmt in (E4M3, INT8):
        prefix = ref.random_cache(fmt, 1, 1500, 2, 128, 43, spread=0.0)
        prefix["Vs"] *= torch.exp2(torch.randint(-6, 7, prefix["Vs"].shape, device="cuda").float())
        prefix["Ks"] *= torch.exp2(torch.randint(-3, 3, prefix["Ks"].shape, device="cuda").float())
        cache = ref.random_cache(fmt, 18, 20, 2, 128, 44)
        Q = 3 * torch.randn(18, 16, 128, device="cuda").bfloat16()
        slots, lens = torch.arange(18, dtype=torch.int32, device="cuda"), torch.arange(18, dtype=torch.int32, device="cuda")
        O = _attend(bm, cache, Q, slots, lens, prefix=prefix, p_len=1500)
        _check_rows(O, *ref.attend(cache, Q, slots, lens, 128 ** -0.5, prefix=(prefix, 0, 1500)))


# ---------------------------------------------------------------- streams, graphs, the loop

def test_streams_and_graph_replay(bm):
    """A captured append + attend follows the device's slots and lengths; two streams with workspaces of their own overlap."""
    kvh, d, qh, B, cap = 2, 128, 16, 4, 600
    prefix = ref.random_cache(E4M3, 1, 700, kvh, d, 51)
    cache = ref.random_cache(E4M3, B, cap, kvh, d, 52)
    h, hp = bm.kv8_cache(**cache), bm.kv8_cache(**prefix)
    slots, index, lens = _i32(0, 1, 2, 3), _i32(10, 20, 30, 299), _i32(11, 21, 31, 300)
    qkv = torch.randn(B, (qh + 2 * kvh) * d, device="cuda").bfloat16()
    Q, O = (torch.empty(B, qh, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(bm.kv8_workspace_bytes(B, qh, kvh, d, cap, 700), dtype=torch.uint8, device="cuda")
    rope = bm.kv8_rope(norm=True, inv_freq=_freqs(d))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        bm.kv8_append(h, qkv, rope, slots, index, Q, stream=side)
        bm.kv8_attend_prefix(h, hp, 0, 700, Q, slots, lens, O, ws, stream=side)
    for step in range(3):
        if step:
            index += 1
            lens += 1
            qkv.copy_(torch.randn_like(qkv))
        if step == 2:
            slots[1] = -1
            O.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        _check_rows(O, *ref.attend(cache, Q, slots, lens, d ** -0.5, prefix=(prefix, 0, 700)))
    slots[1] = 1
    a = _attend(bm, cache, Q, slots, lens, stream=side)
    b = _attend(bm, cache, Q, slots, lens)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_two_streams_at_once(bm):
    """Calls that overlap on the GPU, each with a workspace of its own, give what they give alone."""
    kvh, d, qh, B, P = 2, 128, 16, 20, 3000
    prefix = ref.random_cache(E4M3, 1, P, kvh, d, 61)
    cache = ref.random_cache(E4M3, B, 2000, kvh, d, 62)
    h, hp = bm.kv8_cache(**cache), bm.kv8_cache(**prefix)
    slots, lens = torch.arange(B, dtype=torch.int32, device="cuda"), torch.randint(1, 2001, (B,)).int().cuda()
    Q = [torch.randn(B, qh, d, device="cuda").bfloat16() for _ in range(2)]
    want = [_attend(bm, cache, q, slots, lens, prefix=prefix, p_len=P) for q in Q]
    O = [torch.zeros_like(q) for q in Q]
    ws = [torch.empty(bm.kv8_workspace_bytes(B, qh, kvh, d, 2000, P), dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            bm.kv8_attend_prefix(h, hp, 0, P, Q[i], slots, lens, O[i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(O[i].view(torch.int16), want[i].view(torch.int16))


def test_serving_loop(bm):
    """Prompt of a shared prefix, then steps of append, attention behind the prefix and sampling: every step's
    cache, attention and token against 64 bits, from the device's own state."""
    qh, kvh, d, B, P, V = 16, 2, 64, 3, 200, 1000
    dev = dict(device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(77)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    empty = lambda slots, cap: {"format": E4M3, "slots": slots, "ctx_cap": cap, "kv_heads": kvh, "head_dim": d,  # noqa: E731
                                "K": torch.zeros(slots, kvh, cap, d, dtype=torch.uint8, **dev),
                                "V": torch.zeros(slots, kvh, cap, d, dtype=torch.uint8, **dev),
                                "Ks": torch.zeros(slots, kvh, cap, **dev), "Vs": torch.zeros(slots, kvh, cap, **dev)}
    pre, own = empty(1, P), empty(B, 16)
    hp, ho = bm.kv8_cache(**pre), bm.kv8_cache(**own)
    embed, head = rnd(V, (qh + 2 * kvh) * d).bfloat16(), rnd(V, qh * d).bfloat16()
    rope = bm.kv8_rope(norm=True, q_norm=(1 + 0.1 * rnd(d)).bfloat16(), inv_freq=_freqs(d))
    prompt = torch.randint(0, V, (P,), generator=g, device="cuda")
    Qp = torch.empty(P, qh, d, dtype=torch.bfloat16, **dev)
    zeros = torch.zeros(P, dtype=torch.int32, **dev)
    bm.kv8_append(hp, embed[prompt], rope, zeros, torch.arange(P, dtype=torch.int32, **dev), Qp)
    slots, lens = _i32(2, 0, 1), _i32(0, 0, 0)
    tokens = prompt[-1:].expand(B).int().contiguous()
    Q, O = (torch.empty(B, qh, d, dtype=torch.bfloat16, **dev) for _ in range(2))
    ws = torch.empty(bm.kv8_workspace_bytes(B, qh, kvh, d, 16, P), dtype=torch.uint8, **dev)
    temp, topk, topp, minp = (torch.tensor(v, **dev) for v in ([0.8, 0.0, 1.2], [50, 0, 0], [0.9, 1.0, 0.95], [0.0, 0.0, 0.02]))
    topk = topk.int()
    for step in range(8):
        u = torch.rand(B, generator=g, device="cuda")
        bm.kv8_append(ho, embed[tokens.long()], rope, slots, lens, Q, rope_pos=lens + P)
        lens += 1
        bm.kv8_attend_prefix(ho, hp, 0, P, Q, slots, lens, O, ws)
        logits = (O.view(B, -1).float() @ head.float().t()).contiguous()
        bm.bm_sample(logits, temp, topk, topp, minp, u, tokens)
        torch.cuda.synchronize()
        _check_rows(O, *ref.attend(own, Q, slots, lens, d ** -0.5, prefix=(pre, 0, P)))
        ids, _, margin = ref.sample(logits, temp.cpu(), topk.cpu(), topp.cpu(), minp.cpu(), u.cpu())
        for b in range(B):
            assert margin[b] < 1e-6 or int(tokens[b]) == ids[b]
    assert int(lens[0]) == 8


# ---------------------------------------------------------------- refusals that need tensors

def test_refusals(bm):
    cache = ref.random_cache(E4M3, 2, 64, 2, 64, 1)
    h = bm.kv8_cache(**cache)
    Q = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    O, slots, lens = torch.empty_like(Q), _i32(0, 1), _i32(3, 4)
    ws = torch.empty(bm.kv8_workspace_bytes(2, 8, 2, 64, 64), dtype=torch.uint8, device="cuda")
    bm.kv8_attend(h, Q, slots, lens, O, ws)
    bad = [lambda: bm.kv8_attend(h, Q.half(), slots, lens, O, ws), lambda: bm.kv8_attend(h, Q, slots.long(), lens, O, ws),
           lambda: bm.kv8_attend(h, Q, slots, lens.cpu(), O, ws), lambda: bm.kv8_attend(h, Q, slots, lens, O, ws[:-1]),
           lambda: bm.kv8_attend(h, Q, slots[:1], lens, O, ws), lambda: bm.kv8_attend(h, Q, slots, lens, O, ws, scale=0.0),
           lambda: bm.kv8_attend(h, Q, slots, lens, O, ws, scale=float("nan")),
           lambda: bm.kv8_attend(h, Q.transpose(0, 1), slots, lens, O, ws),
           lambda: bm.kv8_attend(h, torch.zeros(2, 18, 64, dtype=torch.bfloat16, device="cuda"), slots, lens, torch.zeros(2, 18, 64, dtype=torch.bfloat16, device="cuda"), ws),
           lambda: bm.kv8_attend_prefix(h, h, 2, 3, Q, slots, lens, O, ws), lambda: bm.kv8_attend_prefix(h, h, 0, 65, Q, slots, lens, O, ws),
           lambda: bm.kv8_read(h, 0, 60, 5, torch.empty(2, 5, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 5, 64, dtype=torch.bfloat16, device="cuda")),
           lambda: bm.kv8_cache(**{**cache, "K": cache["K"][:1]}),
           lambda: bm.kv8_append(h, torch.zeros(2, 100, dtype=torch.bfloat16, device="cuda"), bm.kv8_rope(), slots, lens, Q),
           lambda: bm.kv8_append(h, torch.zeros(2, 772, dtype=torch.bfloat16, device="cuda"), bm.kv8_rope(), slots, lens, Q)]
    for i, call in enumerate(bad):
        with pytest.raises(bm.BitMoeError):
            call()
            pytest.fail(f"call {i} was accepted")
