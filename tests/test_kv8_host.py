"""Refusals of the 8-bit cache calls and of the sampler, without a device: every
check is made on the host before any device work."""

import ctypes

import pytest

import bit_moe_decode_w4a16_gb300 as bm


@pytest.fixture(scope="module", autouse=True)
def built():
    bm.build()
    return bm.lib()


def _cache(**kw):
    v = {"format": 0, "slots": 4, "ctx_cap": 100, "kv_heads": 2, "head_dim": 64, "K": 1 << 20, "V": 1 << 20, "Ks": 1 << 20, "Vs": 1 << 20}
    v.update(kw)
    return bm.bm_kv8_cache(**v)


def _a(x):
    return ctypes.addressof(x)


P = 1 << 20   # an aligned address that no refused call may touch
BAD_CACHES = [{"format": 2}, {"format": -1}, {"slots": 0}, {"ctx_cap": 0}, {"kv_heads": 0}, {"head_dim": 96}, {"head_dim": 0},
              {"K": None}, {"Vs": None}, {"K": P + 8}, {"Ks": P + 2}]


def _append(c, ld=6 * 64, qh=2, qkv=P, rope=True, slots=P, index=P, Q=P, T=3, **r):
    rr = bm.bm_kv8_rope(**{"norm": 1, "eps": 1e-6, "inv_freq": P, **r})
    return bm.lib().kv8_append(_a(c), qkv, ld, qh, _a(rr) if rope else None, slots, index, None, Q, T, None)


def _attend(c, B=3, qh=4, scale=0.125, Q=P, slots=P, lens=P, O=P, ws=P, short=0):
    n = bm.kv8_workspace_bytes(B, qh, c.kv_heads, c.head_dim, c.ctx_cap)
    return bm.lib().kv8_attend(_a(c), Q, slots, lens, qh, scale, O, B, ws, max(n - short, 0), None)


def _prefix(c, p, slot=0, n=5, ws=1 << 30, null=False):
    return bm.lib().kv8_attend_prefix(_a(c), None if null else _a(p), slot, n, P, P, P, 4, 0.125, P, 3, P, ws, None)


@pytest.mark.parametrize("kw", BAD_CACHES, ids=lambda k: f"{list(k)[0]}={list(k.values())[0]}")
def test_bad_caches(kw):
    c = _cache(**kw)
    assert _append(c) == 1 and "kv8_append" in bm.last_error()
    assert bm.lib().kv8_read(_a(c), 0, 0, 1, P, P, None) == 1 and "kv8_read" in bm.last_error()
    assert _attend(c) == 1 and "kv8_attend" in bm.last_error()
    assert _prefix(_cache(), c) == 1 and "kv8_attend_prefix" in bm.last_error()


def test_append_refusals():
    c = _cache()
    for kw in ({"ld": 6 * 64 - 8}, {"ld": 6 * 64 + 4}, {"qh": 0}, {"qkv": None}, {"qkv": P + 8}, {"rope": False}, {"slots": None},
               {"index": None}, {"Q": None}, {"Q": P + 4}, {"T": 0}, {"T": -1}, {"eps": -1.0}, {"eps": float("nan")}, {"q_norm": P + 2}):
        assert _append(c, **kw) == 1, kw
        assert bm.last_error().startswith("kv8_append: ")


def test_read_refusals():
    c = _cache()
    read = lambda slot, first, n, K=P, V=P: bm.lib().kv8_read(_a(c), slot, first, n, K, V, None)  # noqa: E731
    assert read(4, 0, 1) == 1 and read(-1, 0, 1) == 1 and read(0, 0, 1, K=None) == 1 and read(0, 0, 1, V=P + 8) == 1
    assert read(0, -1, 1) == 2 and read(0, 100, 1) == 2 and read(0, 0, 101) == 2 and read(0, 0, -1) == 2
    assert read(0, 2 ** 31 - 1, 2 ** 31 - 1) == 2
    assert read(0, 100, 0) == 0 and bm.last_error() == ""


def test_attend_refusals():
    c = _cache()
    for kw in ({"B": 0}, {"B": 1025}, {"qh": 3}, {"qh": 0}, {"qh": 18}, {"scale": 0.0}, {"scale": -1.0}, {"scale": float("inf")},
               {"scale": float("nan")}, {"Q": None}, {"Q": P + 8}, {"O": P + 2}, {"ws": None}, {"ws": P + 4}, {"lens": None}, {"slots": None},
               {"short": 1}):
        assert _attend(c, **kw) == 1, kw
        assert bm.last_error().startswith("kv8_attend: ")


def test_prefix_refusals():
    c = _cache()
    assert _prefix(c, c, null=True) == 1
    for other in ({"format": 1}, {"kv_heads": 4}, {"head_dim": 128}):
        assert _prefix(c, _cache(**other)) == 1 and "format, kv_heads" in bm.last_error()
    assert _prefix(c, c, slot=4) == 1 and _prefix(c, c, slot=-1) == 1
    assert _prefix(c, c, n=101) == 2 and _prefix(c, c, n=-1) == 2
    assert _prefix(c, c, ws=8) == 1 and "workspace" in bm.last_error()


def test_workspace_sizes():
    assert bm.kv8_workspace_bytes(0, 8, 2, 64, 10) == 0 and bm.kv8_workspace_bytes(1, 9, 2, 64, 10) == 0
    assert bm.kv8_workspace_bytes(1, 8, 2, 64, 0) == 0 and bm.kv8_workspace_bytes(1, 8, 2, 64, 10, -1) == 0
    one = bm.kv8_workspace_bytes(1, 8, 2, 64, 256)
    assert one > 0 and bm.kv8_workspace_bytes(3, 8, 2, 64, 256) >= 3 * one > 0
    assert bm.kv8_workspace_bytes(1, 8, 2, 64, 256, 5000) > one
    # a prefix of the largest length, for many kv heads: chunks of 2^30 positions at most
    assert bm.kv8_workspace_bytes(1, 1000, 500, 64, 256, 2 ** 31 - 1) == 1000 * (1 + 2) * (64 + 2) * 4
    # a stream has a bounded number of chunks, however long
    assert bm.kv8_workspace_bytes(1, 8, 2, 64, 131072) == bm.kv8_workspace_bytes(1, 8, 2, 64, 2 ** 31 - 1)


def test_sample_refusals():
    f = lambda x=P, dtype=0, ld=100, V=100, B=2, u=P, ids=P: bm.lib().bm_sample(x, dtype, ld, V, B, None, None, None, None, u, ids, None, None)  # noqa: E731
    for kw in ({"x": None}, {"u": None}, {"ids": None}, {"dtype": 2}, {"V": 0}, {"V": 524289, "ld": 524289}, {"B": 0}, {"B": 65536},
               {"ld": 99}, {"x": P + 2}, {"x": P + 1, "dtype": 1}):
        assert f(**kw) == 1, kw
        assert bm.last_error().startswith("bm_sample: ")
