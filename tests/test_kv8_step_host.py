"""Refusals and sizes of the ragged-step calls, without a device: every check
is made on the host before any device work."""

import ctypes

import pytest

import bit_moe_decode_w4a16_gb300 as bm

P = 1 << 20   # an aligned address that no refused call may touch


@pytest.fixture(scope="module", autouse=True)
def built():
    bm.build()
    return bm.lib()


def _cache(**kw):
    v = {"format": 0, "slots": 4, "ctx_cap": 100, "kv_heads": 2, "head_dim": 64, "K": P, "V": P, "Ks": P, "Vs": P}
    v.update(kw)
    return bm.bm_kv8_cache(**v)


BAD_CACHES = [{"format": 2}, {"slots": 0}, {"ctx_cap": 0}, {"kv_heads": 0}, {"head_dim": 96}, {"K": None}, {"Vs": None}, {"K": P + 8}, {"Ks": P + 2}]


def _plan(c=None, qh=4, v=(P,) * 9, B=3, T=10, plan=P, short=0):
    c = _cache() if c is None else c
    n = max(bm.kv8_plan_bytes(B, T, qh, c.kv_heads) - short, 0)
    return bm.lib().kv8_plan(ctypes.addressof(c), qh, *v, B, T, plan, n, None)


def _attend(c=None, qh=4, B=3, T=10, plan=P, Q=P, O=P, ws=P, scale=0.125, short=0, short_plan=0):
    c = _cache() if c is None else c
    n = max(bm.kv8_plan_bytes(B, T, qh, c.kv_heads) - short_plan, 0)
    w = max(bm.kv8_rows_workspace_bytes(B, T, qh, c.kv_heads, c.head_dim, c.ctx_cap) - short, 0)
    return bm.lib().kv8_attend_rows(ctypes.addressof(c), plan, n, Q, qh, scale, O, B, T, ws, w, None)


def _accept(v=(P,) * 7, plan=P, n=1 << 30, B=3, T=10):
    return bm.lib().kv8_tree_accept(plan, n, *v, B, T, None)


def _keep(c=None, plan=P, n=1 << 30, path=P, kept=P, B=3):
    c = _cache() if c is None else c
    return bm.lib().kv8_tree_keep(ctypes.addressof(c), plan, n, path, kept, B, None)


@pytest.mark.parametrize("kw", BAD_CACHES, ids=lambda k: f"{list(k)[0]}={list(k.values())[0]}")
def test_bad_caches(kw):
    for call, name in ((_plan, "kv8_plan"), (_attend, "kv8_attend_rows"), (_keep, "kv8_tree_keep")):
        assert call(_cache(**kw)) == 1 and bm.last_error().startswith(name + ": ")


SIZES = [{"B": 0}, {"B": -1}, {"B": 1025}, {"T": 0}, {"T": -5}, {"T": (1 << 20) + 1}]


def test_plan_refusals():
    for kw in SIZES + [{"qh": 0}, {"qh": 3}, {"qh": 18}, {"qh": 1026}, {"plan": None}, {"plan": P + 8}, {"short": 1}]:
        assert _plan(**kw) == 1, kw
        assert bm.last_error().startswith("kv8_plan: ")
    for i in range(9):                       # slots lens counts parents row_start after row_slot row_index row_pos
        assert _plan(v=[P + 2 if i == j else P for j in range(9)]) == 1 and "aligned" in bm.last_error()
        if i not in (3, 8):
            assert _plan(v=[None if i == j else P for j in range(9)]) == 1 and "null" in bm.last_error()


def test_attend_refusals():
    for kw in SIZES + [{"qh": 0}, {"qh": 3}, {"qh": 18}, {"plan": None}, {"plan": P + 8}, {"Q": None}, {"Q": P + 8}, {"O": None}, {"O": P + 2},
                       {"ws": None}, {"ws": P + 4}, {"scale": 0.0}, {"scale": -1.0}, {"scale": float("inf")}, {"scale": float("nan")},
                       {"short": 1}, {"short_plan": 1}]:
        assert _attend(**kw) == 1, kw
        assert bm.last_error().startswith("kv8_attend_rows: ")


def test_accept_refusals():
    for kw in SIZES + [{"plan": None}, {"plan": P + 4}, {"n": 100}]:
        assert _accept(**kw) == 1, kw
        assert bm.last_error().startswith("kv8_tree_accept: ")
    for i in range(7):
        for bad in (None, P + 1):
            assert _accept(v=[bad if i == j else P for j in range(7)]) == 1, i
            assert bm.last_error().startswith("kv8_tree_accept: ")


def test_keep_refusals():
    for kw in ({"B": 0}, {"B": 1025}, {"plan": None}, {"plan": P + 4}, {"n": 100}, {"path": None}, {"path": P + 2}, {"kept": None}, {"kept": P + 1}):
        assert _keep(**kw) == 1, kw
        assert bm.last_error().startswith("kv8_tree_keep: ")


def test_sizes():
    assert bm.kv8_plan_bytes(0, 1, 4, 2) == 0 and bm.kv8_plan_bytes(1, 0, 4, 2) == 0 and bm.kv8_plan_bytes(1, 1, 5, 2) == 0
    assert bm.kv8_plan_bytes(1, 1, 9, 1) == 0 and bm.kv8_plan_bytes(1025, 1, 4, 2) == 0 and bm.kv8_plan_bytes(1024, 1 << 20, 1024, 128) > 0
    assert bm.kv8_rows_workspace_bytes(1, 1, 4, 2, 96, 10) == 0 and bm.kv8_rows_workspace_bytes(1, 1, 4, 2, 64, 0) == 0
    assert bm.kv8_rows_workspace_bytes(1, 1, 4, 2, 64, 10) > 0


@pytest.mark.parametrize("kvh", [1, 2, 4, 16, 32, 50, 76, 77, 152, 400])
def test_a_plan_and_a_workspace_do_for_everything_smaller(kvh):
    qh = 2 * kvh if kvh <= 400 else kvh
    rising = lambda sizes: all(a <= b for a, b in zip(sizes, sizes[1:]))  # noqa: E731
    counts = sorted({max(1, n + e) for n in [1, 100, 1000, 30000, 2 ** 19, 2 ** 20 - 2] + [64 * t for t in range(1, 300)] for e in (-1, 0, 1)})
    caps = sorted({max(1, n + e) for n in [1, 2 ** 29, 2 ** 31 - 2] + [2048 * 4 ** k for k in range(9)] + [128 * t for t in range(1, 400)] for e in (-1, 0, 1)})
    streams = range(1, 1025)
    ws = lambda B=3, T=700, cap=9000: bm.kv8_rows_workspace_bytes(B, T, qh, kvh, 64, cap)  # noqa: E731
    assert rising([bm.kv8_plan_bytes(3, n, qh, kvh) for n in counts]) and rising([bm.kv8_plan_bytes(b, 700, qh, kvh) for b in streams])
    assert rising([ws(T=n) for n in counts]) and rising([ws(B=b) for b in streams]) and rising([ws(cap=c) for c in caps])


def test_wrong_tensors_are_refused():
    """The binding refuses what has no shape, another type or another number of dimensions, with its own error."""
    import torch
    c = _cache()
    raw, c.address, c.device = _cache(), P, bm.binding._here()
    i, j, f = torch.zeros(3, dtype=torch.int32), torch.zeros(7, dtype=torch.int32), torch.zeros(3)
    many, plan = torch.zeros(3, 64, dtype=torch.int32), torch.zeros(10, dtype=torch.uint8)
    Q = torch.zeros(7, 4, 64, dtype=torch.bfloat16)
    start = torch.zeros(4, dtype=torch.int32)
    bad = [lambda: bm.kv8_plan(c, 4, None, i, i, start, i, j, j, j, plan), lambda: bm.kv8_plan(c, 4, i, i, i, start, i, None, j, j, plan),
           lambda: bm.kv8_plan(c, 4, i, f, i, start, i, j, j, j, plan), lambda: bm.kv8_plan(raw, 4, i, i, i, start, i, j, j, j, plan),
           lambda: bm.kv8_plan(c, 4, i, i, i, i, i, j, j, j, plan), lambda: bm.kv8_plan(c, 4, i, i, i, start, i, j, j, i, plan),
           lambda: bm.kv8_plan(c, 4, i, i, i, start, i, j, j, j, None), lambda: bm.kv8_plan(c, 4, i, i, i, start, i, j, j, j, plan, parents=i),
           lambda: bm.kv8_attend_rows(c, plan, None, Q, 3, plan), lambda: bm.kv8_attend_rows(c, plan, Q[0], Q, 3, plan),
           lambda: bm.kv8_attend_rows(c, plan, Q, Q[:6], 3, plan), lambda: bm.kv8_attend_rows(c, None, Q, Q, 3, plan),
           lambda: bm.kv8_attend_rows(None, plan, Q, Q, 3, plan), lambda: bm.kv8_attend_rows(c, plan, Q[:, :, :32].contiguous(), Q, 3, plan),
           lambda: bm.kv8_attend_rows(c, plan, Q, Q, 3, None), lambda: bm.kv8_tree_accept(plan, None, j, many, i, many, i, i),
           lambda: bm.kv8_tree_accept(plan, j, i, many, i, many, i, i), lambda: bm.kv8_tree_accept(plan, j, j, many[:, :60], i, many, i, i),
           lambda: bm.kv8_tree_accept(plan, j, j, many, None, many, i, i), lambda: bm.kv8_tree_keep(c, plan, i, i),
           lambda: bm.kv8_tree_keep(c, plan, many, None), lambda: bm.kv8_tree_keep(raw, plan, many, i)]
    for n, call in enumerate(bad):
        with pytest.raises(bm.BitMoeError) as e:
            call()
        assert "kv8_" in str(e.value), n


def test_hold_refusals():
    for args in ((-1, 0, 0), (5, 0, 0), (1, -1, 0), (1, 0, -1)):
        assert bm.lib().bm_test_kv8_rows_hold(*args) == 1 and bm.last_error().startswith("bm_test_kv8_rows_hold: ")
    assert bm.lib().bm_test_kv8_rows_hold(0, 0, 0) == 0


def test_status_without_a_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    with pytest.raises(bm.BitMoeError) as e:
        bm.kv8_rows_status()
    assert e.value.status == 5 and "kv8_rows_status" in e.value.message
