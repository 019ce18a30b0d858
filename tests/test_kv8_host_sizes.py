"""Sizes, addresses and shapes that the 8-bit cache calls and the sampler accept or refuse, without a device."""

import ctypes

import pytest

import bit_moe_decode_w4a16_gb300 as bm


@pytest.fixture(scope="module", autouse=True)
def built():
    bm.build()
    return bm.lib()


@pytest.mark.parametrize("kvh", [1, 2, 3, 4, 8, 16, 32, 50, 152, 400])
def test_a_workspace_does_for_everything_smaller(kvh):
    size = lambda B=3, cap=300, P=0: bm.kv8_workspace_bytes(B, 2 * kvh, kvh, 64, cap, P)  # noqa: E731
    lengths = sorted({max(1, n + e) for n in [1, 100, 2 ** 22, 2 ** 29, 2 ** 30, 2 ** 31 - 2] + [128 * t for t in range(1, 500)] for e in (-1, 0, 1)})
    for name in ("P", "cap"):
        sizes = [size(**{name: n}) for n in lengths]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), name
    sizes = [size(B=b, P=5000) for b in range(1, 512 // kvh + 2)]
    assert all(a < b for a, b in zip(sizes, sizes[1:]))


P = 1 << 20   # an aligned address that no refused call may touch


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_vectors_are_refused(off):
    """int32 and fp32 vectors off a 4-byte boundary: refused on the host, as the GPU would fault on them."""
    L, bad = bm.lib(), P + off
    c = bm.bm_kv8_cache(0, 4, 100, 2, 64, P, P, P, P)
    a = ctypes.addressof(c)
    for i in range(4):
        v = [bad if i == j else P for j in range(4)]           # slots, index, rope_pos, inv_freq
        r = bm.bm_kv8_rope(0, 0.0, None, None, v[3])
        assert L.kv8_append(a, P, 6 * 64, 2, ctypes.addressof(r), v[0], v[1], v[2], P, 3, None) == 1, i
        assert bm.last_error().startswith("kv8_append: ")
    for slots, lens in ((bad, P), (P, bad)):
        assert L.kv8_attend(a, P, slots, lens, 4, 0.125, P, 3, P, 1 << 30, None) == 1
        assert bm.last_error().startswith("kv8_attend: ")
        assert L.kv8_attend_prefix(a, a, 0, 5, P, slots, lens, 4, 0.125, P, 3, P, 1 << 30, None) == 1
        assert bm.last_error().startswith("kv8_attend_prefix: ")
    for i in range(7):
        v = [bad if i == j else P for j in range(7)]           # temperature, top_k, top_p, min_p, u, ids, logprobs
        assert L.bm_sample(P, 0, 100, 100, 2, *v, None) == 1, i
        assert bm.last_error().startswith("bm_sample: ")


def test_missing_and_wrongly_shaped_arguments():
    """The binding refuses what has no shape or another number of dimensions, with its own error."""
    import torch
    c, r = bm.bm_kv8_cache(0, 4, 100, 2, 64, P, P, P, P), bm.bm_kv8_rope(0, 0.0, None, None, None)
    raw, c.address, r.address, r.fits = bm.bm_kv8_cache(0, 4, 100, 2, 64, P, P, P, P), P, P, set()
    c.device = r.device = bm.binding._here()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i, ws, x = torch.zeros(3, dtype=torch.int32), torch.zeros(10, dtype=torch.uint8), torch.zeros(3)
    Q = bf(3, 4, 64)
    bad = [lambda: bm.kv8_append(c, bf(3, 512), r, i, i, bf(3, 256)), lambda: bm.kv8_append(c, bf(3, 512), r, i, i, None),
           lambda: bm.kv8_append(c, None, r, i, i, Q), lambda: bm.kv8_append(c, bf(3, 8, 64), r, i, i, Q),
           lambda: bm.kv8_append(None, bf(3, 512), r, i, i, Q), lambda: bm.kv8_append(c, bf(3, 512), None, i, i, Q),
           lambda: bm.kv8_append(raw, bf(3, 512), r, i, i, Q), lambda: bm.kv8_read(None, 0, 0, 1, Q, Q),
           lambda: bm.kv8_attend(c, bf(3, 256), i, i, Q, ws), lambda: bm.kv8_attend(c, None, i, i, Q, ws),
           lambda: bm.kv8_attend(None, Q, i, i, Q, ws), lambda: bm.kv8_attend_prefix(c, None, 0, 5, Q, i, i, Q, ws),
           lambda: bm.kv8_attend_prefix(c, c, 0, 5, bf(64), i, i, Q, ws), lambda: bm.bm_sample(x, None, None, None, None, x, i),
           lambda: bm.bm_sample(None, None, None, None, None, x, i), lambda: bm.bm_sample(torch.zeros(1, 3, 4), None, None, None, None, x, i)]
    for n, call in enumerate(bad):
        with pytest.raises(bm.BitMoeError) as e:
            call()
        assert e.value.args and ("kv8_" in str(e.value) or "bm_sample" in str(e.value)), n
