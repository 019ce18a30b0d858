"""Sizes, addresses and shapes that the 8-bit cache calls and the sampler accept or refuse, without a device."""

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
