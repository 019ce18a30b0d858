"""No position of a long stream or prefix is lost or counted twice where tiles and chunks meet.

Keys on both sides of every multiple of 128 are parallel to one of eight
queries, so that few positions hold a query's weight and each of them shows
in the output: the test works out that leaving out any one of them would be
seen, before it looks at the kernel's output."""

import pytest
import torch

import kv8_ref as ref
from test_gpu_kv8 import BF16_HALF, E4M3, INT8, _attend, _check_rows, _i32, _spoil, bm  # noqa: F401

pytestmark = pytest.mark.gpu

ROWS = 8


def _marked(fmt, n, d, kvh, slots, slot, seed):
    """(cache, Q): positions 0, n - 1 and 128 i - 1, 128 i of the slot are keys of one of the queries each."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q = rnd(ROWS, kvh, d).bfloat16()
    k = 0.05 * rnd(slots, kvh, n + 2, d)
    marks = sorted({p for i in range(0, n + 129, 128) for p in (i - 1, i) if 0 <= p < n} | {n - 1})
    m = torch.tensor(marks, device="cuda")
    row = torch.arange(len(marks), device="cuda") % ROWS
    unit = q.float() / q.float().square().sum(-1, keepdim=True)
    k[slot][:, m] = (14 * d ** 0.5 * unit)[row].transpose(0, 1)      # a score of about 14
    cache = ref.random_cache(fmt, slots, n + 2, kvh, d, seed)
    s = k.abs().amax(-1, keepdim=True) / ref.CODE_MAX[fmt]
    y = k / s
    cache["K"] = (y.to(torch.float8_e4m3fn) if fmt == E4M3 else y.round().to(torch.int8)).view(torch.uint8)
    cache["Ks"] = s.squeeze(-1).contiguous()
    return cache, q, m, row


def _every_mark_shows(cache, slot, n, q, m, row, want, bound):
    """Without any one marked position its query's output would be off by twice what is allowed."""
    fmt, d = cache["format"], q.shape[-1]
    k, v = (ref.decode(cache[x][slot, :, :n], fmt) * cache[x + "s"][slot, :, :n].double().unsqueeze(-1) for x in ("K", "V"))
    for r in range(ROWS):
        p = torch.softmax(torch.einsum("hd,hnd->hn", q[r].double(), k) * d ** -0.5, -1)
        mine = m[row == r]
        pj = p[:, mine].unsqueeze(-1)
        shift = (pj / (1 - pj) * (want[r].unsqueeze(1) - v[:, mine])).abs()
        tol = (BF16_HALF * want[r].abs() + bound[r] * (1 + BF16_HALF)).unsqueeze(1)
        assert (shift > 2 * tol).any(-1).all(), r


# chunks of 256, 512, 1024 and 2048 positions
@pytest.mark.parametrize("n", [1000, 4096, 4097, 16384, 16385, 40001, 65537])
@pytest.mark.parametrize("fmt,d", [(E4M3, 128), (INT8, 128), (E4M3, 64)])
def test_borders_of_a_stream(bm, fmt, d, n):
    kvh = 2
    cache, q, m, row = _marked(fmt, n, d, kvh, 2, 1, n)
    _spoil(cache, 1, n)
    slots, lens = _i32(*[1] * ROWS), _i32(*[n] * ROWS)
    want, bound = ref.attend(cache, q, slots, lens, d ** -0.5)
    _every_mark_shows(cache, 1, n, q, m, row, want, bound)
    _check_rows(_attend(bm, cache, q, slots, lens), want, bound)


# chunks of one tile, of several, and several chunks to a CTA (300 streams)
@pytest.mark.parametrize("P,kvh,streams", [(1000, 2, 8), (9728, 2, 8), (9729, 2, 8), (20001, 8, 8), (9999, 4, 300), (40000, 2, 8)])
@pytest.mark.parametrize("fmt,d", [(E4M3, 128), (INT8, 64)])
def test_borders_of_a_prefix(bm, fmt, d, P, kvh, streams):
    prefix, q, m, row = _marked(fmt, P, d, kvh, 2, 1, P)
    _spoil(prefix, 1, P)
    cache = ref.random_cache(fmt, streams, 8, kvh, d, 91)
    Q = torch.randn(streams, kvh, d, device="cuda").bfloat16()
    at = streams - ROWS                                              # the marked rows are the last
    Q[at:] = q
    slots = torch.arange(streams, dtype=torch.int32, device="cuda")
    lens = torch.zeros(streams, dtype=torch.int32, device="cuda")
    want, bound = ref.attend(cache, Q[at:], slots[at:], lens[at:], d ** -0.5, prefix=(prefix, 1, P))
    _every_mark_shows(prefix, 1, P, q, m, row, want, bound)
    O = _attend(bm, cache, Q, slots, lens, prefix=prefix, p_slot=1, p_len=P)
    _check_rows(O[at:], want, bound)
