"""Waits inside kv8_attend_rows that run out: a part of what one CTA makes is
held back from who waits for it.  Its rows become NaN, the others keep their bytes, the status
tells of it once, and the next call on the same plan and workspace is right.
The waits end after about a second; nothing faults."""

import random

import pytest
import torch

from kv8_ref import E4M3, INT8
from test_gpu_kv8_step import FILL, HEAD, ITEM, Step, _filled, _rows, _tree

pytestmark = pytest.mark.gpu

KEYS, VALUES, QUERIES, WEIGHTS = 1, 2, 3, 4
SMS = 152


@pytest.fixture(scope="module")
def bm():
    import bit_moe_decode_w4a16_gb300 as m
    m.build()
    return m


@pytest.fixture(autouse=True)
def nothing_left(bm):
    bm.kv8_rows_status()
    yield
    bm.bm_test_kv8_rows_hold(0)
    torch.cuda.synchronize()


def _pieces_of(s, cta):
    """(stream, kv head, block, tiles, query rows from the block's first on) of each piece that a CTA has, in its order."""
    raw = s.plan.cpu().numpy()
    head = raw[:64].view(HEAD)[0]
    items = raw[64 + 64 * s.B + (s.T + 1) // 2 * 16:].view(ITEM)[:head["items"]]
    _, streams = s.want()
    out = []
    for r in range(len(items) // SMS + 1):
        i = r * SMS + (SMS - 1 - cta if r & 1 else cta)
        if i < len(items):
            it = items[i]
            b, block = int(it["who"]) & 1023, int(it["what"]) & 65535
            rows = streams[b][1] * (s.qh // s.cache["kv_heads"]) - 256 * block
            out.append((b, int(it["who"]) >> 10, block, int(it["t1"] - it["t0"]), rows))
    return out


def _case(name, bm):
    rs = random.Random(3)
    fmt, qh, kvh, d, parents = E4M3, 32, 4, 128, None
    if name == "wide":                       # whole blocks of more than 128 query rows
        counts, lens = [300, 64, 200], [0, 40, 7]
    elif name == "wide cut":
        counts, lens = [100], [6000]
    elif name == "narrow":                   # whole blocks of up to 128: both halves have the same rows
        counts, lens, fmt = [10, 3, 16], [100, 300, 20], INT8
    elif name == "narrow cut":
        counts, lens, parents = [13], [4096], _tree(13, rs)
    else:                                    # CTAs with many pieces, of one or two tiles
        lens = [rs.randrange(250) for _ in range(300)]
        counts, kvh, d = [rs.choice([1, 2, 7, 20]) for _ in lens], 8, 64
    cache = _filled(fmt, lens, counts, kvh, d, 50)
    return Step(bm, cache, qh, list(range(len(lens))), lens, counts, sum(counts) + 1, None if parents is None else parents + [-1])


@pytest.mark.parametrize("what", [KEYS, VALUES, QUERIES, WEIGHTS], ids=["keys", "values", "queries", "weights"])
@pytest.mark.parametrize("name,cta,share", [("wide", 0, 0.0), ("wide", 5, 0.6), ("wide cut", 1, 0.5), ("narrow", 2, 0.0), ("narrow", 0, 0.9),
                                            ("narrow cut", 3, 0.5), ("many", 7, 0.0), ("many", 11, 0.4), ("many", 1, 0.9)])
def test_a_wait_that_runs_out(bm, name, cta, share, what):
    s = _case(name, bm)
    Q = _rows(s.T, s.qh, s.cache["head_dim"])
    want = s.attend(Q)
    bm.kv8_rows_status()
    pieces = _pieces_of(s, cta)
    assert pieces
    if what == QUERIES:
        n = len(pieces)
    elif what == WEIGHTS:                    # the first half's steps: all tiles, or every second where the halves have the same rows
        n = sum(p[3] if p[4] > 128 else (p[3] + 1) // 2 for p in pieces)
    else:
        n = sum(p[3] for p in pieces)
    bm.bm_test_kv8_rows_hold(what, cta, int(share * n))
    got = s.attend(Q)
    bm.bm_test_kv8_rows_hold(0)
    with pytest.raises(bm.BitMoeError) as e:
        bm.kv8_rows_status()
    assert e.value.status == 8 and "in 1 CTAs" in e.value.message
    bm.kv8_rows_status()                     # told once
    _, streams = s.want()
    G = s.qh // s.cache["kv_heads"]
    bad = torch.zeros(s.T, s.qh, dtype=torch.bool)
    for b, kh, block, _, _ in pieces:
        start, rows, _ = streams[b]
        for q in range(256 * block, min(256 * block + 256, rows * G)):
            bad[start + q // G, kh * G + q % G] = True
    bad = bad.cuda()
    assert got[bad].isnan().all()
    assert torch.equal(got[~bad], want[~bad]) and (got[-1] == FILL).all()
    assert torch.equal(s.attend(Q), want)    # the same plan and workspace
    bm.kv8_rows_status()


def test_a_tile_that_the_cta_does_not_have(bm):
    s = _case("wide", bm)
    Q = _rows(s.T, s.qh, 128)
    want = s.attend(Q)
    bm.bm_test_kv8_rows_hold(KEYS, 0, 1000)
    assert torch.equal(s.attend(Q), want)
    bm.kv8_rows_status()


def test_status_refuses_a_captured_stream(bm):
    s = _case("narrow", bm)
    Q = _rows(s.T, s.qh, 128)
    O = s.attend(Q)
    want = O.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.attend(Q, O)
        with pytest.raises(bm.BitMoeError) as e:
            bm.kv8_rows_status()
    assert e.value.status == 1
    O.fill_(FILL)
    g.replay()
    bm.kv8_rows_status()
    assert torch.equal(O, want)


def test_threads_that_ask_at_once(bm):
    """Each CTA is told of once, to one of them."""
    import re
    import threading
    s = _case("wide", bm)
    Q = _rows(s.T, s.qh, 128)
    for cta in (0, 3, 9):
        bm.bm_test_kv8_rows_hold(KEYS, cta, 0)
        s.attend(Q)
    bm.bm_test_kv8_rows_hold(0)
    told, others = [], []
    stream = torch.cuda.current_stream()

    def ask():
        for _ in range(20):
            try:
                bm.kv8_rows_status(stream)
            except bm.BitMoeError as e:
                (told if e.status == 8 else others).append(int(re.search(r"in (\d+) CTAs", e.message).group(1)))

    threads = [threading.Thread(target=ask) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sum(told) == 3 and not others
