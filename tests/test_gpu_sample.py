"""bm_sample against its definition in 64 bits.

A token has to be the 64-bit one wherever no comparison of the row is closer
than 2^-26 of the weight it is made with (the weights are exact to better than
2^-29 each); the log probability is within fp32 rounding."""

import numpy as np
import pytest
import torch

import kv8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bm():
    import bit_moe_decode_w4a16_gb300 as m
    m.build()
    return m


def _call(bm, x, temp=None, top_k=None, top_p=None, min_p=None, u=None, logp=True, stream=None):
    B = x.shape[0]
    f = lambda v: None if v is None else torch.as_tensor(np.asarray(v, np.float32)).cuda()  # noqa: E731
    ids = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((B,), 7.0, device="cuda") if logp else None
    k = None if top_k is None else torch.as_tensor(np.asarray(top_k, np.int32)).cuda()
    bm.bm_sample(x, f(temp), k, f(top_p), f(min_p), f(u), ids, lp, stream=stream)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), None if lp is None else lp.double().cpu().numpy()


def _check(bm, x, temp, top_k, top_p, min_p, u, least=0.9):
    f32 = lambda v: np.asarray(v, np.float32)  # noqa: E731
    temp, top_p, min_p, u, top_k = f32(temp), f32(top_p), f32(min_p), f32(u), np.asarray(top_k)
    ids, lp = _call(bm, x, temp, top_k, top_p, min_p, u)
    want, wlp, margin = ref.sample(x, temp, top_k, top_p, min_p, u)
    clear = margin > 2.0 ** -26
    assert clear.mean() >= least
    np.testing.assert_array_equal(ids[clear], want[clear])
    fine = clear & np.isfinite(wlp)
    # the logarithm is rounded to fp32; a weight and the sum are each within 2^-29
    assert (np.abs(lp - wlp)[fine] <= 2.0 ** -24 * np.abs(wlp[fine]) + 2.0 ** -27).all(), np.abs(lp - wlp)[fine].max()
    assert (lp[clear & ~np.isfinite(wlp)] == -np.inf).all()
    return ids


def _logits(B, V, seed, dtype=torch.float32, spread=2.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (spread * torch.randn(B, V, generator=g, device="cuda")).to(dtype)


VOCABS = [1, 2, 31, 257, 1000, 4099, 50257, 151936, 300001]


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_settings(bm, V, dtype):
    """Every filter alone and together, from one kept token to all."""
    rows = [(1.0, 0, 1.0, 0.0), (0.7, 1, 1.0, 0.0), (1.3, 2, 1.0, 0.0), (1.0, 50, 1.0, 0.0), (1.0, V, 1.0, 0.0),
            (1.0, V - 1, 1.0, 0.0), (1.0, 5000, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (0.6, 0, 0.5, 0.0), (1.0, 0, 0.999, 0.0),
            (1.0, 0, 1e-6, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 0.05), (1.0, 0, 1.0, 1.0), (1.0, 0, 1.0, 2.0),
            (0.8, 50, 0.95, 0.02), (1.2, 400, 0.5, 0.001), (2.0, 3000, 0.99, 1e-5), (0.05, 0, 0.9, 0.0), (50.0, 0, 0.9, 0.0),
            (1000.0, 7, 0.3, 0.0), (0.0, 5, 0.5, 0.1), (-1.0, 0, 1.0, 0.0), (float("nan"), 0, 1.0, 0.0),
            (1.0, -3, -0.5, -1.0), (1.0, 0, float("nan"), float("nan"))]
    temp, k, p, m = zip(*rows)
    p = np.where(np.isnan(p), 1.0, p)
    m = np.where(np.isnan(m), 0.0, m)
    u = np.random.RandomState(V).randint(0, 1 << 24, len(rows)) / float(1 << 24)
    _check(bm, _logits(len(rows), V, V, dtype), temp, k, p, m, u, least=0.8)


def test_many_draws_of_one_row(bm):
    """The whole range of u over one distribution: 0, the last one below 1, and a grid."""
    V, B = 3000, 512
    x = _logits(1, V, 3).expand(B, V)             # rows of stride 0 are refused below; these are copies
    u = np.concatenate([[0.0, 1 - 2.0 ** -24], np.linspace(0, 1, B - 2, endpoint=False)])
    ids = _check(bm, x.contiguous(), np.ones(B), np.zeros(B, int), np.ones(B), np.zeros(B), u)
    assert (np.diff(ids[2:]) >= 0).all() and ids[0] == 0


def test_ties_go_to_the_lowest_index(bm):
    V = 5000
    x = torch.zeros(6, V, device="cuda")
    x[1, ::2] = 1.0
    x[2, 100:] = -float("inf")
    x[3] = 5.0 * (torch.arange(V, device="cuda") % 3 == 1)
    x[4] = -0.0
    x[4, ::5] = 0.0
    k, p = [10, 10, 0, 40, 5000, 3], [1.0, 1.0, 0.5, 1.0, 0.25, 1.0]
    for u in (0.0, 0.51, 0.999):
        ids = _check(bm, x, np.ones(6), k, p, np.zeros(6), np.full(6, u), least=0.5)
        assert ids[0] < 10 and ids[1] % 2 == 0 and ids[1] < 20 and ids[2] < 50 and ids[3] % 3 == 1 and ids[3] < 120
        assert ids[4] < 1250 and ids[5] < 3


def test_greedy_is_the_first_maximum(bm):
    x = _logits(5, 10000, 9, torch.bfloat16)
    x[0, 77] = x[0, 5000] = 50
    x[1, 9999] = 60
    x[2, 0] = 60
    ids, lp = _call(bm, x, temp=np.zeros(5), u=np.full(5, 0.9))
    want = [int((x[b] == x[b].max()).nonzero()[0]) for b in range(5)]
    assert ids.tolist() == want and ids[0] == 77 and (lp == 0).all()


def test_masked_infinite_and_nan_logits(bm):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    V = 3000
    x = _logits(9, V, 4)
    x[0] = -inf
    x[1] = nan
    x[2] = -inf
    x[2, 1234] = -3.0
    x[3] = low
    x[4, 1:] = low
    x[5, 7] = x[5, 2000] = inf
    x[6, ::2] = nan
    x[7] = low
    x[7, 50:60] = 3.0
    x[8] = torch.finfo(torch.float32).max
    x[8, ::3] = low
    for T in (1.0, 0.0, 1e-30, 1e30):
        for u in (0.0, 0.6):
            ids, lp = _call(bm, x, temp=np.full(9, T), u=np.full(9, u))
            assert ids[0] == -1 and ids[1] == -1 and lp[0] == -np.inf and lp[1] == -np.inf
            assert ids[2] == 1234 and lp[2] == 0
            assert ids[3] == (0 if T == 0 else int(u * V))
            assert ids[4] == 0 or T == 1e30
            assert ids[5] == (7 if u < 0.5 or T == 0 else 2000)
            assert ids[6] % 2 == 1
            assert 50 <= ids[7] < 60 or T == 1e30
            assert ids[8] % 3 != 0 or T == 1e30


def test_rows_strides_streams_and_optional_arguments(bm):
    big = _logits(6, 2100, 5)
    x = big[:, 3:2003]                      # rows of stride 2100 that start off a 16-byte boundary
    u = np.linspace(0, 0.99, 6)
    whole = _check(bm, x, np.ones(6), np.full(6, 20), np.full(6, 0.9), np.zeros(6), u, least=0.5)
    for b in range(6):
        solo, _ = _call(bm, x[b:b + 1], np.ones(1), [20], [0.9], [0.0], u[b:b + 1])
        assert solo[0] == whole[b]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids, none = _call(bm, x, np.ones(6), np.full(6, 20), np.full(6, 0.9), u=u, logp=False, stream=side)
    assert none is None and (ids == whole).all()
    plain, _ = _call(bm, x, u=u)
    want, _, margin = ref.sample(x, np.ones(6), np.zeros(6), np.ones(6), np.zeros(6), np.float32(u))
    assert (plain == want)[margin > 2.0 ** -26].all()
    odd = _logits(3, 1001, 6, torch.bfloat16)[:, 1:]
    _check(bm, odd, np.ones(3), [5, 0, 0], [1, 0.5, 1], [0, 0, 0.1], [0.1, 0.5, 0.9], least=0.3)


def test_temperatures_at_the_ends(bm):
    """An infinite temperature makes all finite logits equal; the smallest ones leave the first of the largest."""
    V = 40000
    x = _logits(4, V, 21)
    x[1, 5:] = -float("inf")
    x[3] = 1.25
    for T in (float("inf"), 3e38):
        for p in (1.0, 0.5):
            ids = _check(bm, x, np.full(4, T), np.zeros(4, int), np.full(4, p), np.zeros(4), np.full(4, 0.3), least=0.0)
            assert ids[1] < 5 and (p == 1.0) <= (abs(ids[0] - 0.3 * V) <= 1) and abs(ids[3] - 0.3 * p * V) <= 1
    ids, lp = _call(bm, x, temp=np.full(4, float("inf")), top_k=np.array([10, 3, 100, V]), u=np.full(4, 0.5))
    top = x[0].topk(10).indices.sort().values.cpu().numpy()
    assert ids[0] == top[5] and ids[1] in x[1].topk(3).indices and ids[3] == V // 2
    np.testing.assert_allclose(lp, -np.log([10, 3, 100, V]), rtol=2 ** -23)
    for T in (1e-45, 1e-38, 1e-20):
        ids, lp = _call(bm, x[:2], temp=np.full(2, T), top_p=np.full(2, 0.9), u=np.full(2, 0.999))
        assert (ids == x[:2].argmax(1).cpu().numpy()).all() and (lp == 0).all()


@pytest.mark.parametrize("V", [151936, 300001])
def test_few_distinct_values(bm, V):
    """Steps that hold far more logits than are gathered: cuts inside runs of equal values, across every CTA."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = torch.randint(0, 3, (6, V), generator=g, device="cuda").float() * 0.01
    x[4:] = torch.randint(0, 400, (2, V), generator=g, device="cuda").float() * 1e-5
    k, p = [7, V // 2, 0, V - V // 5, 60000, 0], [1.0, 1.0, 0.4, 0.9, 0.7, 0.55]
    _check(bm, x, np.full(6, 0.9), k, p, np.zeros(6), [0.99, 0.7, 0.8, 0.999, 0.6, 0.1], least=0.5)


def test_u_outside_its_range(bm):
    x = _logits(4, 500, 8)
    ids, _ = _call(bm, x, u=[-1.0, float("nan"), 1.0, 5.0])
    assert ids[0] == 0 and ids[1] == 0 and ids[2] == 499 and ids[3] == 499


def test_largest_vocabulary(bm):
    V = 524288
    x = _logits(2, V, 12)
    _check(bm, x, [1.0, 0.9], [0, 100], [0.95, 0.9], [0, 0], [0.3, 0.7], least=0.5)


def test_graph_replay_takes_new_numbers(bm):
    x = _logits(4, 20000, 13)
    u, temp = torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        bm.bm_sample(x, temp, None, None, None, u, ids, stream=side)
    for v in (0.1, 0.5, 0.9):
        u.fill_(v)
        graph.replay()
        torch.cuda.synchronize()
        want, _, margin = ref.sample(x, np.ones(4), np.zeros(4), np.ones(4), np.zeros(4), np.full(4, np.float32(v)))
        assert (ids.cpu().numpy() == want)[margin > 2.0 ** -26].all()


def test_after_decode_step(bm):
    """The engine's logits, sampled on the device, feed its next step; a temperature of 0 gives its own greedy ids."""
    import synth
    from gpu_side import build_engine, seed_stream
    name, cfg = "tiny_layer", synth.CONFIGS["tiny_layer"]
    e = build_engine(name, cfg, 1, max_streams=4, ctx_cap=128, gen_device="cpu")
    try:
        slots = [seed_stream(e, name, cfg, i, L, 1, gen_device="cpu") for i, L in enumerate(cfg["lens"])]
        B, V = len(slots), cfg["vocab"]
        toks = torch.tensor([1 + i for i in range(B)], dtype=torch.int32, device="cuda")
        nxt = torch.empty(B, dtype=torch.int32, device="cuda")
        logits = torch.empty(B, V, device="cuda")
        rs = np.random.RandomState(1)
        for _ in range(4):
            bm.decode_step(e, slots, toks, nxt, logits)
            greedy, _ = _call(bm, logits, temp=np.zeros(B), u=np.zeros(B))
            assert (greedy == nxt.cpu().numpy()).all()
            u = rs.rand(B).astype(np.float32)
            ids = _check(bm, logits, np.full(B, 0.8), np.full(B, 40), np.full(B, 0.95), np.zeros(B), u, least=0.0)
            toks = torch.from_numpy(ids.astype(np.int32)).cuda()
        bm.bm_engine_sync(e)
    finally:
        bm.bm_engine_destroy(e)


def test_refusals(bm):
    x = _logits(2, 100, 1)
    u, ids = torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [lambda: bm.bm_sample(x.half(), None, None, None, None, u, ids), lambda: bm.bm_sample(x.t(), None, None, None, None, u, ids),
           lambda: bm.bm_sample(x, None, None, None, None, None, ids), lambda: bm.bm_sample(x, u.double(), None, None, None, u, ids),
           lambda: bm.bm_sample(x, None, u, None, None, u, ids), lambda: bm.bm_sample(x, None, None, None, None, u[:1], ids),
           lambda: bm.bm_sample(x.cpu(), None, None, None, None, u, ids),
           lambda: bm.bm_sample(x[:1].expand(2, 100), None, None, None, None, u, ids),
           lambda: bm.bm_sample(torch.zeros(1, 524289, device="cuda"), None, None, None, None, u[:1], ids[:1])]
    for i, call in enumerate(bad):
        with pytest.raises(bm.BitMoeError):
            call()
            pytest.fail(f"call {i} was accepted")


@pytest.mark.parametrize("V", [1000, 20000, 60000])
def test_rows_do_not_depend_on_the_batch(bm, V):
    """From one row to a thousand the work is cut into clusters of 16 to 1 CTAs; ids and log probabilities are the same bits."""
    n = 7
    x = _logits(n, V, 31)
    x[5, 100:] = -float("inf")
    x[6] = x[6].bfloat16().float()
    s = dict(temp=[1.0, 0.7, 1.3, 0.9, 0.0, 1.0, 1.0], top_k=[0, 50, 0, 5000, 0, 0, 0], top_p=[0.9, 0.95, 1, 0.5, 1, 0.8, 0.7],
             min_p=[0, 0, 0.02, 0.001, 0, 0, 0], u=[0.5, 0.1, 0.9, 0.3, 0.2, 0.6, 0.999])
    alone = [_call(bm, x[i:i + 1], **{k: [v[i]] for k, v in s.items()}) for i in range(n)]
    want, wlp = np.concatenate([a[0] for a in alone]), np.concatenate([a[1] for a in alone])
    for B in (n, 15, 16, 33, 65, 130, 257, 1000):
        row = np.arange(B) % n
        ids, lp = _call(bm, x[torch.as_tensor(row).cuda()], **{k: np.asarray(v)[row] for k, v in s.items()})
        np.testing.assert_array_equal(ids, want[row])
        np.testing.assert_array_equal(lp, wlp[row])


@pytest.mark.parametrize("V", [1000, 20000, 151936])
def test_top_k_of_every_size(bm, V):
    """k below, at and above what the threads' largest logits can bound, in rows whose largest lie together or apart."""
    ks = [1, 2, 31, 32, 33, 127, 128, 129, 500, 1024, 1025, 2048, 2049, 5000, V - 1, V]
    n = len(ks)
    x = _logits(n, V, 41)
    x[1::4] = x[1::4].sort(dim=1, descending=True).values       # the largest in one thread's and one warp's runs
    x[2::4] = (x[2::4] * 4).round() / 4                         # runs of equal logits at every cut
    x[3::4, 7:] = torch.where(torch.arange(7, V, device="cuda") % 5 == 0, x[3::4, 7:], -float("inf"))
    u = (np.arange(n) + 0.5) / n
    _check(bm, x, np.full(n, 1.1), ks, np.ones(n), np.zeros(n), u, least=0.8)
    _check(bm, x, np.full(n, 0.8), ks, np.full(n, 0.9), np.zeros(n), 1 - u, least=0.8)
