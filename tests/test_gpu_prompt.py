"""Whole-prompt attention and the tile masses against 64-bit definitions.

Bounds, per element of a row (counted before any run).  The weights are
rounded to fp16 once, half a step = 2^-11 of each; the output once, 2^-11 of
it; a score is a sum of d products in fp32, off by at most d 2^-24 of the sum
of their magnitudes, which a weight takes over as a relative error, with a few
units of 2^-24 for the exponential, the sum and the product.
"""

import math

import numpy as np
import pytest
import torch

from quantized_paged_kv_tile_b200 import build, kvq

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -11, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kvq.load_library()


def config(hkv, g, d=128, t=64):
    return kvq.Config(num_kv_heads=hkv, group_size=g, tile_tokens=t, bits_k=4, bits_v=4, iters=4, head_dim=d)


def rows(cfg, n, seed, std=1.0, pad=0):
    """q, k, v as slices of one projection with `pad` extra columns of NaN."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim
    x = torch.full((n, (hq + 2 * hkv) * d + pad), math.nan, dtype=torch.float16, device="cuda")
    y = torch.randn((n, hq + 2 * hkv, d), generator=gen, device="cuda")
    y[:, :hq] *= std
    x[:, :(hq + 2 * hkv) * d] = y.flatten(1).half()
    q = x[:, :hq * d].unflatten(1, (hq, d))
    k = x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = x[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    return q, k, v


def definition(cfg, q, k, v, lens, window=0, scale=None, starts=None):
    """(out, lse, mass, bound of out, bound of lse, relative bound of a weight) in 64 bits."""
    d, g, t = cfg.head_dim, cfg.group_size, cfg.tile_tokens
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    e_out, e_lse = torch.zeros_like(out), torch.zeros_like(lse)
    tiles = max(1, -(-max(lens) // t))
    mass = torch.zeros((len(lens), tiles), dtype=torch.float64, device="cuda")
    worst = 0.0
    at = 0
    for s, n in enumerate(lens):
        if starts is not None:
            at = starts[s]
        if n:
            see = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
            for h in range(cfg.num_q_heads):
                qq, kk, vv = q[at:at + n, h].double(), k[at:at + n, h // g].double(), v[at:at + n, h // g].double()
                x = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
                size = (qq.abs() @ kk.abs().T * scale).masked_fill(~see, 0.0).amax(1)
                lse[at:at + n, h] = torch.logsumexp(x, 1)
                p = torch.exp(x - lse[at:at + n, h, None])
                out[at:at + n, h] = p @ vv
                eps = d * U32 * size + 16 * U32 + U32 * lse[at:at + n, h].abs()
                worst = max(worst, float(eps.max()))
                e_out[at:at + n, h] = (U16 + 2 * eps)[:, None] * (p @ vv.abs()) + U16 * out[at:at + n, h].abs() + 2.0 ** -24
                # a weight below 2^-14 of the row's largest is rounded as a
                # subnormal fp16, to a multiple of 2^-24: off by half of that
                # (the maximum it is relative to is never above the row's)
                top = p.amax(1, keepdim=True)
                e_out[at:at + n, h] += 2.0 ** -25 * top * (((p < 1.01 * 2.0 ** -14 * top) & see).double() @ vv.abs())
                e_lse[at:at + n, h] = 2 * eps + 4 * U32 * lse[at:at + n, h].abs()
                counted = p[max(0, n - window) if window else 0:].sum(0)
                mass[s].index_add_(0, torch.arange(n, device="cuda") // t, counted)
        at += n
    return out, lse, mass, e_out, e_lse, worst


def call(cfg, q, k, v, lens, window=None, cu=None, max_len=None, scale=None, stream=None):
    n = q.shape[0]
    cu = np.concatenate([[0], np.cumsum(lens)]) if cu is None else cu
    cu = torch.tensor(np.asarray(cu), dtype=torch.int32, device="cuda")
    max_len = max(lens) if max_len is None else max_len
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mass = ws = None
    if window is not None:
        mass = torch.zeros((len(cu) - 1, max(1, -(-max_len // cfg.tile_tokens))), dtype=torch.float32, device="cuda")
        need = kvq.prompt_workspace_bytes(cfg, len(cu) - 1, n, max_len, window)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN where nothing writes
    kvq.prompt_attention(cfg, q, k, v, out, cu, max_len, lse=lse, mass=mass, mass_window=window or 0, workspace=ws,
                         softmax_scale=scale, dev_status=status, stream=stream)
    torch.cuda.synchronize()
    return out, lse, mass, int(status)


def check(cfg, q, k, v, lens, window=None, scale=None):
    out, lse, mass, status = call(cfg, q, k, v, lens, window, scale=scale)
    assert status == 0
    ref, ref_lse, ref_mass, e_out, e_lse, eps = definition(cfg, q, k, v, lens, window or 0, scale)
    assert bool(((out.double() - ref).abs() <= e_out).all()), float(((out.double() - ref).abs() / e_out).max())
    assert bool(((lse.double() - ref_lse).abs() <= e_lse).all()), float(((lse.double() - ref_lse).abs() / e_lse).max())
    if window is not None:
        # a mass is a sum of weights, each off by its relative bound, summed in
        # fp32 over at most 128 rows a step and a few thousand partial sums
        tol = (2 * eps + 4096 * U32) * ref_mass + 1e-30
        assert bool(((mass.double() - ref_mass).abs() <= tol).all()), float(((mass.double() - ref_mass).abs() / tol).max())


LENS = [[1], [2, 1], [0, 5, 0, 1, 0], [127], [128], [129], [31, 32, 33, 64, 65], [300, 1, 511], [700]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths(d, lens):
    cfg = config(2, 4, d)
    check(cfg, *rows(cfg, sum(lens), 1), lens)


@pytest.mark.parametrize("g", range(1, 9))
def test_groups(g):
    cfg = config(2, g)
    lens = [300, 7, 140]
    check(cfg, *rows(cfg, sum(lens), 2), lens, window=0)


@pytest.mark.parametrize("t", [32, 64, 128])
@pytest.mark.parametrize("window", [0, 1, 16, 33, 1000])
def test_masses(t, window):
    cfg = config(2, 3, t=t)
    lens = [400, 0, 1, 31, 129, 64]
    check(cfg, *rows(cfg, sum(lens), 3), lens, window=window)


@pytest.mark.parametrize("d", [64, 256])
def test_masses_other_head_sizes(d):
    cfg = config(1, 5, d, t=32)
    lens = [333, 40]
    check(cfg, *rows(cfg, sum(lens), 4), lens, window=0)
    check(cfg, *rows(cfg, sum(lens), 4), lens, window=50)


@pytest.mark.parametrize("std", [8.0, 40.0])
def test_peaked_scores(std):
    # scores spread over tens and hundreds: the running maximum moves often
    cfg = config(2, 4)
    lens = [600, 129]
    check(cfg, *rows(cfg, sum(lens), 5, std=std), lens, window=0)


def test_rising_scores():
    # every key beats all earlier ones by several log2 units, and falling
    cfg = config(1, 2)
    n = 500
    q, k, v = rows(cfg, n, 6)
    q.fill_(1.0)
    k.copy_((torch.arange(n, device="cuda", dtype=torch.float32) / 64.0).half()[:, None, None].expand_as(k))
    check(cfg, q, k, v, [n], window=0, scale=0.25)
    k.copy_(-k)
    check(cfg, q, k, v, [n], window=0, scale=0.25)


def test_padded_rows_and_strides():
    cfg = config(2, 4)
    lens = [100, 140]
    check(cfg, *rows(cfg, sum(lens), 7, pad=8), lens, window=0)


@pytest.mark.parametrize("g", [1, 3, 4, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_sequences(d, g):
    # enough work for every SM: units of two query tiles
    cfg = config(2, g, d, t=32)
    lens = [300, 7, 140, 0, 129, 64, 1] * 16
    check(cfg, *rows(cfg, sum(lens), 22), lens, window=0)
    lens = [1100, 700, 1333, 64, 1]
    cfg = config(2, 8, d)
    check(cfg, *rows(cfg, sum(lens), 25, std=4.0), lens, window=0)
    check(cfg, *rows(cfg, sum(lens), 26), lens, window=150)


@pytest.mark.parametrize("n", [129, 250, 384, 385, 900, 1500])
@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_over_many_keys(d, n):
    # less work than SMs: a query tile's keys go to two streams
    cfg = config(1, 2, d)
    check(cfg, *rows(cfg, n, 23, std=4.0), [n], window=0)
    check(cfg, *rows(cfg, n, 24), [n], window=20)


def test_long_and_many():
    cfg = config(1, 8)
    check(cfg, *rows(cfg, 3000, 8), [3000], window=0)
    lens = [int(x) for x in np.random.default_rng(9).integers(0, 40, 200)]
    cfg = config(2, 2)
    check(cfg, *rows(cfg, sum(lens), 9), lens, window=0)


def test_more_sequences_than_are_sorted():
    cfg = config(1, 2, d=64)
    lens = [int(x) for x in np.random.default_rng(10).integers(0, 4, 1500)]
    lens[700] = 300
    check(cfg, *rows(cfg, sum(lens), 10), lens, window=0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_hidden_values_stay_hidden(d, bad):
    """Later tokens, the next sequence and rows in no sequence hold values that
    would spoil everything they reach: the rows that do not see them keep the
    bits they have without them."""
    hidden_values(config(1, 4, d), bad, 0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_hidden_values_stay_hidden_among_many(d):
    hidden_values(config(2, 4, d), math.nan, 100)


def hidden_values(cfg, bad, more):
    lens, cu = [150, 70] + [1] * more, [3, 153] + list(range(223, 224 + more))
    n = 240 + more  # rows 0..2 and the last 17 are in no sequence
    q, k, v = rows(cfg, n, 11)
    clean_k, clean_v = k.clone(), v.clone()
    want, want_lse, want_mass, status = call(cfg, q, clean_k, clean_v, lens, 0, cu=cu, max_len=150)
    assert status == 0
    for x in (k, v):
        x[:3] = bad
        x[223 + more:] = bad
        x[3 + 100] = bad          # token 100 of the first sequence
        x[153 + 69] = bad         # the last token of the second
    got, got_lse, _, status = call(cfg, q, k, v, lens, 0, cu=cu, max_len=150)
    assert status == 0
    seen = torch.zeros(n, dtype=torch.bool)
    seen[3 + 100:153] = True
    seen[153 + 69] = True
    inside = torch.zeros(n, dtype=torch.bool)
    inside[3:223 + more] = True
    clean = (inside & ~seen).cuda()
    assert torch.equal(got[clean], want[clean]) and torch.equal(got_lse[clean], want_lse[clean])
    assert bool((got[~inside.cuda()] == 7.0).all()) and bool((got_lse[~inside.cuda()] == 7.0).all())
    # the bad key's own score is infinite or NaN, so the rows that see it are not finite
    assert not bool(torch.isfinite(got[seen.cuda()]).any())


def test_infinite_values_reach_the_rows_that_see_them():
    cfg = config(1, 2)
    n = 200
    q, k, v = rows(cfg, n, 12)
    v[90, 0, 5] = math.inf
    v[140, 0, 5] = -math.inf
    v[199, 0, 9] = math.nan
    out, _, _, status = call(cfg, q, k, v, [n])
    assert status == 0
    o = out.float()
    assert bool(torch.isfinite(o[:90]).all())
    assert bool((o[90:140, :, 5] == math.inf).all())
    assert bool(torch.isnan(o[140:, :, 5]).all())
    assert bool(torch.isnan(o[199, :, 9]).all()) and bool(torch.isfinite(o[:199, :, 9]).all())
    rest = torch.ones(cfg.head_dim, dtype=torch.bool)
    rest[[5, 9]] = False
    assert bool(torch.isfinite(o[:, :, rest.cuda()]).all())


def test_two_calls_give_the_same_bits():
    cfg = config(2, 4, t=32)
    lens = [800, 333, 5]
    q, k, v = rows(cfg, sum(lens), 13)
    a, b = call(cfg, q, k, v, lens, 0), call(cfg, q, k, v, lens, 0)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))


def test_mass_adds_to_what_is_there():
    cfg = config(1, 4)
    q, k, v = rows(cfg, 200, 14)
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    mass = torch.zeros((1, 9), dtype=torch.float32, device="cuda")
    mass[0, 5] = 3.0
    ws = torch.empty(kvq.prompt_workspace_bytes(cfg, 1, 200, 200), dtype=torch.uint8, device="cuda")
    out = torch.empty((200, 4, 128), dtype=torch.float16, device="cuda")
    for _ in range(2):
        kvq.prompt_attention(cfg, q, k, v, out, cu, 200, mass=mass, workspace=ws)
    # every row adds 1: 800 rows a call
    assert abs(float(mass[0, :4].sum()) - 1600.0) < 1600.0 * 1e-4
    assert float(mass[0, 5]) == 3.0 and float(mass[0, 4]) == 0.0 and float(mass[0, 6:].sum()) == 0.0


def test_bad_prefix_sums_are_reported():
    cfg = config(1, 4)
    q, k, v = rows(cfg, 100, 15)
    want = call(cfg, q, k, v, [40, 60])[0]
    for cu, good in (([0, 40, 101], slice(0, 40)), ([-1, 40, 100], slice(40, 100)), ([0, 40, 30], slice(0, 40)),
                     ([0, 40, 100], slice(0, 40))):
        out, _, _, status = call(cfg, q, k, v, [40, 60], cu=cu, max_len=60 if cu[2] != 100 or cu[0] else 59)
        assert status == kvq.KVQ_ERR_DEVICE_BOUNDS
        assert torch.equal(out[good], want[good])
        rest = torch.ones(100, dtype=torch.bool, device="cuda")
        rest[good] = False
        assert bool((out[rest] == 7.0).all())


def test_other_stream_and_graph():
    cfg = config(2, 4)
    lens = [300, 90]
    n = sum(lens)
    q, k, v = rows(cfg, n, 16)
    want, want_lse, want_mass, _ = call(cfg, q, k, v, lens, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(cfg, q, k, v, lens, 0, stream=side)
    assert torch.equal(got[0], want) and torch.equal(got[2], want_mass)
    cu = torch.tensor([0, 300, 390], dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    mass = torch.zeros_like(want_mass)
    ws = torch.empty(kvq.prompt_workspace_bytes(cfg, 2, n, 300), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mass.zero_()
        kvq.prompt_attention(cfg, q, k, v, out, cu, 300, lse=lse, mass=mass, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(mass, want_mass)


def test_offsets_past_32_bits():
    # 2^31 output elements are passed: the last sequences lie behind them
    cfg = config(8, 8)
    n = 262144 + 600
    lens = [128] * 2048 + [7, 593]
    q = torch.zeros((n, 64, 128), dtype=torch.float16, device="cuda")
    k = torch.zeros((n, 8, 128), dtype=torch.float16, device="cuda")
    v = torch.zeros((n, 8, 128), dtype=torch.float16, device="cuda")
    tq, tk, tv = rows(cfg, 600, 17)
    q[-600:], k[-600:], v[-600:] = tq, tk, tv
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    lse = torch.full((n, 64), 7.0, dtype=torch.float32, device="cuda")
    kvq.prompt_attention(cfg, q, k, v, out, cu, 593, lse=lse)
    ref, ref_lse, _, e_out, e_lse, _ = definition(cfg, tq, tk, tv, [7, 593])
    assert bool(((out[-600:].double() - ref).abs() <= e_out).all())
    assert bool(((lse[-600:].double() - ref_lse).abs() <= e_lse).all())
    assert bool((out[:-600] == 0).all())  # values of zero
    uniform = torch.log(torch.arange(1, 129, device="cuda", dtype=torch.float32))  # scores of zero: ln of the keys seen
    assert bool(((lse[262016:262144] - uniform[:, None]).abs() < 1e-5).all())


def test_calls_at_once_on_two_streams():
    cfg = config(2, 4)
    lens = [900, 40, 333]
    n = sum(lens)
    data = [rows(cfg, n, 18 + i) for i in range(2)]
    want = [call(cfg, *x, lens, 0) for x in data]
    cu = torch.tensor([0, 900, 940, 1273], dtype=torch.int32, device="cuda")
    need = kvq.prompt_workspace_bytes(cfg, 3, n, 900)
    sets = [dict(out=torch.zeros_like(want[0][0]), lse=torch.zeros_like(want[0][1]),
                 mass=torch.zeros_like(want[0][2]), ws=torch.empty(need, dtype=torch.uint8, device="cuda"),
                 stream=torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s in sets:
            with torch.cuda.stream(s["stream"]):
                s["mass"].zero_()
        for x, s in zip(data, sets):
            kvq.prompt_attention(cfg, *x, s["out"], cu, 900, lse=s["lse"], mass=s["mass"], workspace=s["ws"],
                                 stream=s["stream"])
    torch.cuda.synchronize()
    for w, s in zip(want, sets):
        assert torch.equal(w[0], s["out"]) and torch.equal(w[1], s["lse"]) and torch.equal(w[2], s["mass"])


def test_tensors_of_another_device_are_refused(monkeypatch):
    cfg = config(1, 1)
    q, k, v = rows(cfg, 4, 20)
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    out = torch.zeros(q.shape, dtype=torch.float16, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        kvq.prompt_attention(cfg, q, k, v, out, cu, 4)


def test_no_row_and_no_length():
    cfg = config(1, 2)
    q, k, v = rows(cfg, 5, 21)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    for cu, top in (([0, 0, 0], 4), ([0], 4), ([0, 5], 0)):
        kvq.prompt_attention(cfg, q, k, v, out, torch.tensor(cu, dtype=torch.int32, device="cuda"), top)
    empty = torch.empty((0, 2, 128), dtype=torch.float16, device="cuda")
    kv = torch.empty((0, 1, 128), dtype=torch.float16, device="cuda")
    kvq.prompt_attention(cfg, empty, kv, kv, empty, torch.tensor([0, 0], dtype=torch.int32, device="cuda"), 0)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
