"""Whole-prompt attention at the edges of its numbers."""

import math

import numpy as np
import pytest
import torch

from quantized_paged_kv_tile_b200 import build, kvq

from test_gpu_prompt import U16, U32, call, check, config, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    return kvq.load_library()


# ------------------------------------------------------------------ masses
@pytest.mark.parametrize("n", [130, 260, 300])
@pytest.mark.parametrize("g", [3, 5, 6, 7])
@pytest.mark.parametrize("d", [64, 128])
def test_masses_of_low_scores(d, g, n):
    # Every score is -128 (-185 in log2 units).  Query tiles straddle a key
    # tile's border here, and few rows: a stream may hold a key tile that some
    # rows of the query tile do not see at all.
    for t, window in ((32, 0), (64, 0), (128, 0), (64, 9)):
        cfg = config(1, g, d, t)
        q, k, v = rows(cfg, n, 31)
        q.fill_(1.0)
        k.fill_(-128.0 / d)
        check(cfg, q, k, v, [n], window=window, scale=1.0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_nan_row_stays_out_of_the_tiles_it_does_not_see(d):
    # token 5 of the first sequence sees tile 0 (of 32 tokens); rows up to
    # token 63 are in the same query tile
    cfg = config(1, 2, d, t=32)
    lens = [100, 40]
    q, k, v = rows(cfg, 140, 32)
    want = call(cfg, q, k, v, lens, 0)[2]
    q[5, 1] = math.nan
    mass = call(cfg, q, k, v, lens, 0)[2]
    assert bool(torch.isnan(mass[0, 0]))
    # the tiles behind it: bit for bit, the row had no weight there
    assert torch.equal(mass[0, 1:], want[0, 1:]) and torch.equal(mass[1], want[1])


# ------------------------------------------------------------------ large scores
def one_channel(cfg, n, q0, k0, seed):
    """Rows whose scores are the products of their first channels: exact in fp32."""
    q, k, v = rows(cfg, n, seed)
    q.zero_()
    k.zero_()
    q[..., 0] = q0
    k[..., 0] = k0
    return q, k, v


@pytest.mark.parametrize("n,hkv", [(300, 1), (700, 40)])
@pytest.mark.parametrize("q0,k0", [(2048.0, 4096.0), (2048.0, -4096.0), (-3000.0, -3500.0), (64.0, -4096.0)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_equal_scores_of_any_size(d, q0, k0, n, hkv):
    """All scores of a row are the same number, up to 1.05e7: the weights are 1 / (i + 1)."""
    cfg = config(hkv, 2, d)
    q, k, v = one_channel(cfg, n, q0, k0, 33)
    out, lse, mass, status = call(cfg, q, k, v, [n], 0, scale=1.0)
    assert status == 0
    count = torch.arange(1, n + 1, device="cuda", dtype=torch.float64)[:, None, None]
    mean = v.double().cumsum(0).div(count).repeat_interleave(2, 1)
    size = v.double().abs().cumsum(0).div(count).repeat_interleave(2, 1)
    # equal weights are rounded alike, to at worst 2^-11 of them; the sums and the quotient in fp32
    bound = (U16 + (n + 16) * U32) * size + U16 * mean.abs() + 2.0 ** -24
    assert bool(((out.double() - mean).abs() <= bound).all())
    score = q0 * k0
    assert bool(((lse.double() - score).abs() <= math.log(n) + 8 * U32 * abs(score)).all())
    # row i gives 1 / (i + 1) to each token it sees, from every query head
    share = (1.0 / count[:, 0, 0]).flip(0).cumsum(0).flip(0) * cfg.num_q_heads
    tiles = torch.zeros(mass.shape[1], dtype=torch.float64, device="cuda")
    tiles.index_add_(0, torch.arange(n, device="cuda") // cfg.tile_tokens, share)
    assert bool(((mass[0].double() - tiles).abs() <= 4096 * U32 * tiles).all())


@pytest.mark.parametrize("base", [0.0, 2048.0, -2048.0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_weights_relative_to_a_large_maximum(d, base):
    """Scores of 2^22 + whole numbers that rise by 0 to 3 a key: the weights
    depend on the differences alone, also where the maximum moves."""
    cfg = config(1, 4, d)
    n = 400
    q, k, v = one_channel(cfg, n, 2048.0, base, 34)
    rise = torch.randint(0, 4, (n,), generator=torch.Generator().manual_seed(35)).cumsum(0)
    q[..., 1] = 1.0
    k[..., 1] = rise.cuda().half()[:, None]
    assert int(rise[-1]) < 2048
    out, _, _, status = call(cfg, q, k, v, [n], scale=math.log(2.0))
    assert status == 0
    see = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
    x = (rise.double().cuda()[None, :] * (math.log(2.0) * math.log2(math.e))).expand(n, n).masked_fill(~see, -math.inf)
    p = torch.softmax(x * math.log(2.0), 1)
    want, size = p @ v[:, 0].double(), p @ v[:, 0].double().abs()
    # weights and output rounded to fp16; an exponent of up to 30 in fp32; small weights to a multiple of 2^-24
    bound = (U16 + 64 * U32) * size + U16 * want.abs() + 2.0 ** -24
    top = p.amax(1, keepdim=True)
    bound += 2.0 ** -25 * top * (((p < 1.01 * 2.0 ** -14 * top) & see).double() @ v[:, 0].double().abs())
    for h in range(4):
        assert bool(((out[:, h].double() - want).abs() <= bound).all())


def hidden_keys(d, q0, k0):
    """Keys whose scores are q0 x k0, minus infinity or as good as that, weigh
    nothing; rows that see no other key are NaN."""
    cfg = config(1, 3, d, t=32)
    n = 300
    q, k, v = rows(cfg, n, 37)
    q[..., 0], k[..., 0] = q0, 0.0
    hidden = torch.zeros(n, dtype=torch.bool)
    hidden[:5] = True
    hidden[[40, 128, 129, 200]] = True
    kk = k[:, 0].double()
    k[hidden.cuda(), :, 0] = k0
    out, lse, mass, status = call(cfg, q, k, v, [n], 0)
    assert status == 0
    assert bool(torch.isnan(out[:5]).all())
    see = torch.ones((n, n), dtype=torch.bool, device="cuda").tril() & (~hidden).cuda()
    for h in range(3):
        qq = q[:, h].double()
        x = (qq @ kk.T * d ** -0.5).masked_fill(~see, -math.inf)[5:]
        p = torch.softmax(x, 1)
        size = (qq[:, 1:].abs() @ kk[:, 1:].abs().T * d ** -0.5).amax()
        eps = float(d * U32 * size + 16 * U32)
        want, absolute = p @ v[:, 0].double(), p @ v[:, 0].double().abs()
        bound = (U16 + 2 * eps) * absolute + U16 * want.abs() + n * 2.0 ** -25 * v.double().abs().amax() + 2.0 ** -24
        assert bool(((out[5:, h].double() - want).abs() <= bound).all())
        ref = torch.logsumexp(x, 1)
        assert bool(((lse[5:, h].double() - ref).abs() <= 2 * eps + 4 * U32 * ref.abs()).all())
    return cfg, q, k, v, out


@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_past_the_limit_count_as_infinite(d):
    cfg, q, k, v, want = hidden_keys(d, 32768.0, -32768.0)
    k[250, 0, 0] = 32768.0  # a score of 2^30 and more
    out = call(cfg, q, k, v, [300])[0]
    assert bool(torch.isnan(out[250:]).all()) and torch.equal(out[5:250], want[5:250])


# ------------------------------------------------------------------ long flat tails
@pytest.mark.parametrize("d,n,hkv", [(64, 1 << 20, 1), (128, 200000, 1), (256, 100000, 1), (128, 30000, 1),
                                     (64, 32768, 1), (128, 20000, 8)])
def test_a_long_flat_tail_keeps_its_weight(d, n, hkv):
    """One key far above all others, every other weight 2^-25.5 of its own.
    A weight rounded to fp16 is off by at most half a step, 2^-25 of 2^-b of
    the row's largest for the smallest ones, with b = ceil(log2 keys) - 13 >= 0:
    over all keys at most 2^-12 of the largest value's size."""
    cfg = config(hkv, 1, d)
    q, k, v = one_channel(cfg, n, 1.0, -17.6875, 36)
    k[0] = 0.0
    v.fill_(1.0)
    v[0] = 0.0
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.prompt_attention(cfg, q, k, v, out, cu, n, softmax_scale=1.0, dev_status=status)
    tail = torch.arange(n, device="cuda", dtype=torch.float64) * math.exp(-17.6875)
    want = (tail / (1.0 + tail))[:, None]
    # the weights' relative error, and the sums': n terms in fp32
    bound = 2.0 ** -12 + (2 * U16 + 64 * U32) * want + 2.0 ** -24
    assert int(status) == 0
    for h in range(hkv):
        assert bool(((out[:, h].double() - want).abs() <= bound).all()), float((out[:, h].double() - want).abs().max())


# ------------------------------------------------------------------ prefix sums that descend
@pytest.mark.parametrize("before", [0, 40, 1100])
def test_sequences_from_a_descent_on_are_skipped(before):
    """Prefix sums that go back and forth over the same rows: the sequences
    before the descent keep their results (masses too), those from it on are
    skipped, and the call reports it.  `before`: sequences of one token ahead."""
    cfg = config(8, 8)
    n = before + 1000
    q, k, v = rows(cfg, n, 38)
    good = [1] * before + [600, 400]
    want, want_lse, want_mass, status = call(cfg, q, k, v, good, 0)
    assert status == 0
    cu = list(np.concatenate([[0], np.cumsum(good)])) + [before, n, before + 500]
    for window in (0, 100):
        out, lse, mass, status = call(cfg, q, k, v, good, window, cu=cu, max_len=1000)
        assert status == kvq.KVQ_ERR_DEVICE_BOUNDS
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert bool((mass[len(good):] == 0).all())
        if window == 0:
            assert torch.equal(mass[:len(good), :want_mass.shape[1]], want_mass)
            assert bool((mass[:, want_mass.shape[1]:] == 0).all())
    out = call(cfg, q, k, v, [n], 0, cu=[n, 0, n], max_len=n)[0]  # nothing before the descent
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_score_of_minus_infinity_has_no_weight(d):
    cfg, q, k, v, want = hidden_keys(d, 2.0, -math.inf)
    k[250, 0, 0] = math.inf  # +inf: every row that sees it is NaN
    out = call(cfg, q, k, v, [300])[0]
    assert bool(torch.isnan(out[250:]).all()) and torch.equal(out[5:250], want[5:250])


# ------------------------------------------------------------------ the largest values
@pytest.mark.parametrize("n,hkv", [(150, 1), (700, 40)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_finite_values_give_finite_rows(d, n, hkv):
    """A mean of values up to fp16's largest stays in its range, however the
    weights are rounded (a weight may be up to 2^15 relative to the running
    maximum, and rounded by 2^-11 of it)."""
    cfg = config(hkv, 3, d)
    q, k, v = rows(cfg, n, 41, std=6.0)
    v.fill_(65504.0)
    v[:, :, 1::2] = -65504.0
    out, _, _, status = call(cfg, q, k, v, [n])
    assert status == 0
    want = v[:1].double().repeat_interleave(3, 1)
    assert bool(((out.double() - want).abs() <= (2 * U16 + n * U32) * 65504.0).all())
    # an infinite value is still infinite, from its token on
    v[70, :, 6] = math.inf
    v[90, :, 9] = -math.inf
    out, _, _, _ = call(cfg, q, k, v, [n])
    assert bool((out[70:, :, 6] == math.inf).logical_or(out[70:, :, 6].isnan()).all())
    assert bool((out[90:, :, 9] == -math.inf).logical_or(out[90:, :, 9].isnan()).all())
    assert bool(torch.isfinite(out[:70]).all())
