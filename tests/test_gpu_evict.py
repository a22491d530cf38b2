"""Decode with tile masses, eviction, and a cache that runs them together.

Masses: a mass grows by the exact weights times (1 + e), e at most the relative
error of a score (its terms in fp32) and a few units of 2^-24, then summed in
fp32 over the query heads.  The rotated query and the hi/lo fp16 products of
the decode hold a score to about 2^-20 of the sum of its terms' magnitudes.
"""

import math

import numpy as np
import pytest
import torch

from quantized_paged_kv_tile_b200 import build, kvq
from quantized_paged_kv_tile_b200.paged import DecodeStepGraph, PagedKVCache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kvq.load_library()


def config(hkv=2, g=4, d=128, t=64, bits=(4, 4), seed=0):
    return kvq.Config(num_kv_heads=hkv, group_size=g, tile_tokens=t, bits_k=bits[0], bits_v=bits[1], iters=2,
                      head_dim=d, rotation_seed=seed)


def rows(cfg, n, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((n, h, cfg.head_dim), generator=gen, device="cuda").half()
            for h in (cfg.num_q_heads, cfg.num_kv_heads, cfg.num_kv_heads)]


def filled(cfg, lens, seed=1, track=True, extra=128, scatter=True):
    blocks = -(-(max(lens) + extra) // 16)
    table = None
    if scatter:
        table = np.random.default_rng(seed).permutation(len(lens) * blocks).astype(np.int32).reshape(len(lens), -1)
    cache = PagedKVCache(cfg, len(lens), blocks * 16, block_table=table, track_mass=track)
    _, k, v = rows(cfg, sum(lens), seed)
    if sum(lens):
        cache.prefill(k, v, lens)
    return cache


def cached_rows(cache, pool, tail, is_v, b, length):
    """The cache's own dequantized K or V of sequence b, fp64 [H_kv][length][d]."""
    cfg = cache.cfg
    t, full = cfg.tile_tokens, length // cfg.tile_tokens
    parts = []
    if full:
        desc = torch.tensor([[b, i] for i in range(full)], dtype=torch.int32, device="cuda")
        o = torch.empty((full, cfg.num_kv_heads, t, cfg.head_dim), dtype=torch.float32, device="cuda")
        kvq.unpack_tiles(cfg, desc, cache.block_tables, pool, is_v, out_orig=o, num_blocks=cache.num_blocks)
        parts.append(o.transpose(0, 1).reshape(cfg.num_kv_heads, full * t, cfg.head_dim).double())
    parts.append(tail[b, :, :length - full * t].double())
    return torch.cat(parts, 1)


def weights(cache, q):
    """Per sequence (weights [H_q][length], relative bound), from the cache's own pages in 64 bits."""
    cfg = cache.cfg
    res = []
    for b, n in enumerate(int(x) for x in cache.seq_lens.cpu()):
        kk = cached_rows(cache, cache.k_pool, cache.k_tail, False, b, n).repeat_interleave(cfg.group_size, 0)
        qq = q[b].double()[:, None]
        x = (qq @ kk.transpose(1, 2))[:, 0] * cfg.head_dim ** -0.5
        # the magnitudes of a score's terms sum to at most |q| |k| in the rotated domain
        size = qq[:, 0].norm(dim=1) * kk.norm(dim=2).amax(1) if n else torch.ones(1, device="cuda").double()
        res.append((torch.softmax(x, 1), float(2.0 ** -20 * size.max()) + 64 * 2.0 ** -24))
    return res


def mass_of(cache, q):
    t = cache.cfg.tile_tokens
    m = torch.zeros((cache.num_seqs, cache.max_tiles), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(m)
    for b, (p, eps) in enumerate(weights(cache, q)):
        w = p.sum(0)
        m[b].index_add_(0, torch.arange(w.numel(), device="cuda") // t, w)
        tol[b] = 2 * eps * m[b] + 1e-30
    return m, tol


def check_decode(cfg, lens, num_splits=0, seed=1):
    cache = filled(cfg, lens, seed)
    q = rows(cfg, len(lens), seed + 50)[0]
    start = torch.rand(cache.mass.shape, device="cuda")
    cache.mass.copy_(start)
    out = cache.decode(q, num_splits=num_splits)
    plain = torch.empty_like(q)
    kvq.paged_decode_attention(cfg, q, plain, cache.seq_lens, cache.block_tables, cache.k_pool, cache.v_pool,
                               cache.k_tail, cache.v_tail, cache.workspace if num_splits == 0 else torch.empty(
                                   kvq.decode_workspace_bytes(cfg, len(lens), num_splits), dtype=torch.uint8,
                                   device="cuda"), num_splits=num_splits, num_blocks=cache.num_blocks)
    assert cache.status() == 0
    assert torch.equal(out, plain)
    ref, tol = mass_of(cache, q)
    got = cache.mass.double() - start.double()
    # adding to what is there rounds once more
    err = (got - ref).abs() - 2.0 ** -24 * (cache.mass.double().abs() + start.double().abs())
    assert bool((err <= tol).all()), float((err / tol).max())
    untouched = ref == 0
    assert torch.equal(cache.mass[untouched], start[untouched])


@pytest.mark.parametrize("t", [32, 64, 128])
@pytest.mark.parametrize("bits", [(4, 4), (4, 2), (2, 2), (2, 4), (3, 3), (2, 3), (3, 2), (3, 4), (4, 3), (8, 8)])
def test_decode_mass_bits(t, bits):
    check_decode(config(t=t, bits=bits), [5 * t + 9, t, t - 1, 1])


@pytest.mark.parametrize("g", range(1, 9))
def test_decode_mass_groups(g):
    check_decode(config(hkv=3, g=g), [700, 64, 0, 3])


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("t", [32, 64, 128])
def test_decode_mass_other_head_sizes(d, t):
    check_decode(config(d=d, t=t, g=3), [5 * t + 9, t, 0, 7])


@pytest.mark.parametrize("num_splits", [1, 3, 40])
def test_decode_mass_splits(num_splits):
    check_decode(config(), [4000, 64, 130], num_splits=num_splits)


def test_decode_mass_many_heads_and_tiles():
    check_decode(config(hkv=8, g=8, t=32, bits=(4, 2)), [20000, 100])
    check_decode(config(hkv=1, g=1, seed=7), [9000])


def test_decode_mass_bad_page_and_long_length():
    cfg = config()
    cache = filled(cfg, [300, 300])
    q = rows(cfg, 2, 3)[0]
    cache.decode(q)
    good = cache.mass.clone()
    cache.mass.zero_()
    cache.block_tables[0, 5] = cache.num_blocks + 3  # a page of tile 1 of sequence 0
    cache.decode(q)
    assert cache.status() == kvq.KVQ_ERR_DEVICE_BOUNDS
    assert torch.equal(cache.mass[1], good[1])
    assert float(cache.mass[0, 1]) == 0.0  # the skipped tile has no weight
    assert abs(float(cache.mass[0].sum()) - cfg.num_q_heads) < 1e-4
    cache.dev_status.zero_()
    cache.seq_lens[0] = 100000  # past the table
    cache.mass.zero_()
    cache.decode(q)
    assert cache.status() == kvq.KVQ_ERR_DEVICE_BOUNDS
    assert torch.equal(cache.mass[1], good[1])


# ------------------------------------------------------------------ eviction
def evict_definition(mass, lens, table, t, keep, sink, recent):
    mass, lens, table = mass.copy(), lens.copy(), table.copy()
    ppt = t // 16
    kept = np.full(mass.shape, -1, dtype=np.int32)
    for b in range(len(lens)):
        n = max(0, int(lens[b])) // t
        e = max(0, n - keep)
        key = [(1, 0.0) if math.isnan(x) else (0, x) for x in mass[b]]
        leave = set(sorted(range(sink, n - recent), key=lambda i: (key[i], i))[:e])
        stay = [i for i in range(n) if i not in leave]
        kept[b, :len(stay)] = stay
        if e:
            perm = stay + sorted(leave)
            table[b, :n * ppt] = table[b, :n * ppt].reshape(n, ppt)[perm].reshape(-1)
            tail = mass[b, n] if n < mass.shape[1] else np.float32(0)
            row = np.zeros_like(mass[b])
            row[:len(stay)] = mass[b, stay]
            if len(stay) < len(row):
                row[len(stay)] = tail
            mass[b] = row
            lens[b] -= e * t
    return mass, lens, table, kept


def check_evict(lens, tiles, t, keep, sink=0, recent=0, seed=0, masses=None, extra_blocks=0, with_kept=True):
    cfg = config(t=t)
    rng = np.random.default_rng(seed)
    b, blocks = len(lens), tiles * (t // 16) + extra_blocks
    mass = rng.exponential(1.0, (b, tiles)).astype(np.float32)
    if masses is not None:
        mass = rng.choice(np.asarray(masses, dtype=np.float32), (b, tiles))
    table = rng.permutation(b * blocks).astype(np.int32).reshape(b, blocks)
    lens = np.asarray(lens, dtype=np.int32)
    dev = [torch.from_numpy(x.copy()).cuda() for x in (mass, lens, table)]
    kept = torch.full((b, tiles), 77, dtype=torch.int32, device="cuda") if with_kept else None
    ws = torch.full((kvq.evict_workspace_bytes(cfg, b, blocks),), 255, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.evict_tiles(cfg, dev[0], dev[1], dev[2], keep, sink, recent, kept=kept, workspace=ws, dev_status=status)
    want = evict_definition(mass, lens, table, t, keep, sink, recent)
    assert int(status) == 0
    for got, ref in zip(dev + [kept], want):
        if got is not None:
            np.testing.assert_array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("t", [32, 64, 128])
@pytest.mark.parametrize("keep,sink,recent", [(0, 0, 0), (1, 0, 1), (1, 1, 0), (5, 2, 3), (9, 1, 1), (40, 4, 8)])
def test_evict(t, keep, sink, recent):
    lens = [0, 1, t - 1, t, t + 1, 5 * t, 6 * t + 3, 39 * t, 40 * t, 41 * t + 7, 47 * t]
    check_evict(lens, 48, t, keep, sink, recent, with_kept=keep != 1)


@pytest.mark.parametrize("masses", [[0.0], [1.0, 1.0, 2.0], [0.0, -0.0, 1e-40, 3.0], [math.nan, 1.0, math.inf],
                                    [math.nan], [-1.0, -math.inf, 0.5, -1e-30]], ids=str)
def test_evict_equal_and_special_masses(masses):
    check_evict([64 * 50, 64 * 33 + 5, 64 * 7], 51, 64, 10, 2, 2, masses=masses)


def test_evict_long_rows_and_odd_tables():
    check_evict([32 * 5000 + 1, 32 * 2049, 32 * 1024, 32 * 1023], 5001, 32, 1000, 4, 16, extra_blocks=1)
    check_evict([128 * 3000], 3000, 128, 2999, extra_blocks=7)  # the tail's entry lies past the row
    check_evict([int(x) for x in np.random.default_rng(5).integers(0, 64 * 300, 300)], 301, 64, 37, 1, 1)


def test_evict_twice_changes_nothing_more():
    cfg = config()
    cache = filled(cfg, [1000, 200], extra=64)
    cache.mass.copy_(torch.rand(cache.mass.shape, device="cuda"))
    cache.evict(5)
    state = [x.clone() for x in (cache.mass, cache.seq_lens, cache.block_tables)]
    cache.evict(5)
    assert all(torch.equal(x, y) for x, y in zip(state, (cache.mass, cache.seq_lens, cache.block_tables)))
    assert list(cache.host_lens) == [5 * 64 + 1000 % 64, 200] == cache.seq_lens.tolist()


def test_evict_length_past_the_table_is_left_alone():
    cfg = config()
    cache = filled(cfg, [400, 400])
    cache.mass.copy_(torch.rand(cache.mass.shape, device="cuda"))
    cache.seq_lens[0] = 1 << 20
    before = [x[0].clone() for x in (cache.mass, cache.seq_lens, cache.block_tables)]
    cache.evict(2)
    assert cache.status() == kvq.KVQ_ERR_DEVICE_BOUNDS
    assert all(torch.equal(x, y[0]) for x, y in zip(before, (cache.mass, cache.seq_lens, cache.block_tables)))
    assert int(cache.seq_lens[1]) == 2 * 64 + 400 % 64


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("d,t", [(128, 64), (128, 32), (64, 64), (256, 128)])
def test_prompt_decode_evict_append(d, t):
    """A serving run: prompts, decode steps, eviction, more steps that fill new
    tiles into the evicted blocks, eviction again.  Against a plain cache of
    dequantized tiles on the side."""
    cfg = config(d=d, t=t, g=4)
    lens = [6 * t + 5, 3 * t, 2]
    blocks = -(-(max(lens) + 2 * t) // 16) // (t // 16) * (t // 16)
    cache = PagedKVCache(cfg, 3, blocks * 16, track_mass=True)
    q, k, v = rows(cfg, sum(lens), 21)
    out = cache.prompt(q, k, v, lens)
    assert cache.status() == 0
    at = 0
    for b, n in enumerate(lens):  # every prompt row adds one per query head
        assert abs(float(cache.mass[b].double().sum()) / (n * cfg.num_q_heads) - 1) < 1e-5
        x = (q[at:at + n, 0].double() @ k[at:at + n, 0].double().T * d ** -0.5)
        x = x.masked_fill(torch.ones_like(x).triu(1).bool(), -math.inf).softmax(1) @ v[at:at + n, 0].double()
        assert float((out[at:at + n, 0].double() - x).norm() / x.norm()) < 1e-3
        at += n

    def side(b):
        n = int(cache.seq_lens[b])
        return [cached_rows(cache, cache.k_pool, cache.k_tail, False, b, n),
                cached_rows(cache, cache.v_pool, cache.v_tail, True, b, n)]

    for step in range(3):
        before = [side(b) for b in range(3)]
        masses, kept = cache.mass.clone(), torch.empty_like(cache.mass, dtype=torch.int32)
        lens_before = cache.seq_lens.tolist()
        cache.evict(4 - step, kept=kept)
        for b in range(3):
            n = lens_before[b]
            stay = [i for i in kept[b].tolist() if i >= 0]
            full = n // t
            assert len(stay) == min(full, 4 - step)
            assert stay == sorted(stay) and (not stay or stay[0] == 0) and (not full or stay[-1] == full - 1)
            for x, y in zip(before[b], side(b)):
                want = torch.cat([x[:, i * t:(i + 1) * t] for i in stay] + [x[:, full * t:]], 1)
                assert torch.equal(want, y)
            assert torch.equal(cache.mass[b, :len(stay)], masses[b, stay])
        for i in range(t + 3):  # every sequence completes a tile
            qs, ks, vs = rows(cfg, 3, 1000 * step + i)
            cache.append(ks, vs)
            if i % 16 == 0:
                start = cache.mass.clone()
                cache.decode(qs)
                ref, tol = mass_of(cache, qs)
                err = (cache.mass.double() - start.double() - ref).abs() - 2.0 ** -23 * cache.mass.double().abs()
                assert bool((err <= tol).all())
        assert cache.status() == 0 and cache.seq_lens.tolist() == list(cache.host_lens)


def test_step_graph_tracks_masses_and_survives_eviction():
    cfg = config()
    a, b = filled(cfg, [700, 130], 31, extra=512), filled(cfg, [700, 130], 31, extra=512)
    graph = DecodeStepGraph(a)
    assert float(a.mass.abs().sum()) == 0.0  # capture leaves the masses alone
    for i in range(40):
        q, k, v = rows(cfg, 2, 400 + i)
        graph.new_k.copy_(k)
        graph.new_v.copy_(v)
        graph.q.copy_(q)
        out = graph.replay()
        b.append(k, v)
        want = b.decode(q)
        assert torch.equal(out, want) and torch.equal(a.mass, b.mass)
        if i % 13 == 12:
            a.evict(6 - i // 13)
            b.evict(6 - i // 13)
            assert torch.equal(a.block_tables, b.block_tables) and torch.equal(a.seq_lens, b.seq_lens)
    assert a.status() == 0
    with pytest.raises(ValueError):
        DecodeStepGraph(a, fused=True)


def test_evict_and_decode_captured_on_another_stream():
    cfg = config()
    cache = filled(cfg, [900, 640], 41)
    q = rows(cfg, 2, 42)[0]
    ref = filled(cfg, [900, 640], 41)
    want = ref.decode(q)
    ref.evict(4)
    want2 = ref.decode(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cache.decode(q, stream=side)
    cache.evict(4, stream=side)
    got2 = cache.decode(q, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want2) and torch.equal(cache.mass, ref.mass)


def test_counts_past_32_bits_and_small_buffers_are_refused():
    cfg = config()
    cache = filled(cfg, [300, 100], 55)
    before = [x.clone() for x in (cache.mass, cache.seq_lens, cache.block_tables)]
    for keep in (2 ** 32, 2 ** 63 - 1):
        with pytest.raises(ValueError, match="keep_tiles"):
            cache.evict(keep, 0, 0)
    with pytest.raises(ValueError, match="sink_tiles"):
        cache.evict(2, 2 ** 32, 0)
    q = rows(cfg, 2, 56)[0]
    args = [cfg, q, torch.empty_like(q), cache.mass, cache.seq_lens, cache.block_tables, cache.k_pool, cache.v_pool,
            cache.k_tail, cache.v_tail, cache.workspace]
    for at, small in ((6, cache.k_pool[:-1]), (7, cache.v_pool[:-1]), (8, cache.k_tail[:1]), (9, cache.v_tail[:, :1])):
        with pytest.raises(ValueError):
            kvq.paged_decode_attention_mass(*args[:at], small, *args[at + 1:], num_blocks=cache.num_blocks)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, (cache.mass, cache.seq_lens, cache.block_tables)))


@pytest.mark.parametrize("lens", [[0, 0], [5, 0], [0, 64]], ids=str)
def test_prompts_without_tokens_or_tiles(lens):
    cfg = config()
    cache = PagedKVCache(cfg, 2, 256, track_mass=True)
    q, k, v = rows(cfg, sum(lens), 51)
    out = cache.prompt(q, k, v, lens)
    torch.cuda.synchronize()
    assert cache.status() == 0 and cache.seq_lens.tolist() == lens and out.shape == q.shape
    for b, n in enumerate(lens):
        assert abs(float(cache.mass[b].sum()) - n * cfg.num_q_heads) < 1e-3
    qs, ks, vs = rows(cfg, 2, 52)
    cache.append(ks, vs)
    cache.decode(qs)
    cache.evict(2, 0, 0)
    assert cache.status() == 0 and cache.seq_lens.tolist() == [n + 1 for n in lens]


def test_calls_of_another_shape_or_device_are_refused(monkeypatch):
    cfg = config()
    cache = filled(cfg, [100, 100], 53)
    q = rows(cfg, 2, 54)[0]
    with pytest.raises(ValueError, match="shape"):
        cache.decode(q[:1].contiguous())
    with pytest.raises(kvq.KvqError):
        cache.evict(1, 1, 1)  # keeps fewer than it protects
    assert list(cache.host_lens) == [100, 100]
    with pytest.raises(RuntimeError, match="empty"):
        cache.prompt(q, q, q, [1, 1])
    with pytest.raises(ValueError):
        filled(cfg, [100], track=False).evict(1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        cache.evict(5)


FIRST_CALL_IN_A_CAPTURE = """
import torch
from quantized_paged_kv_tile_b200 import kvq
from quantized_paged_kv_tile_b200.paged import PagedKVCache
cfg = kvq.Config(num_kv_heads=2, group_size=4, tile_tokens=64, bits_k=4, bits_v=4, iters=2)
cache = PagedKVCache(cfg, 2, 1024, track_mass=True)
gen = torch.Generator(device="cuda").manual_seed(1)
q, k, v = (torch.randn((1400, h, 128), generator=gen, device="cuda").half() for h in (8, 2, 2))
cache.prefill(k, v, [700, 700])
cu = torch.tensor([0, 700, 1400], dtype=torch.int32, device="cuda")
out, step = torch.zeros_like(q), torch.zeros_like(q[:2])
ws = torch.empty(kvq.prompt_workspace_bytes(cfg, 2, 1400, 700), dtype=torch.uint8, device="cuda")
ews = torch.empty(kvq.evict_workspace_bytes(cfg, 2, 64), dtype=torch.uint8, device="cuda")
mass = torch.zeros((2, 11), device="cuda")
args = (cache.block_tables, cache.k_pool, cache.v_pool, cache.k_tail, cache.v_tail, cache.workspace)

def run():
    kvq.prompt_attention(cfg, q, k, v, out, cu, 700, mass=mass, workspace=ws)
    kvq.paged_decode_attention_mass(cfg, q[:2], step, cache.mass, cache.seq_lens, *args)
    kvq.evict_tiles(cfg, cache.mass, cache.seq_lens, cache.block_tables, 4, workspace=ews)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (out, step, mass, cache.seq_lens, cache.block_tables)]
again = PagedKVCache(cfg, 2, 1024, track_mass=True)
again.prefill(k, v, [700, 700])
cache = again
args = (cache.block_tables, cache.k_pool, cache.v_pool, cache.k_tail, cache.v_tail, cache.workspace)
mass.zero_()
run()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, (out, step, mass, cache.seq_lens, cache.block_tables)))
assert got[3].tolist() == [4 * 64 + 700 % 64] * 2
print("same")
"""


def test_the_first_calls_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0 and "same" in res.stdout, res.stdout + res.stderr
