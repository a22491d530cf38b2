"""Host-side checks of the decode with masses and of the eviction: what they refuse before any launch."""

import ctypes

import pytest

from quantized_paged_kv_tile_b200 import build, kvq


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kvq.load_library()


def cfg(**kw):
    base = dict(num_kv_heads=2, group_size=4, tile_tokens=64, bits_k=4, bits_v=4, iters=4)
    return kvq.Config(**{**base, **kw})


def evict(lib, c=None, mass=16, tiles=8, keep=4, sink=1, recent=1, lens=16, b=1, table=16, blocks=32, kept=None,
          ws=16, ws_bytes=1 << 20):
    return lib.kvq_evict_tiles(ctypes.byref((c or cfg()).c()), mass, tiles, keep, sink, recent, lens, b, table,
                               blocks, kept, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw", [
    dict(mass=None), dict(lens=None), dict(table=None), dict(ws=None), dict(mass=20), dict(kept=8), dict(tiles=0),
    dict(keep=-1, sink=0, recent=0), dict(sink=-1), dict(recent=-1), dict(keep=1), dict(sink=5), dict(recent=4),
    dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1, keep=2 ** 31 - 1), dict(b=-1), dict(b=65536), dict(blocks=0),
], ids=str)
def test_evict_refused(lib, kw):
    assert evict(lib, **kw) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_last_error()


def test_evict_workspace(lib):
    need = kvq.evict_workspace_bytes(cfg(), 3, 32)
    assert need >= 3 * (32 + 2 * 8) * 4
    assert evict(lib, b=3, ws_bytes=need - 1) == kvq.KVQ_ERR_WORKSPACE
    assert evict(lib, b=0, mass=None, lens=None, table=None, ws=None) == kvq.KVQ_OK
    out = ctypes.c_size_t(0)
    c = cfg().c()
    assert lib.kvq_evict_workspace_bytes(ctypes.byref(c), -1, 4, ctypes.byref(out)) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_evict_workspace_bytes(ctypes.byref(c), 1, 0, ctypes.byref(out)) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_evict_workspace_bytes(ctypes.byref(c), 1, 4, None) == kvq.KVQ_ERR_INVALID_ARG


def decode(lib, mass=16, tiles=2, q=16, out=16, b=2, blocks=8, splits=1, scale=0.1, ws=16, ws_bytes=0, c=None):
    return lib.kvq_paged_decode_attention_mass(ctypes.byref((c or cfg()).c()), q, out, mass, tiles, 16, b, 16, blocks,
                                               8, 16, 16, 16, 16, scale, ws, ws_bytes, splits, None, None)


@pytest.mark.parametrize("kw", [
    dict(mass=None), dict(mass=20), dict(tiles=1), dict(tiles=2, blocks=9), dict(q=None), dict(out=None), dict(b=-1),
    dict(b=65536), dict(splits=-1), dict(splits=65536), dict(scale=0.0), dict(ws=None),
], ids=str)
def test_decode_mass_refused(lib, kw):
    assert decode(lib, **kw) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_last_error()


def test_decode_mass_arguments_that_need_no_device(lib):
    assert decode(lib, b=0, q=None, out=None, mass=None, ws=None) == kvq.KVQ_OK
    out = ctypes.c_size_t(0)
    c = cfg().c()
    for bad in ((-1, 8, 1), (1, 0, 1), (1, 8, -1)):
        assert lib.kvq_decode_mass_workspace_bytes(ctypes.byref(c), *bad, ctypes.byref(out)) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_decode_mass_workspace_bytes(ctypes.byref(c), 1, 8, 1, None) == kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [2 ** 31, 2 ** 32, 2 ** 63 - 1, -2 ** 31 - 1])
def test_integers_are_not_wrapped(bad):
    with pytest.raises(ValueError, match="keep_tiles"):
        kvq._int(bad, "keep_tiles")
    with pytest.raises(TypeError):
        kvq._int(1.5, "keep_tiles")
    assert kvq._int(2 ** 31 - 1, "keep_tiles") == 2 ** 31 - 1
