"""Host-side checks of the prompt attention call: what it refuses before any launch."""

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


def prompt(lib, c=None, q=16, qs=1024, k=16, ks=256, v=16, vs=256, out=16, lse=None, cu=16, b=1, n=10, top=10,
           scale=0.1, mass=None, tiles=0, window=0, ws=None, ws_bytes=0):
    return lib.kvq_prompt_attention(ctypes.byref((c or cfg()).c()), q, qs, k, ks, v, vs, out, lse, cu, b, n, top,
                                    scale, mass, tiles, window, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu=None), dict(q=24), dict(lse=8),
    dict(qs=1016), dict(ks=248), dict(vs=260), dict(qs=1028), dict(b=-1), dict(n=-1), dict(top=-1), dict(b=65536),
    dict(top=(1 << 20) + 1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(window=5), dict(window=-1), dict(mass=16, tiles=0), dict(mass=16, tiles=1, top=65, n=65),
    dict(mass=16, tiles=1, ws=None), dict(n=2 ** 31 - 1, top=1, b=65535, c=cfg(num_kv_heads=4096)),
], ids=str)
def test_refused(lib, kw):
    assert prompt(lib, **kw) == kvq.KVQ_ERR_INVALID_ARG
    assert kvq.load_library().kvq_last_error()


def test_refused_configurations(lib):
    assert prompt(lib, cfg(head_dim=96)) == kvq.KVQ_ERR_UNSUPPORTED
    assert prompt(lib, cfg(group_size=9)) == kvq.KVQ_ERR_UNSUPPORTED


def test_nothing_to_do(lib):
    # no sequence, no row or no length: no pointer is looked at
    for kw in (dict(b=0), dict(n=0), dict(top=0)):
        assert prompt(lib, q=None, k=None, v=None, out=None, cu=None, **kw) == kvq.KVQ_OK


def test_workspace_bytes_arguments(lib):
    need = ctypes.c_size_t(0)
    c = cfg().c()
    assert lib.kvq_prompt_workspace_bytes(ctypes.byref(c), 1, 10, 10, 0, None) == kvq.KVQ_ERR_INVALID_ARG
    for bad in ((-1, 10, 10, 0), (1, -1, 10, 0), (1, 10, -1, 0), (1, 10, 10, -1), (1, 10, (1 << 20) + 1, 0)):
        assert lib.kvq_prompt_workspace_bytes(ctypes.byref(c), *bad, ctypes.byref(need)) == kvq.KVQ_ERR_INVALID_ARG


def test_binding_checks_tensors():
    import torch
    x = torch.zeros((4, 8, 128), dtype=torch.float16)
    with pytest.raises(TypeError, match="CUDA"):
        kvq.prompt_attention(cfg(), x, x, x, x, torch.zeros(2, dtype=torch.int32), 4)
