"""Integers past 32 bits reach no call of the prompt, mass and eviction operators (ctypes would wrap them)."""

import pytest
import torch

from quantized_paged_kv_tile_b200 import build, kvq

CFG = kvq.Config(num_kv_heads=2, group_size=4, tile_tokens=64, bits_k=4, bits_v=4, iters=4)
LARGE = [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, -2 ** 31 - 1, -2 ** 32 + 1]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kvq.load_library()


@pytest.mark.parametrize("bad", LARGE)
@pytest.mark.parametrize("call,good", [(kvq.prompt_workspace_bytes, (1, 10, 10, 0)),
                                       (kvq.decode_mass_workspace_bytes, (1, 8, 1)),
                                       (kvq.evict_workspace_bytes, (1, 8))], ids=lambda x: getattr(x, "__name__", ""))
def test_size_queries(call, good, bad):
    for at in range(len(good)):
        with pytest.raises(ValueError, match="32 bits"):
            call(CFG, *good[:at], bad, *good[at + 1:])


@pytest.mark.parametrize("bad", LARGE)
@pytest.mark.parametrize("name", ["num_splits", "num_blocks"])
def test_decode_with_masses(name, bad):
    q = torch.zeros((1, 8, 128), dtype=torch.float16)
    tail = torch.zeros((1, 2, 64, 128), dtype=torch.float16)
    pool = torch.zeros((8, 2, 1152), dtype=torch.uint8)
    with pytest.raises(ValueError, match=f"{name}.*32 bits"):
        kvq.paged_decode_attention_mass(CFG, q, q, torch.zeros((1, 2)), torch.zeros(1, dtype=torch.int32),
                                        torch.zeros((1, 8), dtype=torch.int32), pool, pool, tail, tail,
                                        torch.zeros(1024, dtype=torch.uint8), **{name: bad})


@pytest.mark.parametrize("bad", LARGE)
@pytest.mark.parametrize("name", ["keep_tiles", "sink_tiles", "recent_tiles"])
def test_eviction(name, bad):
    args = {"keep_tiles": 4, "sink_tiles": 1, "recent_tiles": 1, name: bad}
    with pytest.raises(ValueError, match=f"{name}.*32 bits"):
        kvq.evict_tiles(CFG, torch.zeros((1, 2)), torch.zeros(1, dtype=torch.int32),
                        torch.zeros((1, 8), dtype=torch.int32), **args)


@pytest.mark.parametrize("bad", LARGE)
@pytest.mark.parametrize("name", ["max_seq_tokens", "mass_window"])
def test_prompt(name, bad):
    q = torch.zeros((4, 8, 128), dtype=torch.float16)
    k = torch.zeros((4, 2, 128), dtype=torch.float16)
    args = {"max_seq_tokens": 4, "mass_window": 0, name: bad}
    with pytest.raises(ValueError, match=f"{name}.*32 bits"):
        kvq.prompt_attention(CFG, q, k, k, q, torch.zeros(2, dtype=torch.int32), **args)
