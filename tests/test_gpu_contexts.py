"""The C calls in a second CUDA context of the device: what a launch needs set
up belongs to the context it runs in."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import ctypes
import numpy as np
from quantized_paged_kv_tile_b200 import build, kvq
build.build()
lib = kvq.load_library()
cu = ctypes.CDLL("libcuda.so.1")

def ok(r):
    assert r == 0, r

ok(cu.cuInit(0))
dev = ctypes.c_int()
ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
rng = np.random.default_rng(5)
heads, g, d, n, t = 2, 4, DIM, 200, 64
cfg = kvq.Config(num_kv_heads=heads, group_size=g, tile_tokens=t, bits_k=4, bits_v=4, iters=2, head_dim=d)
c = cfg.c()
lay = kvq.get_layout(cfg)
half = lambda *s: rng.standard_normal(s).astype(np.float16)
host = dict(q=half(n, heads * g, d), k=half(n, heads, d), v=half(n, heads, d), cu=np.array([0, n], np.int32),
            kt=half(1, heads, t, d), vt=half(1, heads, t, d), lens=np.array([37], np.int32),
            table=np.arange(8, dtype=np.int32), pool=np.zeros(8 * lay["block_stride_k"], np.uint8))

def run():
    '''A prompt and a decode step of the raw tail, in the current context.'''
    held = []

    def memory(size):
        p = ctypes.c_uint64()
        ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(max(size, 16))))
        held.append(p)
        return p.value

    def up(x):
        p = memory(x.nbytes)
        ok(cu.cuMemcpyHtoD_v2(ctypes.c_uint64(p), x.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(x.nbytes)))
        return p

    def down(p, like):
        x = np.empty_like(like)
        ok(cu.cuMemcpyDtoH_v2(x.ctypes.data_as(ctypes.c_void_p), ctypes.c_uint64(p), ctypes.c_size_t(x.nbytes)))
        return x

    b = {k: up(x) for k, x in host.items()}
    out, step, mass = up(np.zeros_like(host["q"])), up(np.zeros_like(host["q"][:1])), up(np.zeros(8, np.float32))
    status = up(np.zeros(4, np.int32))
    vp = ctypes.c_void_p
    need = ctypes.c_size_t()
    assert lib.kvq_prompt_workspace_bytes(ctypes.byref(c), 1, n, n, 0, ctypes.byref(need)) == 0
    assert lib.kvq_prompt_attention(ctypes.byref(c), b["q"], heads * g * d, b["k"], heads * d, b["v"], heads * d, out,
                                    None, b["cu"], 1, n, n, d ** -0.5, mass, 8, 0, memory(need.value), need.value,
                                    status, None) == 0, lib.kvq_last_error()
    assert lib.kvq_decode_mass_workspace_bytes(ctypes.byref(c), 1, 8, 0, ctypes.byref(need)) == 0
    ws = memory(need.value)
    assert lib.kvq_paged_decode_attention_mass(ctypes.byref(c), b["q"], step, mass, 8, b["lens"], 1, b["table"], 8, 8,
                                               b["pool"], b["pool"], b["kt"], b["vt"], d ** -0.5, ws, need.value, 0,
                                               status, None) == 0, lib.kvq_last_error()
    assert lib.kvq_paged_decode_attention(ctypes.byref(c), b["q"], step, b["lens"], 1, b["table"], 8, 8, b["pool"],
                                          b["pool"], b["kt"], b["vt"], d ** -0.5, ws, need.value, 0, status,
                                          None) == 0, lib.kvq_last_error()
    ok(cu.cuCtxSynchronize())
    res = [down(out, host["q"]), down(step, host["q"][:1]), down(mass, np.zeros(8, np.float32))]
    # the library's own scratch is this context's
    assert lib.kvq_paged_decode_attention_static_scratch(
        ctypes.byref(c), b["q"], step, b["lens"], 1, b["table"], 8, 8, b["pool"], b["pool"], b["kt"], b["vt"],
        2 * d ** -0.5, 0, status, None) == 0, lib.kvq_last_error()
    ok(cu.cuCtxSynchronize())
    res.append(down(step, host["q"][:1]))
    assert not np.array_equal(res[1], res[3])
    assert down(status, np.zeros(4, np.int32))[0] == 0
    for p in held:
        ok(cu.cuMemFree_v2(p))
    return res

ctx = ctypes.c_void_p()
ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(ctx), dev))
ok(cu.cuCtxSetCurrent(ctx))
want = run()
assert all(np.isfinite(x.astype(np.float32)).all() and x.any() for x in want)
for _ in range(2):  # contexts may come to lie where an earlier one was
    second = ctypes.c_void_p()
    ok(cu.cuCtxCreate_v2(ctypes.byref(second), 0, dev))
    got = run()
    assert all(np.array_equal(x, y) for x, y in zip(want, got))
    ok(cu.cuCtxSetCurrent(ctx))
    assert all(np.array_equal(x, y) for x, y in zip(want, run()))
    ok(cu.cuCtxSetCurrent(second))
    ok(cu.cuCtxDestroy_v2(second))
    ok(cu.cuCtxSetCurrent(ctx))
print("same")
"""


@pytest.mark.parametrize("d", [64, 128, 256])
def test_calls_in_a_second_context(d):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", PROGRAM.replace("DIM", str(d))], cwd=root, capture_output=True,
                         text=True, timeout=300)
    assert res.returncode == 0 and "same" in res.stdout, res.stdout + res.stderr
