"""Every wait of the bounded-wait self-test runs out: they run one after
another on one stream, so the call takes the sum of their limits."""

import time

import pytest
import torch

from quantized_paged_kv_tile_b200 import build, kvq

pytestmark = pytest.mark.gpu


def test_each_of_the_four_waits_runs_its_limit():
    build.build()
    kvq.load_library()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.monotonic()
    kvq.selftest_bounded_wait(status)
    torch.cuda.synchronize()
    elapsed = time.monotonic() - t0
    assert int(status.item()) == kvq.KVQ_ERR_DEVICE_TIMEOUT
    # quantize, decode, prefill and prompt kernels, 2 s each: three give 6 s
    assert 7.5 < elapsed < 40.0
