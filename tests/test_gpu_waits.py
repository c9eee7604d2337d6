"""Every bounded wait of the kernels ends at its limit of about 2 s: the self-test reports a timeout
only when all of them have given up, and is done soon after."""
import time

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def test_every_wait_gives_up_at_its_limit():
    import sparse_attention_long_04_b200 as dsa
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert dsa.dsa_selftest_wait_timeout(status) == dsa.DSA_OK
    assert dsa.dsa_read_device_status(status) == (dsa.DSA_ERR_TIMEOUT, dsa.DSA_DEVICE_TIMEOUT)
    assert 1.0 < time.perf_counter() - t0 < 5.0
    # several at once, on streams of their own, take no longer
    words = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in words]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for w, s in zip(words, streams):
        assert dsa.dsa_selftest_wait_timeout(w, s) == dsa.DSA_OK
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert all(int(w.item()) == dsa.DSA_DEVICE_TIMEOUT for w in words)
