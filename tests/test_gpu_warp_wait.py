"""A whole warp's bounded wait ends for all lanes together, although each lane has a limit of its own, and the device
stays usable (the self-check kernel; nothing hangs: the lane with the shortest limit ends the wait)."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_us", [1, 200, 20000])
def test_lanes_give_up_together(kv, limit_us):
    torch.cuda.synchronize()
    assert kv.kvarn_device_error() == 0
    t0 = time.perf_counter()
    kv.kvarn_check_bounded_wait(limit_us)
    with pytest.raises(kv.KvarnError) as e:
        kv.kvarn_device_error()
    elapsed = time.perf_counter() - t0
    assert e.value.status == kv.KVARN_ERR_TIMEOUT and e.value.code == 8
    assert 2e-6 * limit_us <= elapsed < 5.0  # the warp's wait and the thread's
    assert kv.kvarn_device_error() == 0
    assert int(torch.arange(100, device="cuda").sum()) == 4950
