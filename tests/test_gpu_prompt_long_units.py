"""Units that take longer than the second that a wait for a step of a tile has: waits that may last for a whole unit have more.

152 heads of 256 rows over 115 M tokens, the same eight pages again and again: each SM works for more than a second on
one unit.  lse is that of the eight pages and the log of how often they come; its sum is off by 2^-24 for each of a
thread's additions (one for each 128 keys).  An output's fp32 sum has lost most digits at this length: it has to be an
average of the values."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_prompt import BF, F32, SCALE, i32

pytestmark = pytest.mark.gpu


def test_units_of_more_than_a_second(kv):
    assert kv.kvarn_device_error() == 0
    heads, P, times = 152, 128, 112500
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(256, heads, 128, generator=g, device="cuda").to(BF)
    kc, vc = (torch.randn(8, heads, P, 128, generator=g, device="cuda").to(BF) for _ in range(2))
    ws = torch.empty(kv.kvarn_prompt_attention_workspace_size(256, heads, heads), dtype=torch.uint8, device="cuda")
    lse = {}
    for n in (1, times):
        table = torch.arange(8, dtype=torch.int32, device="cuda").repeat(n)[None]
        out, lse[n] = torch.full_like(q, math.nan), torch.full((256, heads), math.nan, dtype=F32, device="cuda")
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        kv.kvarn_prompt_attention(q, kc, vc, table, i32([0, 256]), i32([8 * P * n]), out, SCALE, ws, causal=False, lse=lse[n])
        end.record()
        assert kv.kvarn_device_error() == 0
    assert begin.elapsed_time(end) > 1000, "the case has become too short"
    assert torch.isfinite(out).all() and out.abs().max() <= vc.abs().max()
    tol = (64 + 8 * times) * 2.0 ** -24 + 2.0 ** -16
    assert np.abs((lse[times] - lse[1] - math.log(times)).cpu().numpy()).max() <= tol
