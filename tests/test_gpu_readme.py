"""The README's serving step, as it stands there."""
import math
import os
import re
import types

import numpy as np
import pytest
import torch

from oracle import serving as o
from tests.test_gpu_serving import BF, i32, np64

pytestmark = pytest.mark.gpu


def test_the_serving_example_runs_and_carries_the_rotation_scale(kv):
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        code = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "kvarn_step_tables" in b)
    # the example's frequencies scaled for a longer context, as its caller would change them: their scale is not 1
    yarn = dict(scaling=kv.KVARN_ROPE_YARN, factor=16.0, original_len=4096.0, low=1.0, high=32.0)
    lib = types.SimpleNamespace(**{n: getattr(kv, n) for n in dir(kv) if n.startswith("kvarn_")})
    lib.kvarn_rope_frequencies = lambda rot, base: kv.kvarn_rope_frequencies(rot, base, **yarn)
    B, Hq, Hkv, T, page_size = 1, 4, 2, 21, 16
    g = torch.Generator(device="cuda").manual_seed(70)
    rows = torch.randn(T, Hq + 2 * Hkv, 128, generator=g, device="cuda").to(BF)
    q_out = torch.empty(T, Hq, 128, dtype=BF, device="cuda")
    k_cache, v_cache = (torch.zeros(4, Hkv, page_size, 128, dtype=BF, device="cuda") for _ in range(2))
    names = dict(kv=lib, torch=torch, B=B, Hq=Hq, Hkv=Hkv, page_size=page_size, lens=i32([0]), n_new=i32([T]), counts=i32([0]),
                 page_table=i32([[-1] * 4]), free_pages=i32([3, 1, 0, 2]), n_free=i32([4]), cu_tokens=i32([0, 0]),
                 positions=i32([0] * T), slots=i32([0] * T), status=i32([-1]), q=rows[:, :Hq], k=rows[:, Hq:Hq + Hkv],
                 v=rows[:, Hq + Hkv:], q_out=q_out, q_last=q_out[T - 1:], k_cache=k_cache, v_cache=v_cache,
                 qw=torch.full((128,), 1.5, device="cuda"), kw=torch.full((128,), 0.5, device="cuda"),
                 out=torch.empty(B, Hq, 128, device="cuda"))
    exec(compile(code, "README.md", "exec"), names)
    assert int(names["status"]) == 0 and names["lens"].tolist() == [T] and kv.kvarn_device_error() == 0
    freqs, scale = kv.kvarn_rope_frequencies(128, 1e6, **yarn)
    assert abs(scale - (0.1 * math.log(16.0) + 1)) < 1e-6
    want = o.norm_rotate(np64(rows[:, :Hq]), np.arange(T), freqs.numpy(), np64(names["qw"]), 1e-6, scale)
    # one rounding to bf16 (2^-8 of the value), beside fp32 errors of the pair that 2^-16 of its size covers
    assert np.all(np.abs(np64(q_out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * np.abs(want).max())
    want = o.paged_attention(np64(q_out[T - 1:]), np64(k_cache), np64(v_cache), names["page_table"].cpu().numpy(), [T],
                             1 / math.sqrt(128))[0]
    # fp32 throughout on identical inputs: scores of some tens, each off by a few 2^-24 of itself
    assert np.all(np.abs(np64(names["out"]) - want) <= 1e-4)
