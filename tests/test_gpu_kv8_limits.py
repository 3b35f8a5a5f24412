"""GPU tests of the 8-bit paged KV cache at the limits of its arguments
(include/apr_kv8.h): what the device arrays may say, sizes left to their
defaults, several host threads, places past 2^32 bytes.

Values are compared with the float64 oracle as tests/test_gpu_kv8.py derives it.
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv8 import Case, as_f32, assert_attention, assert_weights, attend, bad_index, starts

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- lengths out of range
@pytest.mark.parametrize("row_start", [True, False])
@pytest.mark.parametrize("length", [129, 130, 1 << 30, -1])
def test_a_length_out_of_range_leaves_its_sequence_alone(q, length, row_start):
    # the table holds 128 tokens; the rows of the other sequence are appended all the same
    c = Case([128, 70], 2, 64, 32, seed=50, extra_width=0).on_gpu(q)
    c.glens[0] = length
    rows = [3, 2] if row_start else [1, 1]
    k, v = (torch.from_numpy(100 * c.rng.normal(size=(sum(rows), 2 * 64)).astype(np.float32)).cuda() for _ in range(2))
    q.apr_kv8_append(c.cache, c.gtable, c.glens, k, v,
                     row_start=torch.from_numpy(starts(rows)).cuda() if row_start else None)
    bad_index(q)
    want = oracle.kv8_append(c.host, c.table, [0, 70], starts(rows), as_f32(k), as_f32(v))
    c.assert_cache(want)


def test_a_length_past_max_len_is_not_evicted_and_receives_no_weight(q):
    c = Case([100, 90], 1, 64, 32, seed=51, spare=2).on_gpu(q)
    fresh = torch.from_numpy(np.array(c.free[:2], np.int32).reshape(2, 1)).cuda()
    w = torch.rand((2, 1, 128), device="cuda")
    q.apr_kv8_evict(c.cache, c.gtable, c.glens, w, 30, 10, fresh, torch.empty_like(c.gtable), torch.empty_like(c.glens),
                    torch.empty((2, 1, 30), device="cuda"), torch.empty((2, 1, 30), dtype=torch.int32, device="cuda"), max_len=95)
    bad_index(q)
    before = {name: a.copy() for name, a in c.host.items()}
    want, *_ = oracle.kv8_evict(before, c.table, [0, 90], w.cpu().numpy(), 30, 10, fresh.cpu().numpy())
    c.assert_cache(want)
    total = w.clone()
    x = torch.randn((2, 2 * 64), device="cuda")
    q.apr_kv8_attention(c.cache, c.gtable, c.glens, x, torch.empty_like(x), 2, weights=total, accumulate=True, max_len=95)
    bad_index(q)
    assert torch.equal(total[0], w[0]) and bool((total[1, :, :89] >= w[1, :, :89]).all())
    np.testing.assert_allclose(float(total[1, 0, :89].sum() - w[1, 0, :89].sum() + total[1, 0, 89]), 2.0, rtol=1e-4)
