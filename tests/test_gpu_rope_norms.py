"""GPU parity of the norm of heads (include/apr_rope.h) over the whole range of magnitudes and of eps, and of the table over that of
its scale, against their oracle.

r = f32(1 / sqrt(mean of x^2 + eps)) is taken to more than 40 bits before its rounding at every magnitude, so a result is the oracle's
but for one head in 2^16 or so: assert_rows of tests/test_gpu_rope.py, with the 3 heads that it allows.
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv8 import TYPES, as_f32, rows_tensor, starts
from test_gpu_rope import assert_rows, ints, table_of

pytestmark = pytest.mark.gpu

# (a head's values are normal numbers times one of these: float32's smallest ones, where squares, their residuals or sums leave
# float32, and the largest)
SIZES = [1e-38, 1e-30, 1e-22, 3e-20, 2.0 ** -63, 2.0 ** -52, 2.0 ** -50, 2.0 ** -48, 1e-9, 1.0, 2.0 ** 48, 2.0 ** 50, 2.0 ** 52, 2.0 ** 58,
         2.0 ** 60, 2.0 ** 62, 2.0 ** 64, 2.0 ** 90, 2.0 ** 120, 2.0 ** 124]


def heads_of(dim, type_, rng):
    """Two rows of a head of each size and of one of equal values of each size, in no order, as float32 values of the type."""
    x = np.concatenate([rng.normal(size=(len(SIZES), dim)), np.ones((len(SIZES), dim))]) * np.tile(SIZES, 2)[:, None]
    x = np.stack([x[rng.permutation(len(x))] for _ in range(2)]).reshape(2, -1)
    return as_f32(torch.from_numpy(x).to(TYPES[type_]))


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-33, 1e-45, 1e33])
@pytest.mark.parametrize("dim,type_", [(64, "f32"), (64, "bf16"), (128, "f32"), (128, "bf16"), (72, "f32"), (256, "f32"), (256, "bf16"), (512, "f32"), (512, "bf16")])
def test_norm_of_heads_of_any_magnitude(q, dim, type_, eps):
    rng = np.random.default_rng(dim)
    x = heads_of(dim, type_, rng)
    heads = x.shape[1] // dim
    table, w = table_of(dim, 10), (1 + 0.2 * rng.normal(size=dim)).astype(np.float32)
    xt = rows_tensor(x, TYPES[type_])
    out = torch.empty_like(xt)
    q.apr_rope_rows(q.Rope(torch.from_numpy(table).cuda()), ints([3, 7]), xt, out, heads, dim, norm=torch.from_numpy(w).cuda(), eps=eps)
    q.apr_stream_status()
    assert bool(torch.isfinite(out).all())
    assert_rows(out, oracle.rope_rows(table, None, False, [[3, 7]], x, heads, w, eps), type_, heads, True)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("dim,type_", [(64, "bf16"), (128, "f32"), (256, "f32"), (256, "bf16")])
def test_norm_on_the_way_into_the_cache(q, dim, type_, eps):
    # the same bits as the rows by themselves, k's and q's
    rng = np.random.default_rng(dim + 1)
    x = heads_of(dim, type_, rng)
    heads = x.shape[1] // dim
    table, w = table_of(dim, 50), torch.from_numpy((1 + 0.2 * rng.normal(size=dim)).astype(np.float32)).cuda()
    rope, k, v = q.Rope(torch.from_numpy(table).cuda()), rows_tensor(x, TYPES[type_]), rows_tensor(rng.normal(size=x.shape), TYPES[type_])
    rows = [rows_tensor(np.full(x.shape, np.nan), TYPES[type_]) for _ in range(2)]
    q.apr_rope_rows(rope, ints([31, 32]), k, rows[0], heads, dim, norm=w, eps=eps)
    caches = [q.Kv8Cache.allocate(3, heads, dim, 32) for _ in range(2)]
    pages, lens, start = ints([[2, 0]]), ints([33]), ints(starts([2]))
    q.apr_rope_kv8_append(caches[0], pages, lens, rope, k, v, k_norm=w, q=k, q_out=rows[1], num_heads=heads, q_norm=w, eps=eps, row_start=start)
    q.apr_kv8_append(caches[1], pages, lens, rows[0], v, row_start=start)
    q.apr_stream_status()
    assert bool(torch.isfinite(rows[0]).all()) and torch.equal(*rows)
    for name in ("K", "V", "k_scale", "v_scale"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name


def test_zeros_and_not_numbers_beside_heads_of_any_magnitude(q):
    # a head of zeros without an eps has no norm, as one with a NaN or an infinity: in its head alone
    dim, rng = 128, np.random.default_rng(5)
    x = rng.normal(size=(9, dim)) * np.array([1, 1e-30, 1, 1e30, 1, 1, 1e-25, 1, 1])[:, None]
    x[2], x[4, 5], x[7, 100] = 0, np.nan, -np.inf
    x, table, w = x.astype(np.float32).reshape(1, -1), table_of(dim, 10), np.ones(dim, np.float32)
    xt = torch.from_numpy(x).cuda()
    out = torch.empty_like(xt)
    q.apr_rope_rows(q.Rope(torch.from_numpy(table).cuda()), ints([4]), xt, out, 9, dim, norm=torch.from_numpy(w).cuda())
    q.apr_stream_status()
    y, keep = out.view(9, dim), [0, 1, 3, 5, 6, 8]
    assert bool(torch.isnan(y[[2, 4, 7]]).all())
    assert_rows(y[keep].reshape(1, -1), oracle.rope_rows(table, None, False, [[4]], x.reshape(9, dim)[keep].reshape(1, -1), 6, w, 0.0), "f32", 6, True)


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -100, -(2.0 ** -99), 2.0 ** 100])
def test_tables_at_the_ends_of_the_scales_range(q, scale):
    # half a step of float32, 2^-24 of a normal value and 2^-150 of a smaller one, and 2^-40 times the scale
    inv = (1.0 / 10000.0 ** (np.arange(36) / 36)).astype(np.float32)
    table = torch.full((1500, 36, 2), float("nan"), device="cuda")
    q.apr_rope_table(torch.from_numpy(inv).cuda(), table, first=5000, scale=scale)
    q.apr_stream_status()
    want = oracle.rope_table(inv, 5000, 1500, scale)
    assert (np.abs(table.cpu().numpy().astype(np.float64) - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -150 + 2.0 ** -40 * abs(scale)).all()
