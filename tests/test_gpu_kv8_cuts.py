"""GPU parity of the attention of chunks (include/apr_kv8.h) where a CTA's part of a segment is cut: 16-bit rows' sums are
taken over every 65536 positions; its small weights, and rows that see nothing.

A table names one page over and over, so the oracle is the attention of that page whose positions count as often as they
are named. Tolerances are those of tests/test_gpu_kv8_prefill.py for such tables: a score off by at most d 2^-24 R, 2^-17 more for the
exponentials and additions, both in a mean of values up to vmax; a weight rounded to fp16 (2^-11), what 65536 / 16 additions
lose (2^-12), 2^-22 for each time that sums are taken over or pieces combined; half a step of the output's type.
"""

import numpy as np
import pytest
import torch

from test_gpu_kv8 import TYPES, Case, as_f32, rows_tensor

pytestmark = pytest.mark.gpu

CUT = 65536


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def check_named_page(q, c, x, length, type_):
    """The chunk attention of rows x, the last ones of `length` positions that are all of c's first page, time after time."""
    n, tokens, heads, dim = len(x), c.tokens, c.heads, c.dim
    page = int(c.table[0, 0])
    x = rows_tensor(x, TYPES[type_])
    out = torch.full_like(x, float("nan"))
    table = torch.full((1, -(-length // tokens)), page, dtype=torch.int32, device="cuda")
    lens, start = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([length], [0, n]))
    q.apr_kv8_prefill_attention(c.cache, table, lens, x, out, heads, row_start=start)
    q.apr_stream_status()
    k, v = (c.host[w][page].astype(np.float64) * c.host[s][page][:, None, None] for w, s in (("K", "k_scale"), ("V", "v_scale")))
    rows = as_f32(x).astype(np.float64).reshape(n, heads, dim)
    score = np.einsum("ngd,gjd->ngj", rows, k) / np.sqrt(dim)
    reach = np.einsum("ngd,gjd->ngj", np.abs(rows), np.abs(k)).max(-1) / np.sqrt(dim)
    sees = length - n + 1 + np.arange(n)
    count = (sees[:, None] - np.arange(tokens) + tokens - 1) // tokens
    p = np.exp(score - score.max(-1, keepdims=True)) * count[:, None, :]
    p /= p.sum(-1, keepdims=True)
    want, size, vmax = np.einsum("ngj,gjd->ngd", p, v), np.einsum("ngj,gjd->ngd", p, np.abs(v)), np.abs(v).max()
    tol = (2 * dim * 2.0 ** -24 * reach + 2.0 ** -17)[..., None] * 2 * vmax + torch.finfo(TYPES[type_]).eps / 2 * np.abs(want)
    tol += ((length / CUT + 4) * 2.0 ** -22 + 2.0 ** -11 + 2.0 ** -12) * size + tokens * 2.0 ** -30 * vmax
    y = as_f32(out).astype(np.float64).reshape(want.shape)
    worst = float((np.abs(y - want) / tol).max())  # (NaN where an output is)
    assert worst <= 1, worst


@pytest.mark.parametrize("score", [-100.0, -200.0, -90.0, 100.0])
@pytest.mark.parametrize("dim,type_", [(64, "f16"), (128, "bf16"), (256, "bf16")])
def test_rows_that_see_nothing_of_the_last_cut(q, dim, type_, score):
    # a segment for each CTA, whose first rows end before a multiple of 65536 and whose last ones behind it: what the former
    # summed up stays, however low their scores are
    heads, n = sms(), 5
    c = Case([256], heads, dim, 256, seed=41)
    c.host["K"][..., 0], c.host["V"][:] = 100, np.abs(c.host["V"])
    c.host["k_scale"][:] = 0.03
    c.on_gpu(q)
    x = c.rng.normal(size=(n, heads, dim))
    x[..., 0] = score * np.sqrt(dim) / 3.0
    for length in (CUT + 2, 2 * CUT + 1):
        check_named_page(q, c, x.reshape(n, -1), length, type_)


@pytest.mark.parametrize("part,length", [((5, 13), 2 ** 19 + 77), ((2, 3), 2 ** 18 + 1), ((1, 3), 2 ** 19 + 200)])
@pytest.mark.parametrize("dim,type_,n", [(64, "bf16", 1), (128, "f16", 150), (256, "bf16", 140), (128, "bf16", 2)])
def test_cut_parts_of_shared_segments(q, dim, type_, n, part, length):
    # fewer heads than SMs, so that a CTA's share begins, ends or lies within a segment, and is longer than two cuts
    heads = sms() * part[0] // part[1] + 1
    assert heads * length // sms() > 2 * CUT
    c = Case([256], heads, dim, 256, seed=42).on_gpu(q)
    check_named_page(q, c, c.rng.normal(size=(n, heads * dim)), length, type_)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("code", [96, 120])
def test_small_weights_of_float32_rows(q, dim, code):
    # the first position's weight of 1 beside 6000 of exp(-s), alike, a head a CTA: each is off by at most 2^-34 of the largest (half of fp16's
    # last step, 2^-24, for its second piece, where the largest stands at 2^9 or more), which all have alike. What else may be off, relatively: the reference (two products of three
    # roundings, of a score of s log2 e < 22: 2^-24 * 3 * 22 * ln 2 < 2.8e-6), exponentials 2^-22, 512 / 16 steps of the tensor cores' sums
    # 2^-24 each (1.9e-6), 12 times that the sums are taken over 2^-22 (2.9e-6), and their total's additions (16 in the first part, 3 at each
    # joining: 3.1e-6), 1.1e-5 in all; scores are exact (a code times a power of two, q a small number)
    heads, length = sms(), 6000
    c = Case([128], heads, dim, 64, seed=43)
    first, other = (int(p) for p in c.table[0, :2])
    c.host["K"][:], c.host["V"][:] = 0, 100
    c.host["k_scale"][:], c.host["v_scale"][:] = 1.0, 1.0
    c.host["K"][first, :, 0, 0], c.host["V"][first, :, 0] = code, 0
    c.on_gpu(q)
    x = torch.zeros((3, heads, dim), device="cuda")
    x[..., 0] = 1.0
    x, out = x.view(3, -1), torch.empty((3, heads * dim), device="cuda")
    table = torch.full((1, 94), other, dtype=torch.int32, device="cuda")
    table[0, 0] = first
    lens, start = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([length], [0, 3]))
    q.apr_kv8_prefill_attention(c.cache, table, lens, x, out, heads, row_start=start, scale=0.125)
    q.apr_stream_status()
    small = np.exp(-code / 8.0) * (length - 3 + np.arange(3))
    worst = float(np.abs(as_f32(out) / (100 * small / (1 + small))[:, None] - 1).max())
    assert worst <= 2.0 ** -34 * np.exp(code / 8.0) + 1.5e-5, worst


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("type_", ["f32", "f16", "bf16"])
def test_rows_that_see_nothing_give_zeros_whatever_they_hold(q, dim, type_):
    # a slot without a sequence, and rows before a sequence's start: zeros, as from the attention of few rows, where a row that
    # sees a position becomes NaN
    c = Case([0, 3, 40], 2, dim, 32, seed=44).on_gpu(q)
    x = torch.from_numpy(c.rng.normal(size=(11, 4 * dim))).cuda().to(TYPES[type_])
    x[:6, 7], x[:6, dim + 9], x[:6, 3 * dim] = float("nan"), float("inf"), -float("inf")
    out, few = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    start = torch.tensor([0, 1, 8, 11], dtype=torch.int32, device="cuda")  # seven rows of a sequence of three tokens
    for call, y in ((q.apr_kv8_prefill_attention, out), (q.apr_kv8_attention, few)):
        call(c.cache, c.gtable, c.glens, x, y, 4, row_start=start)
    q.apr_stream_status()
    nan = torch.zeros((11, 4), dtype=torch.bool, device="cuda")
    nan[5, [0, 1, 3]] = True
    for y in (out, few):
        assert not y[:5].any() and torch.equal(torch.isnan(y.view(11, 4, dim)).all(-1), nan) and torch.equal(torch.isnan(y.view(11, 4, dim)).any(-1), nan)


@pytest.mark.parametrize("dim,type_", [(64, "f16"), (128, "bf16"), (256, "f16"), (64, "f32"), (128, "f32"), (256, "f32")])
@pytest.mark.parametrize("steps", [3.0, 3.9998, 4.0, 4.1, 7.9998, 8.0])
@pytest.mark.parametrize("grown", [1.0, 1.999, 4.0])
def test_weights_at_the_top_of_their_range(q, dim, type_, steps, grown):
    # scores of 0 under V scales of 1, then one position whose score is `steps` higher in base 2, in a page of a larger
    # scale: weights next to the largest that a reference and a scale are kept for, which no fp16 number may end below
    heads = sms()
    c = Case([128], heads, dim, 64, seed=45)
    plain, high = (int(p) for p in c.table[0, :2])
    c.host["K"][:], c.host["V"][:] = 0, 100
    c.host["k_scale"][:], c.host["v_scale"][plain], c.host["v_scale"][high] = 1.0, 1.0, grown
    c.host["K"][high, :, 5, 0] = 64
    c.on_gpu(q)
    x = torch.zeros((2, heads, dim), device="cuda")
    x[..., 0] = 1.0
    x = x.view(2, -1).to(TYPES[type_])
    out = torch.empty_like(x)
    table = torch.tensor([[plain] * 5 + [high] + [plain] * 5], dtype=torch.int32, device="cuda")
    lens, start = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([11 * 64], [0, 2]))
    q.apr_kv8_prefill_attention(c.cache, table, lens, x, out, heads, row_start=start, scale=steps / 1.4426950408889634 / 64)
    q.apr_stream_status()
    total = np.array([11 * 64 - 2, 11 * 64 - 1]) + 2.0 ** steps
    want = 100 * ((total - 63 - 2.0 ** steps) + (63 + 2.0 ** steps) * grown) / total
    # a weight rounded to fp16, the output to its type; float32: two pieces, the exponentials, sums of 11 * 64 / 16 steps
    tol = 2.0 ** -11 + torch.finfo(TYPES[type_]).eps / 2 + 2.0 ** -18 if type_ != "f32" else 2.0 ** -18
    worst = float(np.abs(as_f32(out) / want[:, None] - 1).max())
    assert worst <= tol, worst
