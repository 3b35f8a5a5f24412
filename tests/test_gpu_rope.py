"""GPU parity of the rotations by position (include/apr_rope.h) against their oracle.

The table: within half a step of float32 of the float64 values, and 2^-40 (of 1) for the two float64 sides' own errors.

Rows without a norm are bit for bit: every rounding is the definition's. With a norm 1 / rms is taken to more than 40
bits before its rounding, so it is the oracle's but where the exact value lies within 2^-41 of the middle of two float32
numbers, of 2^-24 apart: one head in 2^16 or so may have all its values one step of float32 off, which moves a
rotated value by at most 2^-22 of the head's largest normed magnitude, and then by one rounding to the type. A
hundred of the 10^4 heads of a test would be a fault; it allows 3.
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv8 import TYPES, Case, as_f32, bad_index, rows_tensor, starts

pytestmark = pytest.mark.gpu


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def table_of(rot, positions, base=10000.0):
    inv = (1.0 / base ** (np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    return oracle.rope_table(inv, 0, positions).astype(np.float32)


def assert_rows(got, want, type_, heads, normed, scale=None):
    w = torch.from_numpy(want).to(TYPES[type_])
    if not normed:
        assert torch.equal(got.cpu(), w)
        return
    y, w = as_f32(got).astype(np.float64), w.float().numpy().astype(np.float64)
    off = (y != w).reshape(len(y), heads, -1).any(-1).sum()
    assert off <= 3, off
    top = np.abs(want.reshape(len(y), heads, -1)).max(-1).repeat(want.shape[1] // heads, 1) * 1.5  # (turned: up to sqrt 2 more)
    assert (np.abs(y - w) <= 2.0 ** -22 * top + torch.finfo(TYPES[type_]).eps * np.abs(w)).all()


# ---------------------------------------------------------------- the table
@pytest.mark.parametrize("pairs,first,positions,scale,base", [
    (4, 0, 1, 1.0, 10000.0), (32, 0, 1000, 1.0, 10000.0), (36, 7, 333, 1.25, 1e6), (128, 1, 5000, 0.9, 5e6),
    (1, 100, 70, 1.0, 1.0), (3, 0, 50, 1.0, 10.0), (64, 131072 - 3, 2100, -1.0, 500000.0), (256, (1 << 30) - 700, 700, 1.0, 1e4),
    (129, 2**24 - 5, 300, 1.0, 100.0)])
def test_table(q, pairs, first, positions, scale, base):
    rng = np.random.default_rng(pairs)
    inv = (1.0 / base ** (np.arange(pairs) / pairs) * np.exp(0.1 * rng.normal(size=pairs))).astype(np.float32)
    table = torch.full((positions, pairs, 2), float("nan"), device="cuda")
    q.apr_rope_table(torch.from_numpy(inv).cuda(), table, first=first, scale=scale)
    q.apr_stream_status()
    want = oracle.rope_table(inv, first, positions, scale)
    y = table.cpu().numpy().astype(np.float64)
    assert (np.abs(y - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -40).all(), float(np.abs(y - want).max())


@pytest.mark.parametrize("value", [0.0, -0.5, 900.0, 1e-30, 1e-40])
def test_table_of_unusual_frequencies(q, value):
    # none at all, backwards, many turns a position, the smallest numbers
    inv = np.array([value, 1.0, value, 0.25], np.float32)
    table = torch.empty((3000, 4, 2), device="cuda")
    q.apr_rope_table(torch.from_numpy(inv).cuda(), table)
    want = oracle.rope_table(inv, 0, 3000)
    y = table.cpu().numpy().astype(np.float64)
    assert (np.abs(y - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -40).all()


def test_table_bits_do_not_depend_on_where_it_begins(q):
    inv = torch.from_numpy((1.0 / 1e5 ** (np.arange(64) / 64)).astype(np.float32)).cuda()
    whole, part = torch.empty((9000, 64, 2), device="cuda"), torch.empty((1234, 64, 2), device="cuda")
    q.apr_rope_table(inv, whole)
    q.apr_rope_table(inv, part, first=4321)
    off = (whole[4321:4321 + 1234] != part).float().mean()
    assert float(off) <= 1e-3  # (the exact value lies next to the middle of two float32 numbers)
    assert float((whole[4321:4321 + 1234] - part).abs().max()) <= 2.0 ** -23


def test_table_past_4_gib(q):
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    inv = np.linspace(0.01, 1, 256).astype(np.float32)
    table = torch.empty((2_200_000, 256, 2), device="cuda")  # 4.5e9 bytes
    q.apr_rope_table(torch.from_numpy(inv).cuda(), table)
    q.apr_stream_status()
    for at in (0, 1_048_575, 1_048_576, 2_097_151, 2_199_990):
        want = oracle.rope_table(inv, at, 10)
        assert np.abs(table[at:at + 10].cpu().numpy() - want).max() <= 2.0 ** -24 + 2.0 ** -40


# ---------------------------------------------------------------- rows
ROWS = [
    # dim, rot, heads, layout, axes, norm, type, rows, pad
    (8, 8, 1, "halves", 1, False, "f32", 1, 0),
    (64, 64, 3, "halves", 1, False, "bf16", 37, 8),
    (64, 16, 5, "pairs", 1, True, "f16", 130, 0),
    (72, 72, 4, "pairs", 2, False, "f16", 77, 16),
    (80, 80, 2, "halves", 2, True, "f32", 61, 4),
    (128, 128, 32, "halves", 3, True, "bf16", 300, 0),
    (128, 96, 7, "pairs", 4, False, "f32", 33, 12),
    (256, 64, 16, "halves", 1, True, "f32", 5, 0),
    (256, 256, 6, "halves", 3, False, "f16", 90, 8),
    (264, 264, 3, "halves", 1, True, "bf16", 40, 8),
    (512, 512, 2, "pairs", 3, True, "f32", 29, 0),
    (512, 24, 1, "halves", 16, False, "bf16", 50, 0),
    (136, 40, 9, "halves", 1, True, "f16", 1000, 0),
    (128, 128, 1, "halves", 1, False, "f32", 2049, 0),
]


def axes_of(pairs, axes, rng):
    return None if axes == 1 else rng.integers(0, axes, pairs).astype(np.uint8)


@pytest.mark.parametrize("dim,rot,heads,layout,axes,norm,type_,rows,pad", ROWS)
@pytest.mark.parametrize("in_place", [False, True])
def test_rows(q, dim, rot, heads, layout, axes, norm, type_, rows, pad, in_place):
    rng = np.random.default_rng(dim + rot + rows)
    table, axis = table_of(rot, 500), axes_of(rot // 2, axes, rng)
    positions = rng.integers(0, 500, (axes, rows))
    weights = (1 + 0.3 * rng.normal(size=dim)).astype(np.float32) if norm else None
    x = rows_tensor(rng.normal(size=(rows, heads * dim)) * np.exp(rng.normal(size=(rows, 1))), TYPES[type_], pad)
    want = oracle.rope_rows(table, axis, layout == "pairs", positions, as_f32(x), heads, weights, 1e-6)
    out = x if in_place else rows_tensor(np.full((rows, heads * dim), np.nan), TYPES[type_], 2 * pad)
    rope = q.Rope(torch.from_numpy(table).cuda(), interleaved=layout == "pairs", pair_axis=None if axis is None else torch.from_numpy(axis).cuda())
    q.apr_rope_rows(rope, ints(positions if axes > 1 else positions[0]), x, out, heads, dim,
                    norm=None if weights is None else torch.from_numpy(weights).cuda(), eps=1e-6)
    q.apr_stream_status()
    assert_rows(out, want, type_, heads, norm)
    if pad and rows > 1:  # what lies between the rows is left alone
        assert bool(torch.isnan(out.as_strided((rows - 1, out.stride(0) - heads * dim), (out.stride(0), 1), out.storage_offset() + heads * dim)).all())


def test_rows_between_other_slices_of_one_buffer(q):
    # q rotated into the place of another slice of the same fused rows, three-dimensional views
    rng = np.random.default_rng(1)
    wide = torch.from_numpy(rng.normal(size=(50, 3, 4, 64)).astype(np.float32)).cuda()
    before = wide.clone()
    table = table_of(64, 100)
    positions = rng.integers(0, 100, 50)
    q.apr_rope_rows(q.Rope(torch.from_numpy(table).cuda()), ints(positions), wide[:, 0], wide[:, 2], 4, 64)
    q.apr_stream_status()
    want = oracle.rope_rows(table, None, False, [positions], before[:, 0].reshape(50, -1).cpu().numpy(), 4)
    assert torch.equal(wide[:, :2], before[:, :2])
    assert np.array_equal(wide[:, 2].reshape(50, -1).cpu().numpy(), want)


def test_norm_of_unusual_heads(q):
    # zeros (with eps: zeros), the smallest and the largest squares, one value beside many small ones, not-numbers in their head alone
    dim, heads = 128, 8
    rng = np.random.default_rng(2)
    x = rng.normal(size=(1, heads * dim)).astype(np.float32).reshape(heads, dim)
    x[0] = 0
    x[1] *= np.float32(2.0 ** 58)
    x[2] *= np.float32(1e-18)
    x[3], x[3, 7] = 1e-4, 1000.0
    x[5, 9], x[6, 100] = np.nan, np.inf
    table = table_of(dim, 10)
    w = (1 + rng.normal(size=dim)).astype(np.float32)
    xt = torch.from_numpy(x.reshape(1, -1)).cuda()
    out = torch.empty_like(xt)
    q.apr_rope_rows(q.Rope(torch.from_numpy(table).cuda()), ints([3]), xt, out, heads, dim, norm=torch.from_numpy(w).cuda(), eps=1e-6)
    q.apr_stream_status()
    y = out.view(heads, dim)
    bad = [5, 6]
    assert bool(torch.isnan(y[bad]).all()) and bool(torch.isfinite(y[[0, 1, 2, 3, 4, 7]]).all())
    keep = [0, 1, 2, 3, 4, 7]
    want = oracle.rope_rows(table, None, False, [[3]], x[keep].reshape(1, -1), len(keep), w, 1e-6)
    assert_rows(y[keep].reshape(1, -1), want, "f32", len(keep), True)
    assert not y[0].any()


def test_rotating_back_gives_the_rows_again(q):
    # by the negative angles, to two roundings of products and one of a sum each way: 2^-22 of the pair's length
    table = table_of(128, 4000)
    back = table * np.array([1, -1], np.float32)
    rng = np.random.default_rng(3)
    x = rng.normal(size=(400, 2 * 128)).astype(np.float32)
    positions, xt = ints(rng.integers(0, 4000, 400)), torch.from_numpy(x).cuda()
    y, z = torch.empty_like(xt), torch.empty_like(xt)
    q.apr_rope_rows(q.Rope(torch.from_numpy(table).cuda()), positions, xt, y, 2, 128)
    q.apr_rope_rows(q.Rope(torch.from_numpy(back).cuda()), positions, y, z, 2, 128)
    q.apr_stream_status()
    pairs = x.reshape(400, 2, 2, 64)
    length = np.sqrt((pairs.astype(np.float64) ** 2).sum(2, keepdims=True)).repeat(2, 2).reshape(x.shape)
    assert (np.abs(z.cpu().numpy() - x) <= 6 * 2.0 ** -24 * length).all()


@pytest.mark.parametrize("what", ["negative", "past", "axis"])
def test_positions_and_axes_that_are_not_there_are_reported(q, what):
    table = torch.from_numpy(table_of(64, 50)).cuda()
    axis = torch.zeros(32, dtype=torch.uint8, device="cuda")
    positions = torch.zeros((2, 9), dtype=torch.int32, device="cuda")
    if what == "axis":
        axis[13] = 2
    else:
        positions[1, 4] = -1 if what == "negative" else 50
        axis[13] = 1
    x = torch.randn((9, 64), device="cuda")
    out = torch.empty_like(x)
    q.apr_rope_rows(q.Rope(table, pair_axis=axis), positions, x, out, 1, 64)
    bad_index(q)
    q.apr_rope_rows(q.Rope(table), positions[:1].contiguous(), x, out, 1, 64)
    q.apr_stream_status()


def test_rows_past_2_to_the_32_elements(q):
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    rows, ld = 40000, 1 << 17
    buf = torch.zeros((rows, ld), dtype=torch.bfloat16, device="cuda")  # 5.2e9 elements, the rows' slice of them random
    x = buf[:, 640:640 + 256]
    x.copy_(torch.randn((rows, 256), device="cuda"))
    small = x.contiguous()
    positions = torch.arange(rows, dtype=torch.int32, device="cuda") % 300
    rope = q.Rope(torch.from_numpy(table_of(64, 300)).cuda())
    out = torch.empty_like(small)
    q.apr_rope_rows(rope, positions, small, out, 4, 64)
    q.apr_rope_rows(rope, positions, x, x, 4, 64)
    q.apr_stream_status()
    assert torch.equal(x, out)
    assert not buf[:, :640].any() and not buf[:, 896:1024].any()


def test_positions_followed_by_a_replayed_graph(q):
    table, rng = table_of(64, 1000), np.random.default_rng(4)
    x = torch.from_numpy(rng.normal(size=(6, 128)).astype(np.float32)).cuda()
    positions, out, rope = ints(np.arange(6)), torch.empty_like(x), q.Rope(torch.from_numpy(table).cuda())
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        q.apr_rope_rows(rope, positions, x, out, 2, 64)
    for at in (np.arange(6), np.arange(6) + 700, np.full(6, 3)):
        positions.copy_(torch.from_numpy(at.astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(as_f32(out), oracle.rope_rows(table, None, False, [at], as_f32(x), 2))


# ---------------------------------------------------------------- on the way into the cache
APPENDS = [
    # lens, rows, dim, rot, tokens, heads, group, layout, axes, norm, type, pad
    ([1, 64, 65, 130, 0, 200], None, 128, 128, 64, 2, 4, "halves", 1, False, "f32", 0),
    ([5, 64, 128, 300], [5, 64, 128, 300], 64, 32, 32, 3, 2, "pairs", 3, True, "bf16", 8),
    ([70, 129, 40, 257], [6, 65, 0, 200], 256, 64, 128, 1, 3, "halves", 1, True, "f16", 24),
    ([3, 10], [5, 10], 256, 256, 256, 2, 1, "halves", 1, False, "f32", 4),       # more rows than positions
    ([900, 20, 0, 333], [700, 20, 0, 1], 256, 256, 256, 2, 2, "pairs", 2, True, "f32", 0),
    ([1000, 300], [999, 64], 128, 128, 256, 4, 1, "halves", 3, True, "bf16", 0),
    ([400], [400], 64, 64, 64, 8, 2, "halves", 1, False, "f16", 0),
]


def append_args(q, c, rows, rot, heads, group, layout, axes, norm, type_, pad):
    n = len(c.lens) if rows is None else sum(rows)
    dim, rng = c.dim, c.rng
    width = (heads * group + 2 * heads) * dim
    qkv = rows_tensor(rng.normal(size=(n, width)) * np.exp(rng.normal(size=(n, 1))), TYPES[type_], pad)
    parts = qkv.split((heads * group * dim, heads * dim, heads * dim), 1)
    table, axis = table_of(rot, 1300), axes_of(rot // 2, axes, rng)
    positions = None if axes == 1 else rng.integers(0, 1300, (axes, n))
    norms = [(1 + 0.3 * rng.normal(size=dim)).astype(np.float32) if norm else None for _ in range(2)]
    rope = q.Rope(torch.from_numpy(table).cuda(), interleaved=layout == "pairs", pair_axis=None if axis is None else torch.from_numpy(axis).cuda())
    return n, parts, table, axis, positions, norms, rope


def places(lens, rows, n):
    at = np.zeros(n, np.int64)
    start = starts([1] * len(lens) if rows is None else rows)
    for b, length in enumerate(lens):
        count = start[b + 1] - start[b]
        at[start[b]:start[b + 1]] = np.maximum(length - count + np.arange(count), 0)
    return at


@pytest.mark.parametrize("lens,rows,dim,rot,tokens,heads,group,layout,axes,norm,type_,pad", APPENDS)
def test_append(q, lens, rows, dim, rot, tokens, heads, group, layout, axes, norm, type_, pad):
    c = Case(lens, heads, dim, tokens, seed=len(lens) + dim).on_gpu(q)
    n, (qx, k, v), table, axis, positions, norms, rope = append_args(q, c, rows, rot, heads, group, layout, axes, norm, type_, pad)
    gnorm = [None if w is None else torch.from_numpy(w).cuda() for w in norms]
    start = None if rows is None else starts(rows)
    gstart = None if rows is None else ints(start)
    at = positions if positions is not None else [places(lens, rows, n)]
    wide = heads * group * dim
    qo = torch.full((n, wide + 8), float("nan"), dtype=TYPES[type_], device="cuda")[:, :wide]
    q.apr_rope_kv8_append(c.cache, c.gtable, c.glens, rope, k, v, positions=None if positions is None else ints(positions),
                          k_norm=gnorm[0], q=qx, q_out=qo, num_heads=heads * group, q_norm=gnorm[1], eps=1e-5, row_start=gstart,
                          max_rows=0 if rows is None else max(rows))
    q.apr_stream_status()
    want = oracle.rope_rows(table, axis, layout == "pairs", at, as_f32(qx), heads * group, norms[1], 1e-5)
    assert_rows(qo, want, type_, heads * group, norm)
    # the same bits as one call after the other
    other = Case(lens, heads, dim, tokens, seed=len(lens) + dim).on_gpu(q)
    kr = torch.empty((n, heads * dim), dtype=TYPES[type_], device="cuda")
    q.apr_rope_rows(rope, ints(np.asarray(at) if axes > 1 else at[0]), k, kr, heads, dim, norm=gnorm[0], eps=1e-5)
    vr = v.contiguous()
    q.apr_kv8_append(other.cache, other.gtable, other.glens, kr, vr, row_start=gstart)
    q.apr_stream_status()
    for name in ("K", "V", "k_scale", "v_scale"):
        assert torch.equal(getattr(c.cache, name), getattr(other.cache, name)), name
    # and, without a norm, the oracle's
    if not norm:
        kw = torch.from_numpy(oracle.rope_rows(table, axis, layout == "pairs", at, as_f32(k), heads)).to(TYPES[type_])
        c.assert_cache(oracle.kv8_append(c.host, c.table, c.lens, start, kw.float().numpy(), as_f32(v)))
    # once more, in place: nothing changes in the cache, q comes out in its own place
    cache = [getattr(c.cache, name).clone() for name in ("K", "V", "k_scale", "v_scale")]
    q.apr_rope_kv8_append(c.cache, c.gtable, c.glens, rope, k, v, positions=None if positions is None else ints(positions),
                          k_norm=gnorm[0], q=qx, q_out=qx, num_heads=heads * group, q_norm=gnorm[1], eps=1e-5, row_start=gstart)
    q.apr_stream_status()
    assert torch.equal(qx, qo)
    for name, a in zip(("K", "V", "k_scale", "v_scale"), cache):
        assert torch.equal(getattr(c.cache, name), a)


@pytest.mark.parametrize("dim,tokens,type_", [(64, 32, "f32"), (128, 256, "bf16"), (256, 64, "f32")])
def test_append_without_q_of_special_values(q, dim, tokens, type_):
    # rows of infinities and not-numbers: stored as the largest code and 0, their page's scale from what is finite
    c = Case([tokens + 9, 5], 2, dim, tokens, seed=5).on_gpu(q)
    x = c.rng.normal(size=(tokens + 14, 2 * dim)).astype(np.float32)
    x[3, 5], x[4, dim + 1], x[tokens + 2, 0] = np.inf, -np.inf, np.nan
    x[9] = 0
    k, table = rows_tensor(x, TYPES[type_]), table_of(dim // 2, 600)
    rows = [tokens + 9, 5]
    q.apr_rope_kv8_append(c.cache, c.gtable, c.glens, q.Rope(torch.from_numpy(table).cuda()), k, k, row_start=ints(starts(rows)))
    q.apr_stream_status()
    kr = torch.empty_like(k)
    other = Case([tokens + 9, 5], 2, dim, tokens, seed=5).on_gpu(q)
    q.apr_rope_rows(q.Rope(torch.from_numpy(table).cuda()), ints(places([tokens + 9, 5], rows, tokens + 14)), k, kr, 2, dim)
    q.apr_kv8_append(other.cache, other.gtable, other.glens, kr, k, row_start=ints(starts(rows)))
    q.apr_stream_status()
    for name in ("K", "V", "k_scale", "v_scale"):
        assert torch.equal(getattr(c.cache, name), getattr(other.cache, name)), name


@pytest.mark.parametrize("what", ["page", "length", "row_start", "position"])
def test_append_reports_what_cannot_be(q, what):
    c = Case([70, 40], 2, 64, 32, seed=6).on_gpu(q)
    k, table = torch.randn((6, 128), device="cuda"), table_of(64, 60 if what == "position" else 100)
    start = ints([0, 4, 6])
    want = [0, 40]
    if what == "page":
        c.gtable[0, 2] = c.cache.K.shape[0]
    elif what == "length":
        c.glens[0] = 1 << 20
    elif what == "row_start":
        start = ints([5, 4, 6])
    q.apr_rope_kv8_append(c.cache, c.gtable, c.glens, q.Rope(torch.from_numpy(table).cuda()), k, k, q=k.clone(), q_out=torch.empty_like(k),
                          num_heads=2, row_start=start)
    bad_index(q)
    if what != "position":  # the other sequence's rows are appended all the same
        rows = as_f32(k)
        kr = oracle.rope_rows(table, None, False, [[0, 0, 0, 0, 38, 39]], rows, 2)
        c.assert_cache(oracle.kv8_append(c.host, c.table, want, [0, 0, 2], kr[4:], rows[4:]))


def test_append_to_many_ragged_sequences(q):
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 200, 1500)
    rows = np.where(rng.random(1500) < 0.3, 0, np.minimum(rng.integers(0, 100, 1500), lens))
    rows[7] = lens[7] + 5
    c = Case(list(lens), 1, 64, 32, seed=8).on_gpu(q)
    start = starts(rows) + np.int32(3)  # packed rows ahead of the first sequence's
    x = [c.rng.normal(size=(int(start[-1]) + 9, 64)).astype(np.float32) for _ in range(3)]
    table = table_of(64, 300)
    k, v, qx = (torch.from_numpy(a).cuda() for a in x)
    qo = torch.full_like(qx, 7)
    q.apr_rope_kv8_append(c.cache, c.gtable, c.glens, q.Rope(torch.from_numpy(table).cuda()), k, v, q=qx, q_out=qo, num_heads=1, row_start=ints(start))
    q.apr_stream_status()
    at = np.zeros(len(x[0]), np.int64)
    at[3:start[-1]] = places(lens, rows, int(start[-1]) - 3)
    kr, qr = (oracle.rope_rows(table, None, False, [at], a, 1) for a in (x[0], x[2]))
    c.assert_cache(oracle.kv8_append(c.host, c.table, c.lens, start, kr, x[1]))
    assert np.array_equal(as_f32(qo)[3:start[-1]], qr[3:start[-1]])
    assert bool((qo[:3] == 7).all()) and bool((qo[int(start[-1]):] == 7).all())  # rows of no sequence


def test_append_step_followed_by_a_replayed_graph_on_another_stream(q):
    # decode steps: lengths grow between replays, positions are the places in the cache
    c = Case([3, 40], 2, 64, 32, seed=9, spare=8, extra_width=2).on_gpu(q)
    c.table[:, 1:4] = c.free[:6].reshape(2, 3) if c.table.shape[1] >= 4 else c.table[:, 1:4]
    c.gtable.copy_(torch.from_numpy(c.table))
    want, table = c.host, table_of(64, 200)
    k, v, x = (torch.zeros((2, n * 64), device="cuda") for n in (2, 2, 4))
    rope, out = q.Rope(torch.from_numpy(table).cuda()), torch.empty_like(x)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        q.apr_rope_kv8_append(c.cache, c.gtable, c.glens, rope, k, v, q=x, q_out=out, num_heads=4)
    for step in range(1, 40):
        c.lens[:] = (3 + step, 40 + step)
        c.glens.copy_(torch.from_numpy(c.lens))
        rows = [c.rng.normal(size=t.shape).astype(np.float32) for t in (k, v, x)]
        for t, a in zip((k, v, x), rows):
            t.copy_(torch.from_numpy(a))
        graph.replay()
        at = [[2 + step, 39 + step]]
        want = oracle.kv8_append(want, c.table, c.lens, None, oracle.rope_rows(table, None, False, at, rows[0], 2), rows[1])
        assert np.array_equal(as_f32(out), oracle.rope_rows(table, None, False, at, rows[2], 4))
    torch.cuda.synchronize()
    c.assert_cache(want)


def test_append_of_a_padded_batch_followed_by_a_replayed_graph(q):
    # one captured call with positions, replayed as rows and lengths change; what stands in the padding is not looked at
    c = Case([200, 120, 90], 2, 64, 32, seed=24).on_gpu(q)
    want, table = c.host, table_of(32, 500)
    rope = q.Rope(torch.from_numpy(table).cuda(), pair_axis=torch.from_numpy((np.arange(16) % 2).astype(np.uint8)).cuda())
    k, v, x = (torch.zeros((150, n * 64), device="cuda") for n in (2, 2, 4))
    out, positions, start = torch.empty_like(x), ints(np.zeros((2, 150))), ints(np.zeros(4))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        q.apr_rope_kv8_append(c.cache, c.gtable, c.glens, rope, k, v, positions=positions, q=x, q_out=out, num_heads=4, row_start=start)
    for lens, rows in (([60, 3, 90], [60, 3, 80]), ([61, 0, 90], [1, 0, 0]), ([200, 120, 90], [139, 11, 0]), ([5, 5, 5], [0, 0, 0])):
        n = sum(rows)
        c.lens[:] = lens
        c.glens.copy_(torch.from_numpy(c.lens))
        start.copy_(torch.from_numpy(starts(rows)))
        data = [c.rng.normal(size=t.shape).astype(np.float32) for t in (k, v, x)]
        at = c.rng.integers(0, 500, (2, 150)).astype(np.int32)
        for a in data:
            a[n:] = np.nan
        at[:, n:] = np.array([[-5], [1 << 20]])
        for t, a in zip((k, v, x, positions), (*data, at)):
            t.copy_(torch.from_numpy(a))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        axis = np.arange(16) % 2
        turned = [oracle.rope_rows(table, axis, False, at[:, :n], data[i][:n], h) for i, h in ((0, 2), (2, 4))]
        if n:
            want = oracle.kv8_append(want, c.table, c.lens, starts(rows), turned[0], data[1][:n])
        c.assert_cache(want)
        assert np.array_equal(as_f32(out)[:n], turned[1]) and bool((out[n:] == 7).all())
    q.apr_stream_status()


def test_two_streams_at_once(q):
    cases = [Case([900, 33], 2, 128, 64, seed=s).on_gpu(q) for s in (25, 26)]
    streams, table = [torch.cuda.Stream() for _ in cases], table_of(128, 1000)
    rope, start = q.Rope(torch.from_numpy(table).cuda()), ints([0, 700, 733])
    rows = [[torch.from_numpy(c.rng.normal(size=(733, w * 128)).astype(np.float32)).cuda() for w in (2, 2, 4)] for c in cases]
    outs, turned = [torch.empty_like(r[2]) for r in rows], [torch.empty_like(r[2]) for r in rows]
    at = places([900, 33], [700, 33], 733)
    gat = ints(at)
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, (k, v, x), out, alone in zip(cases, streams, rows, outs, turned):
            q.apr_rope_kv8_append(c.cache, c.gtable, c.glens, rope, k, v, q=x, q_out=out, num_heads=4, row_start=start, stream=s)
            q.apr_rope_rows(rope, gat, x, alone, 4, 128, stream=s)
    for s in streams:
        q.apr_stream_status(s)
    for c, (k, v, x), out, alone in zip(cases, rows, outs, turned):
        assert torch.equal(out, alone)
        assert np.array_equal(as_f32(out), oracle.rope_rows(table, None, False, [at], as_f32(x), 4))
        kr = oracle.rope_rows(table, None, False, [at], as_f32(k), 2)
        host = c.host
        for _ in range(10):
            host = oracle.kv8_append(host, c.table, c.lens, [0, 700, 733], kr, as_f32(v))
        c.assert_cache(host)
