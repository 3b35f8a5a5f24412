"""GPU parity of the attention of chunks of rows over the 8-bit paged cache (include/apr_kv8.h) against its float64 oracle.

float32 rows are held to what the attention of few rows is (tests/test_gpu_kv8.py): a score is off by at most
d 2^-24 R, R the largest sum of |scale q_c k_c| over a position that a row sees, 2^-17 more for the exponentials and
additions, in a mean of values up to vmax; and 1e-5 over all elements. For the additions the tensor cores lose up to
2^-24 of a sum at each of the at most 2 * 512 / 16 steps before a sum is taken over, 2^-18 in all, within the 2^-17.

16-bit rows: the softmax weights enter the second product rounded to fp16, each off by at most 2^-11 of itself (eps / 2)
where it is normal, by 2^-25 of 2^-7 of the largest otherwise: 2^-11 of the sum of p_j |V_j|, and positions * 2^-31 of vmax.
fp16 sums lose 2^-24 a step over all of a sequence's steps of 16 positions: positions * 2^-28 of the sum of p_j |V_j|. The output adds
half a step of its type.
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv8 import EXACT_REL, TYPES, Case, as_f32, bad_index, rows_tensor, starts
from test_gpu_kv8_limits import both_at_once, us_of

pytestmark = pytest.mark.gpu


def attend(q, c, num_heads, rows=None, type_="f32", pad=0, scale=0.0, qh=None, **more):
    n = len(c.lens) if rows is None else sum(rows)
    qh = c.rng.normal(size=(n, num_heads * c.dim)) if qh is None else qh
    qt = rows_tensor(qh, TYPES[type_], pad)
    out = rows_tensor(np.full((n, num_heads * c.dim), np.nan), TYPES[type_], 2 * pad)
    gstart = None if rows is None else torch.from_numpy(starts(rows)).cuda()
    q.apr_kv8_prefill_attention(c.cache, c.gtable, c.glens, qt, out, num_heads, row_start=gstart, scale=scale, **more)
    q.apr_stream_status()
    if pad and n > 1:
        assert bool(torch.isnan(out.as_strided((n - 1, 2 * pad), (out.stride(0), 1), out.storage_offset() + out.shape[1])).all())
    return out, qt


def check(c, out, qt, num_heads, rows=None, type_="f32", scale=0.0, frobenius=True):
    start = None if rows is None else starts(rows)
    want, _, reach = oracle.kv8_attention(c.host, c.table, c.lens, start, as_f32(qt), num_heads, scale)
    host = dict(c.host, V=np.abs(c.host["V"].astype(np.int16)))
    size = oracle.kv8_attention(host, c.table, c.lens, start, as_f32(qt), num_heads, scale)[0] if type_ != "f32" else 0.0
    y = as_f32(out).astype(np.float64).reshape(want.shape)
    vmax = float((np.abs(c.host["V"].astype(np.float64)) * c.host["v_scale"][..., None, None]).max())
    half = torch.finfo(TYPES[type_]).eps / 2
    tol = (2 * c.dim * 2.0 ** -24 * reach + 2.0 ** -17)[..., None] * 2 * vmax + half * np.abs(want)
    if type_ != "f32":
        tol = tol + (2.0 ** -11 + max(c.lens) * 2.0 ** -28) * size + max(c.lens) * 2.0 ** -31 * vmax
    assert np.isfinite(y).all()
    assert (np.abs(y - want) <= tol).all(), float((np.abs(y - want) / tol).max())
    if frobenius and np.linalg.norm(want):
        rel = np.linalg.norm(y - want) / np.linalg.norm(want)
        assert rel <= EXACT_REL if type_ == "f32" else rel <= half + 2.0 ** -11 * max(1.0, np.linalg.norm(size) / np.linalg.norm(want)), rel


def both(q, c, num_heads, rows=None, type_="f32", scale=0.0, frobenius=True, **more):
    out, qt = attend(q, c, num_heads, rows, type_, scale=scale, **more)
    check(c, out, qt, num_heads, rows, type_, scale, frobenius)
    return out


# ---------------------------------------------------------------- heads, types, pages, lengths
@pytest.mark.parametrize("dim,heads,group,tokens,type_", [
    (64, 2, 1, 32, "f32"), (64, 1, 8, 64, "bf16"), (64, 2, 3, 256, "f16"), (128, 2, 4, 64, "f32"), (128, 3, 7, 32, "f16"),
    (128, 1, 16, 128, "bf16"), (256, 2, 4, 64, "f32"), (256, 1, 5, 256, "bf16"), (256, 2, 2, 32, "f16"), (64, 1, 33, 32, "f32")])
@pytest.mark.parametrize("rows,lens", [
    ([3, 0, 7, 1], [50, 300, 70, 1]),                     # few rows, a sequence without, one of one token
    ([40, 17, 64], [40, 400, 64]),                        # whole prompts and a chunk behind a prefix
    ([130, 1, 65], [1000, 777, 129]),                     # a chunk beside a single token
])
def test_heads_types_and_pages(q, dim, heads, group, tokens, type_, rows, lens):
    c = Case(lens, heads, dim, tokens, seed=dim + group + len(lens)).on_gpu(q)
    both(q, c, heads * group, rows, type_, pad=8)


LENS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 257, 511, 1000]


@pytest.mark.parametrize("dim,type_", [(64, "f16"), (128, "bf16"), (256, "f32"), (128, "f32"), (256, "f16"), (64, "f32")])
def test_single_rows(q, dim, type_):
    c = Case(LENS, 2, dim, 32, seed=dim).on_gpu(q)
    out = both(q, c, 6, None, type_)
    assert not out[0].any()  # a slot without positions


@pytest.mark.parametrize("dim,type_,group", [(64, "f32", 2), (128, "bf16", 4), (256, "f32", 1), (256, "bf16", 3), (128, "f32", 5), (64, "f16", 7)])
@pytest.mark.parametrize("n,length", [(127, 127), (128, 300), (129, 129), (255, 256), (256, 700), (257, 320), (600, 601)])
def test_rows_around_the_tiles(q, dim, type_, group, n, length):
    c = Case([length], 1, dim, 64, seed=n + dim).on_gpu(q)
    both(q, c, group, [n], type_)


def test_rows_before_a_sequences_start_see_nothing(q):
    c = Case([3, 10, 0], 2, 128, 32, seed=1).on_gpu(q)
    for type_ in ("f32", "bf16"):
        out = both(q, c, 4, [9, 300, 5], type_)
        assert not out[:6].any() and not out[9:299].any() and not out[309:].any()


@pytest.mark.parametrize("dim,type_,heads,group", [(64, "f32", 1, 2), (128, "bf16", 1, 4), (256, "f32", 1, 1), (256, "f16", 1, 2)])
def test_long_sequences_beside_short_ones(q, dim, type_, heads, group):
    # pieces of one tile on every SM
    c = Case([20011, 3, 700], heads, dim, 64, seed=8).on_gpu(q)
    both(q, c, heads * group, [5, 3, 200], type_)


@pytest.mark.parametrize("dim,type_,length,n", [
    (128, "f16", 2 ** 18 + 77, 3), (256, "f32", 2 ** 16 + 5, 3), (128, "f32", 2 ** 16 + 5, 2), (64, "f32", 2 ** 17, 1),
    (256, "bf16", 2 ** 18 + 1, 2), (64, "bf16", 2 ** 29 + 77, 1)])
def test_positions_without_end(q, dim, type_, length, n):
    # A table that names one page over and over: the attention of a page whose positions count as often as they are named.
    # Each of 152 heads is a piece of its own, whose sums are taken over every 512 positions (float32) or 65536: between,
    # 2 * 512 / 16 or 65536 / 16 steps lose 2^-24 each, and a join rounds the mean, what is added, both factors and the sum,
    # 2^-22 in all. The longest takes the SMs some seconds.
    heads, tokens, width = 152, 256, -(-length // 256)
    c = Case([tokens], heads, dim, tokens, seed=23).on_gpu(q)
    page = int(c.table[0, 0])
    x = rows_tensor(c.rng.normal(size=(n, heads * dim)), TYPES[type_])
    out = torch.full_like(x, float("nan"))
    table = torch.full((1, width), page, dtype=torch.int32, device="cuda")
    lens, start = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([length], [0, n]))
    q.apr_kv8_prefill_attention(c.cache, table, lens, x, out, heads, row_start=start)
    q.apr_stream_status()
    k, v = (c.host[w][page].astype(np.float64) * c.host[s][page][:, None, None] for w, s in (("K", "k_scale"), ("V", "v_scale")))
    score = np.einsum("ngd,gjd->ngj", as_f32(x).astype(np.float64).reshape(n, heads, dim), k) / np.sqrt(dim)
    reach = np.einsum("ngd,gjd->ngj", np.abs(as_f32(x).astype(np.float64).reshape(n, heads, dim)), np.abs(k)).max(-1) / np.sqrt(dim)
    sees = length - n + 1 + np.arange(n)
    count = (sees[:, None] - np.arange(tokens) + tokens - 1) // tokens
    p = np.exp(score - score.max(-1, keepdims=True)) * count[:, None, :]
    p /= p.sum(-1, keepdims=True)
    want, size, vmax = np.einsum("ngj,gjd->ngd", p, v), np.einsum("ngj,gjd->ngd", p, np.abs(v)), np.abs(v).max()
    half, fold = torch.finfo(TYPES[type_]).eps / 2, 512 if type_ == "f32" else 65536
    tol = (2 * dim * 2.0 ** -24 * reach + 2.0 ** -17)[..., None] * 2 * vmax + half * np.abs(want)
    tol += (length / fold * 2.0 ** -22 + (0 if type_ == "f32" else 2.0 ** -11 + 2.0 ** -12)) * size + tokens * 2.0 ** -30 * vmax
    y = as_f32(out).astype(np.float64).reshape(want.shape)
    assert (np.abs(y - want) <= tol).all(), float((np.abs(y - want) / tol).max())


@pytest.mark.parametrize("type_", ["f32", "bf16"])
def test_many_sequences(q, type_):
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 90, 700)
    rows = np.minimum(rng.integers(0, 9, 700), lens)
    rows[100:200] = 0
    c = Case(list(lens), 1, 64, 32, seed=9).on_gpu(q)
    both(q, c, 2, list(rows), type_)


def test_thousands_of_sequences_and_default_sizes(q):
    rng = np.random.default_rng(10)
    lens = rng.integers(0, 40, 3001)
    rows = np.minimum(rng.integers(0, 4, 3001), lens)
    c = Case(list(lens), 1, 64, 32, seed=10).on_gpu(q)
    both(q, c, 3, list(rows), "f16", max_rows=3, max_len=39)
    both(q, c, 3, list(rows), "f16")


def test_rows_of_no_sequence_are_left_alone(q):
    # packed rows ahead of the first sequence's and behind the last one's, as in a padded batch
    c = Case([300, 40], 1, 128, 64, seed=11).on_gpu(q)
    x = torch.from_numpy(c.rng.normal(size=(60, 2 * 128)).astype(np.float32)).cuda()
    out = torch.full_like(x, 7.0)
    start = np.array([4, 30, 41], np.int32)
    x[:4], x[41:] = float("nan"), float("inf")
    q.apr_kv8_prefill_attention(c.cache, c.gtable, c.glens, x, out, 2, row_start=torch.from_numpy(start).cuda())
    q.apr_stream_status()
    assert bool((out[:4] == 7).all()) and bool((out[41:] == 7).all())
    check(c, out[4:41], x[4:41], 2, [26, 11])


def test_agrees_with_the_attention_of_few_rows(q):
    c = Case([900, 33, 257], 2, 128, 64, seed=12).on_gpu(q)
    for type_ in ("f32", "bf16"):
        out, qt = attend(q, c, 8, [5, 9, 1], type_)
        few = torch.empty_like(out)
        q.apr_kv8_attention(c.cache, c.gtable, c.glens, qt, few, 8, row_start=torch.from_numpy(starts([5, 9, 1])).cuda())
        q.apr_stream_status()
        torch.testing.assert_close(out, few, rtol=2 ** -6 if type_ == "bf16" else 1e-4, atol=2e-3 if type_ == "bf16" else 1e-5)


# ---------------------------------------------------------------- values out of the ordinary
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("type_", ["f32", "f16"])
def test_a_dominant_position_and_rising_scores(q, dim, type_):
    # scores that rise from page to page by more than any reference is kept for, one position that takes all, and
    # pages whose scales differ by 2^20, large ones last
    c = Case([500, 300, 400], 1, dim, 32, seed=13)
    c.host["K"][:] = c.rng.integers(-3, 4, c.host["K"].shape)
    for i in range(15):
        c.host["K"][c.table[0, i], 0, 5, 0] = 8 * (i + 1)
    c.host["K"][c.table[1, 4], 0, 3, 0] = 127
    c.host["v_scale"][c.table[2, ::2][:6]] = 2.0 ** -18
    c.host["v_scale"][c.table[2, 1::2][:6]] = 4.0
    c.host["k_scale"][c.table[0, :15]] = 0.5
    c.host["k_scale"][c.table[1, :9]] = 1.0
    c.on_gpu(q)
    for n in (1, 90):
        qh = np.zeros((3 * n, 2 * dim))
        qh[:, 0], qh[:, dim] = np.sqrt(dim), 3 * np.sqrt(dim)
        both(q, c, 2, [n] * 3, type_, qh=qh, frobenius=False)


@pytest.mark.parametrize("type_,rtol", [("f32", 1e-4), ("bf16", 2.0 ** -8 + 2.0 ** -10)])
def test_small_weights_of_many_positions_add_up(q, type_, rtol):
    # one weight of 1 beside 6000 of 3e-7: what they carry together is kept
    c = Case([6000], 1, 64, 64, seed=14)
    c.host["K"][:], c.host["V"][:] = 0, 100
    c.host["k_scale"][:], c.host["v_scale"][:] = 1.0, 1.0
    c.host["K"][c.table[0, 50], 0, 9, 0] = 100
    c.host["V"][c.table[0, 50], 0, 9, :] = 0
    c.on_gpu(q)
    qh = np.zeros((3, 64))
    qh[:, 0] = 8.0 * 12.0 / 100.0  # a score of 12 against 0 (a bf16 number or nearly)
    out, qt = attend(q, c, 1, [3], type_, qh=qh)
    want = oracle.kv8_attention(c.host, c.table, c.lens, [0, 3], as_f32(qt), 1)[0]
    np.testing.assert_allclose(as_f32(out), want[:, 0], rtol=rtol)


@pytest.mark.parametrize("type_", ["f32", "bf16"])
def test_custom_scale_and_zero_query(q, type_):
    c = Case([300, 77], 2, 128, 64, seed=15).on_gpu(q)
    both(q, c, 4, [140, 60], type_, scale=0.31, frobenius=False)
    both(q, c, 4, [140, 60], type_, qh=np.zeros((200, 4 * 128)))


@pytest.mark.parametrize("type_", ["f32", "bf16"])
def test_tiny_and_huge_queries(q, type_):
    c = Case([150, 150, 150], 1, 64, 32, seed=16)
    c.host["k_scale"][:] = 1e-12
    c.on_gpu(q)
    both(q, c, 1, None, type_, qh=c.rng.normal(size=(3, 64)) * np.array([[1e12], [1e-30], [1e10]]))


@pytest.mark.parametrize("dim,type_,lens", [(64, "f32", [300, 2500]), (256, "bf16", [70, 600]), (128, "f32", [400, 33])])
@pytest.mark.parametrize("exponent", [105, 115, -90])
def test_values_at_the_ends_of_the_range(q, dim, type_, lens, exponent):
    c = Case(lens, 1, dim, 64, seed=17)
    c.host["v_scale"][:] *= np.float32(2.0 ** exponent) / c.host["v_scale"].mean()
    c.host["V"][:] = np.abs(c.host["V"]) // 2 + 60
    c.on_gpu(q)
    both(q, c, 2, [20, 30], type_)


@pytest.mark.parametrize("dim,type_", [(64, "f32"), (128, "bf16"), (256, "f32"), (256, "f16")])
def test_pages_of_zero_scales(q, dim, type_):
    # pages whose rows were all zeros: their positions have scores of 0 and carry nothing; whatever codes stand in them
    c = Case([500], 1, dim, 32, seed=18)
    c.host["v_scale"][c.table[0, [0, 3, 4, 9]]] = 0
    c.host["k_scale"][c.table[0, [0, 2, 7]]] = 0
    c.on_gpu(q)
    both(q, c, 2, [77], type_)
    c.cache.v_scale.zero_()
    out, _ = attend(q, c, 2, [77], type_)
    assert not out.any()


def test_nan_and_infinite_queries_stay_in_their_row(q):
    c = Case([100, 400], 1, 128, 64, seed=19).on_gpu(q)
    qh = c.rng.normal(size=(60, 4 * 128))
    for type_ in ("f32", "f16", "bf16"):
        clean, _ = attend(q, c, 4, [20, 40], type_, qh=qh)
        spoilt = qh.copy()
        spoilt[1, 5], spoilt[2, 128 * 2 + 9], spoilt[59, 128 * 3], spoilt[30, 128 + 1] = np.nan, np.inf, -np.inf, np.nan
        out, _ = attend(q, c, 4, [20, 40], type_, qh=spoilt)
        bad = torch.zeros((60, 4), dtype=torch.bool, device="cuda")
        bad[1, 0] = bad[2, 2] = bad[59, 3] = bad[30, 1] = True
        assert torch.equal(torch.isnan(out.reshape(60, 4, 128)).all(-1), bad)
        assert torch.equal(out.reshape(60, 4, 128)[~bad], clean.reshape(60, 4, 128)[~bad])


@pytest.mark.parametrize("dim,type_", [(64, "bf16"), (128, "f32"), (256, "f32"), (128, "f16")])
def test_what_lies_past_a_length_does_not_matter(q, dim, type_):
    c = Case([33, 70, 300], 2, dim, 64, seed=20).on_gpu(q)
    qh = c.rng.normal(size=(110, 8 * dim))
    a, _ = attend(q, c, 8, [10, 50, 50], type_, qh=qh)
    for b, n in enumerate((33, 70, 300)):  # other codes behind the last position, NaN scales in pages that are not theirs
        page = int(c.table[b, n // 64])
        c.cache.K[page, :, n % 64:] = -128
        c.cache.V[page, :, n % 64:] = 127
    used = {int(p) for b in range(3) for p in c.table[b, : -(-int(c.lens[b]) // 64)]}
    for p in range(c.cache.K.shape[0]):
        if p not in used:
            c.cache.k_scale[p] = float("nan")
            c.cache.v_scale[p] = float("nan")
    b, _ = attend(q, c, 8, [10, 50, 50], type_, qh=qh)
    assert torch.equal(a, b)


@pytest.mark.parametrize("type_", ["f32", "bf16"])
def test_repeats_are_bitwise_the_same(q, type_):
    c = Case([5000, 40, 1300, 0, 77], 2, 128, 64, seed=21).on_gpu(q)
    qh = c.rng.normal(size=(361, 8 * 128))
    outs = [attend(q, c, 8, [300, 40, 20, 0, 1], type_, qh=qh)[0] for _ in range(4)]
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


# ---------------------------------------------------------------- streams, graphs, threads, what the device arrays say
def test_two_streams_at_once(q):
    cases = [Case([900, 33], 2, 128, 64, seed=s).on_gpu(q) for s in (30, 31)]
    streams = [torch.cuda.Stream() for _ in cases]
    qs = [torch.from_numpy(c.rng.normal(size=(300, 8 * 128)).astype(np.float32)).cuda() for c in cases]
    outs = [torch.empty_like(x) for x in qs]
    start = torch.from_numpy(starts([270, 30])).cuda()
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, x, out in zip(cases, streams, qs, outs):
            q.apr_kv8_prefill_attention(c.cache, c.gtable, c.glens, x, out, 8, row_start=start, stream=s)
    for s in streams:
        q.apr_stream_status(s)
    for c, x, out in zip(cases, qs, outs):
        check(c, out, x, 8, [270, 30])


def test_two_threads_attend_on_one_stream(q):
    stream = torch.cuda.Stream()
    cases = [Case([3000, 33], 2, 128, 64, seed=70).on_gpu(q), Case([40, 1700, 900], 2, 128, 64, seed=71).on_gpu(q)]
    rows = [[9, 30], [40, 3, 50]]
    xs = [torch.from_numpy(c.rng.normal(size=(sum(r), 8 * 128)).astype(np.float32)).cuda() for c, r in zip(cases, rows)]
    start = [torch.from_numpy(starts(r)).cuda() for r in rows]

    def call(i):
        def run(out):
            if out is None:
                return torch.full_like(xs[i], 9.0)
            q.apr_kv8_prefill_attention(cases[i].cache, cases[i].gtable, cases[i].glens, xs[i], out, 8, row_start=start[i], stream=stream)

        return run

    outs = both_at_once([call(0), call(1)], 100)
    q.apr_stream_status(stream)
    for i, c in enumerate(cases):
        check(c, outs[i][0], xs[i], 8, rows[i])
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])


def test_lengths_and_rows_followed_by_a_replayed_graph(q):
    # one captured call of a padded batch, replayed as rows and lengths change
    c = Case([500, 700, 300], 1, 128, 64, seed=32).on_gpu(q)
    x = torch.from_numpy(c.rng.normal(size=(400, 4 * 128)).astype(np.float32)).cuda()
    out, start = torch.full_like(x, 7.0), torch.zeros(4, dtype=torch.int32, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        q.apr_kv8_prefill_attention(c.cache, c.gtable, c.glens, x, out, 4, row_start=start)
    for lens, rows in (([500, 700, 300], [300, 1, 99]), ([1, 0, 300], [1, 0, 300]), ([64, 700, 2], [10, 256, 2]), ([500, 5, 5], [0, 0, 0])):
        c.lens[:] = lens
        c.glens.copy_(torch.from_numpy(c.lens))
        start.copy_(torch.from_numpy(starts(rows)))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        n = sum(rows)
        assert bool((out[n:] == 7).all())
        if n:
            check(c, out[:n], x[:n], 4, rows)
    q.apr_stream_status()


@pytest.mark.parametrize("what", ["page", "length", "negative", "row_start", "past", "max_rows", "max_len", "last"])
def test_what_the_device_arrays_say_is_checked(q, what):
    c = Case([70, 90, 100], 2, 64, 32, seed=33).on_gpu(q)
    x = torch.from_numpy(c.rng.normal(size=(30, 4 * 64)).astype(np.float32)).cuda()
    start, more = np.array([0, 10, 20, 30], np.int32), {}
    if what == "page":
        c.gtable[0, 1] = c.cache.K.shape[0]
    elif what == "length":
        c.glens[0] = 1 << 28
    elif what == "negative":
        c.glens[0] = -5
    elif what == "row_start":
        start[1] = -3
    elif what == "past":
        start[3] = 31
    elif what == "max_rows":
        more = {"max_rows": 9}
    elif what == "max_len":
        more = {"max_len": 95}
    elif what == "last":
        c.glens[2], start[3] = 1 << 20, 20  # a sequence without rows
    out = torch.full((34, 4 * 64), 7.0, device="cuda")
    q.apr_kv8_prefill_attention(c.cache, c.gtable, c.glens, x, out[2:32], 4, row_start=torch.from_numpy(start).cuda(), **more)
    bad_index(q)
    assert bool((out[:2] == 7).all()) and bool((out[32:] == 7).all())
    fine = {"page": 1, "length": 1, "negative": 1, "max_len": 0, "last": 1}.get(what)
    if fine is not None:  # the other sequences' rows are right all the same
        one = Case([70, 90, 100], 2, 64, 32, seed=33)
        want = oracle.kv8_attention(one.host, one.table[fine:fine + 1], one.lens[fine:fine + 1], [0, 10], as_f32(x[10 * fine:10 * fine + 10]), 4)[0]
        y = as_f32(out[2 + 10 * fine:12 + 10 * fine]).reshape(want.shape)
        assert np.linalg.norm(y - want) <= EXACT_REL * np.linalg.norm(want)
    q.apr_kv8_prefill_attention(c.cache, c.gtable[1:2], c.glens[1:2].clamp(0, 90), x[:10], out[:10], 4, row_start=torch.tensor([0, 10], dtype=torch.int32, device="cuda"))
    q.apr_stream_status()


def test_row_ranges_that_overlap_are_counted_without_harm(q):
    # every sequence claims all rows; the next falls: flagged or not, no access outside the arrays
    c = Case([400] * 40, 1, 64, 64, seed=34).on_gpu(q)
    x = torch.randn((300, 4 * 64), device="cuda")
    out = torch.full((304, 4 * 64), 7.0, device="cuda")
    start = torch.tensor([0, 300] * 20 + [0], dtype=torch.int32, device="cuda")
    q.apr_kv8_prefill_attention(c.cache, c.gtable, c.glens, x, out[2:302], 4, row_start=start)
    bad_index(q)
    assert bool((out[:2] == 7).all()) and bool((out[302:] == 7).all())


def test_tables_of_no_pages(q):
    cache = q.Kv8Cache.allocate(4, 2, 64, 32)
    table, lens = torch.empty((2, 0), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.ones((2, 4 * 64), device="cuda")
    out = torch.ones_like(x)
    q.apr_kv8_prefill_attention(cache, table, lens, x, out, 4)
    q.apr_stream_status()
    assert not out.any()


@pytest.mark.parametrize("type_", ["f32", "bf16"])
def test_pages_past_4_gib(q, type_):
    # the same attention over the last pages of two arrays of 4.3e9 codes and over the first of two small ones: the same bits
    pages, heads, tokens, dim, n = 8200, 8, 256, 256, 700
    assert (pages - 8) * heads * tokens * dim >= 1 << 32
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    gen = torch.Generator("cuda").manual_seed(91)
    k, v = (torch.randn((n, heads * dim), generator=gen, device="cuda") for _ in range(2))
    x = torch.randn((90, heads * dim), generator=gen, device="cuda").to(TYPES[type_])
    outs = []
    for count in (pages, 8):
        cache = q.Kv8Cache.allocate(count, heads, dim, tokens)
        table = torch.tensor([[count - 1, count - 6, count - 3]], dtype=torch.int32, device="cuda")
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        q.apr_kv8_append(cache, table, lens, k, v, row_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        outs.append(torch.empty_like(x))
        q.apr_kv8_prefill_attention(cache, table, lens, x, outs[-1], heads, row_start=torch.tensor([0, 90], dtype=torch.int32, device="cuda"))
        q.apr_stream_status()
    assert torch.equal(*outs) and bool(outs[0].any())


def test_the_time_does_not_grow_with_the_sequences_that_have_no_rows(q):
    # one chunk alone, and as the last of 4000 sequences: a search of the rows, no look at every sequence by every thread
    cache = q.Kv8Cache.allocate(40, 4, 128, 64)
    x = torch.randn((512, 16 * 128), device="cuda").to(torch.bfloat16)
    out, times = torch.empty_like(x), []
    for count in (1, 4000):
        table = torch.arange(40, dtype=torch.int32, device="cuda").repeat(count, 1)
        lens = torch.full((count,), 2500, dtype=torch.int32, device="cuda")
        start = torch.zeros(count + 1, dtype=torch.int32, device="cuda")
        start[-1] = 512
        times.append(us_of(lambda: q.apr_kv8_prefill_attention(cache, table, lens, x, out, 16, row_start=start), 15))
    q.apr_stream_status()
    assert times[1] <= 2 * times[0] + 20, times


# ---------------------------------------------------------------- as they are used together
@pytest.mark.parametrize("type_", ["f32", "bf16"])
def test_a_prompt_in_chunks_is_the_prompt_at_once(q, type_):
    # rotation and append of each chunk, then its attention: float64 attention over the rows read back from the cache, which
    # are those that one append of the whole prompt leaves, but for pages whose scale a later chunk raised
    heads, kv, dim, n = 8, 2, 128, 700
    rng = np.random.default_rng(40)
    qkv = torch.from_numpy(rng.normal(size=(n, (heads + 2 * kv) * dim))).cuda().to(TYPES[type_])
    inv = torch.from_numpy((1.0 / 10000.0 ** (np.arange(dim // 2) / (dim // 2))).astype(np.float32)).cuda()
    table = torch.empty((1024, dim // 2, 2), device="cuda")
    q.apr_rope_table(inv, table)
    rope, norm = q.Rope(table), torch.ones(dim, device="cuda")
    cache, pages = q.Kv8Cache.allocate(12, kv, dim, 64), torch.randperm(12, device="cuda").int()[None, :11].contiguous()
    outs, at = [], 0
    for chunk in (300, 1, 128, 71, 200):
        part = qkv[at:at + chunk].clone()
        at += chunk
        lens, start = torch.tensor([at], dtype=torch.int32, device="cuda"), torch.tensor([0, chunk], dtype=torch.int32, device="cuda")
        qx, k, v = part.split((heads * dim, kv * dim, kv * dim), 1)
        q.apr_rope_kv8_append(cache, pages, lens, rope, k, v, k_norm=norm, q=qx, q_out=qx, num_heads=heads, q_norm=norm, eps=1e-6, row_start=start)
        out = torch.empty((chunk, heads * dim), dtype=TYPES[type_], device="cuda")
        q.apr_kv8_prefill_attention(cache, pages, lens, qx, out, heads, row_start=start)
        kb, vb = (torch.empty((at, kv * dim), device="cuda") for _ in range(2))
        q.apr_kv8_read(cache, pages, lens, kb, vb, row_start=torch.tensor([0, at], dtype=torch.int32, device="cuda"))
        K, V = (t.double().view(at, kv, dim).repeat_interleave(heads // kv, 1) for t in (kb, vb))
        scores = torch.einsum("ihd,jhd->hij", qx.double().reshape(chunk, heads, dim), K) / dim ** 0.5
        hidden = torch.arange(at, device="cuda") > torch.arange(at - chunk, at, device="cuda")[:, None]
        want = torch.einsum("hij,jhd->ihd", torch.softmax(scores.masked_fill(hidden, -np.inf), -1), V).reshape(chunk, -1)
        rel = float((out.double() - want).norm() / want.norm())
        assert rel <= (EXACT_REL if type_ == "f32" else 2.0 ** -8), rel
        outs.append(out)
    q.apr_stream_status()
    # the whole prompt at once: rotated rows and cache differ by roundings of raised scales alone, half a step of 1 / 127 of a
    # page's largest value each: a few hundredths at most
    whole, cache2 = qkv.clone(), q.Kv8Cache.allocate(12, kv, dim, 64)
    qx, k, v = whole.split((heads * dim, kv * dim, kv * dim), 1)
    lens, start = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q.apr_rope_kv8_append(cache2, pages, lens, rope, k, v, k_norm=norm, q=qx, q_out=qx, num_heads=heads, q_norm=norm, eps=1e-6, row_start=start)
    out = torch.empty((n, heads * dim), dtype=TYPES[type_], device="cuda")
    q.apr_kv8_prefill_attention(cache2, pages, lens, qx, out, heads, row_start=start)
    q.apr_stream_status()
    got = torch.cat(outs).double()
    assert float((got - out.double()).norm() / out.double().norm()) <= 0.05
