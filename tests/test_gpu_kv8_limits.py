"""GPU tests of the 8-bit paged KV cache at the limits of its arguments
(include/apr_kv8.h): what the device arrays may say, sizes left to their
defaults, several host threads, places past 2^32 bytes.

Values are compared with the float64 oracle as tests/test_gpu_kv8.py derives it.
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv8 import Case, as_f32, assert_attention, assert_weights, attend, bad_index, rows_tensor, starts

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


# ---------------------------------------------------------------- ragged batches, max_rows left out
def us_of(call, calls=5):
    """The median time of a call on the GPU."""
    call()
    times = []
    for _ in range(calls):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return sorted(times)[calls // 2]


@pytest.mark.parametrize("dim,heads,group,max_rows", [(64, 2, 2, 0), (64, 1, 3, 40), (256, 1, 2, 0), (128, 1, 9, 0)])
def test_ragged_rows_over_a_wide_table(q, dim, heads, group, max_rows):
    # segments that are divided, sequences of 0 to 3 rows beside one window of 40, one sequence long enough for every CTA
    rng = np.random.default_rng(dim + group)
    lens = rng.integers(0, 90, 150)
    rows = np.minimum(rng.integers(0, 4, 150), lens)
    lens[70], rows[70], lens[149], rows[149], rows[:2], rows[100:105] = 1500, 40, 2000, 2, 0, 0
    c = Case(list(lens), heads, dim, 64, seed=60).on_gpu(q)
    out, w, ref = attend(q, c, heads * group, rows=list(rows), weights=True, max_rows=max_rows)
    assert_attention(c, out, ref)
    assert_weights(c, w, ref)
    out, _, ref = attend(q, c, heads * group, rows=list(rows), type_="bf16", max_rows=max_rows)
    assert_attention(c, out, ref, "bf16")


def test_thousands_of_sequences_find_their_rows(q):
    # more sequences than one round of the search looks at, ranges of rows that begin at the same place
    rng = np.random.default_rng(61)
    lens = rng.integers(0, 40, 2100)
    rows = np.minimum(rng.integers(0, 3, 2100), lens)
    lens[2050], rows[2050] = 1400, 3
    rows[500:900] = 0
    c = Case(list(lens), 1, 64, 32, seed=61).on_gpu(q)
    out, _, ref = attend(q, c, 1, rows=list(rows))
    assert_attention(c, out, ref)


@pytest.mark.parametrize("rows,max_rows", [([2] * 1024, 0), ([400] + [1] * 600, 400)])
def test_the_time_does_not_grow_with_the_rows_that_a_sequence_may_have(q, rows, max_rows):
    # the same pairs as one sequence each take no more than a few times as long however they are spread over sequences: a
    # grid of the most rows by all sequences would take some 20 ms where the work is 100 us
    count, total = len(rows), sum(rows)
    cache = q.Kv8Cache.allocate(20, 4, 64, 64)
    table = torch.zeros((count, 20), dtype=torch.int32, device="cuda")
    lens = torch.full((count,), 450, dtype=torch.int32, device="cuda")
    x = torch.randn((total, 32 * 64), device="cuda")
    out, start = torch.empty_like(x), torch.from_numpy(starts(rows)).cuda()
    ragged = us_of(lambda: q.apr_kv8_attention(cache, table, lens, x, out, 32, row_start=start, max_rows=max_rows))
    table1, lens1 = (t.repeat_interleave(torch.tensor(rows, device="cuda"), 0) for t in (table, lens))
    single = us_of(lambda: q.apr_kv8_attention(cache, table1, lens1, x, out, 32))
    q.apr_stream_status()
    assert ragged <= 4 * single, (ragged, single)


# ---------------------------------------------------------------- host threads that share a stream
def both_at_once(calls, times):
    """Two threads make their calls `times` times, both on one stream: the outputs of each."""
    import threading

    ready, outs, failed = threading.Barrier(2), [[], []], []

    def work(i):
        try:
            ready.wait()
            for k in range(times):
                calls[i](outs[i][k])
        except Exception as e:  # (an assertion of the main thread's)
            failed.append(e)

    for i, call in enumerate(calls):
        outs[i] = [call(None) for _ in range(times)]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    return outs


def test_two_threads_attend_on_one_stream(q):
    # each call's second launch reads what its first left in the stream's scratch
    stream = torch.cuda.Stream()
    cases = [Case([3000, 33], 2, 128, 64, seed=70).on_gpu(q), Case([40, 1700, 900], 2, 128, 64, seed=71).on_gpu(q)]
    rows = [torch.from_numpy(c.rng.normal(size=(len(c.lens), 8 * 128)).astype(np.float32)).cuda() for c in cases]

    def call(i):
        c, x = cases[i], rows[i]

        def run(out):
            if out is None:
                return torch.full_like(x, 9.0), torch.full((len(c.lens), 2, c.table.shape[1] * 64), 9.0, device="cuda")
            q.apr_kv8_attention(c.cache, c.gtable, c.glens, x, out[0], 8, weights=out[1], stream=stream)

        return run

    outs = both_at_once([call(0), call(1)], 200)
    q.apr_stream_status(stream)
    for i, c in enumerate(cases):
        ref = oracle.kv8_attention(c.host, c.table, c.lens, None, as_f32(rows[i]), 8)
        assert_attention(c, outs[i][0][0], ref)
        assert_weights(c, outs[i][0][1], ref)
        for out, w in outs[i][1:]:
            assert torch.equal(out, outs[i][0][0]) and torch.equal(w, outs[i][0][1])


def test_two_threads_multiply_on_one_stream(q):
    # the GEMM's fp16 copy of its rows, the FFN sublayer's normed rows and activations
    import synth
    from gpu_util import assert_f16_leg, dev

    stream = torch.cuda.Stream()
    cases = [synth.make_case(synth.Q4_0, 1024, 2048, T, seed=72 + T) for T in (64, 200)]
    ins = [(dev(c["W"]), dev(c["X"])) for c in cases]

    def call(i):
        W, X = ins[i]

        def run(out):
            if out is None:
                return torch.full((X.shape[0], 1024), 9.0, device="cuda")
            q.apr_qgemm(synth.Q4_0, W, 1024, 2048, X, X.shape[0], out, stream=stream)

        return run

    outs = both_at_once([call(0), call(1)], 200)
    q.apr_stream_status(stream)
    for c, ys in zip(cases, outs):
        assert_f16_leg(ys[0].cpu().numpy(), oracle.qgemm_f64(synth.Q4_0, c["W"], 1024, 2048, c["X"]))
        assert all(torch.equal(y, ys[0]) for y in ys[1:])
    layers = []
    for i in range(2):
        ws = [dev(synth.quantize(synth.Q4_0, synth.weight_f32(n, k, 80 + 3 * i + j))) for j, (n, k) in enumerate(((1024, 512), (1024, 512), (512, 1024)))]
        layers.append((ws, torch.ones(512, device="cuda"), dev(synth.activations(40 + 60 * i, 512, 90 + i))))

    def sublayer(i):
        ws, norm, X = layers[i]

        def run(out):
            if out is None:
                return X.clone()
            q.apr_ffn_sublayer(synth.Q4_0, *ws, 512, 1024, out.shape[0], norm, 1e-6, out, stream=stream)

        return run

    outs = both_at_once([sublayer(0), sublayer(1)], 100)
    q.apr_stream_status(stream)
    for i, ys in enumerate(outs):
        alone = layers[i][2].clone()
        q.apr_ffn_sublayer(synth.Q4_0, *layers[i][0], 512, 1024, alone.shape[0], layers[i][1], 1e-6, alone)
        assert all(torch.equal(y, alone) for y in ys)


# ---------------------------------------------------------------- values out of the ordinary
@pytest.mark.parametrize("lens", [[70, 33], [70, 1700], [2100, 1]])  # whole and divided segments
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_a_bad_row_gives_no_weight_to_positions_behind_it(q, bad, lens):
    c = Case(lens, 2, 64, 64, seed=80, extra_width=0).on_gpu(q)
    rows = [min(5, n) for n in lens]
    qh = c.rng.normal(size=(sum(rows), 4 * 64))
    qh[1, 70] = bad  # the second row's head 1, of the first KV head: it does not see the last three positions
    qt, out = rows_tensor(qh, torch.float32), torch.empty((sum(rows), 4 * 64), device="cuda")
    w = torch.full((2, 2, c.table.shape[1] * 64), 3.0, device="cuda")
    q.apr_kv8_attention(c.cache, c.gtable, c.glens, qt, out, 4, row_start=torch.from_numpy(starts(rows)).cuda(), weights=w)
    q.apr_stream_status()
    sees = lens[0] - 3
    finite = np.where(np.isfinite(qh), as_f32(qt), 0.0)  # (whatever the row gives, it gives to the first `sees` positions)
    _, want, reach = oracle.kv8_attention(c.host, c.table, c.lens, starts(rows), finite, 4)
    want[0, 0, :sees] = np.nan
    got = w.cpu().numpy()
    tol = (4 * 64 * 2.0 ** -24 * float(reach.max()) + 2.0 ** -20) * max(1.0, float(np.nanmax(want)))
    for b, n in enumerate(lens):
        np.testing.assert_allclose(got[b, :, :n], want[b, :, :n], rtol=0, atol=tol)
        assert not got[b, :, n:].any()


@pytest.mark.parametrize("dim,type_,lens", [(64, "f32", [300, 2500]), (256, "bf16", [70, 600]), (128, "f32", [400, 33])])
@pytest.mark.parametrize("exponent", [105, 115, -90])
def test_values_at_the_ends_of_the_range(q, dim, type_, lens, exponent):
    # values of 10^33 and 10^36, all of one sign, whose sums over a few hundred positions no float32 holds; and of 10^-26
    c = Case(lens, 1, dim, 64, seed=81)
    c.host["v_scale"][:] *= np.float32(2.0 ** exponent) / c.host["v_scale"].mean()
    c.host["V"][:] = np.abs(c.host["V"]) // 2 + 60
    c.on_gpu(q)
    out, _, ref = attend(q, c, 2, type_=type_)
    assert_attention(c, out, ref, type_)


@pytest.mark.parametrize("dim,heads,group,rows", [(64, 2, 4, 1), (128, 1, 8, 2), (128, 2, 3, 6), (256, 1, 4, 2)])
def test_weights_around_the_length_from_which_segments_are_divided(q, dim, heads, group, rows):
    # one segment a KV head (up to 16 pairs) and more, at lengths on either side of 192 and 512 x 128 codes
    lens = [512 * 128 // dim, 512 * 128 // dim - 1, 192 * 128 // dim + 1, 192 * 128 // dim, 7]
    c = Case(lens, heads, dim, 32, seed=90).on_gpu(q)
    for longest in (192 * 128 // dim, 192 * 128 // dim + 1, 512 * 128 // dim):
        c.lens[:] = np.minimum(lens, longest)
        c.glens.copy_(torch.from_numpy(c.lens))
        out, w, ref = attend(q, c, heads * group, rows=[rows] * 5, weights=True, max_rows=rows, max_len=longest)
        assert_attention(c, out, ref)
        assert_weights(c, w, ref)


# ---------------------------------------------------------------- places past 2^32
def test_every_operator_on_pages_past_4_gib(q):
    # the same steps on the last pages of two arrays of 4.3e9 codes and on the first of two small ones: the same bits
    pages, heads, tokens, dim, n = 8200, 8, 256, 256, 700
    assert (pages - 8) * heads * tokens * dim >= 1 << 32
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    gen = torch.Generator("cuda").manual_seed(91)
    k, v, x = (torch.randn((rows, heads * dim), generator=gen, device="cuda") for rows in (n, n, 2))
    weights = torch.rand((1, heads, 3 * tokens), generator=gen, device="cuda")
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    results = []
    for count in (pages, 8):
        first = count - 8
        cache = q.Kv8Cache.allocate(count, heads, dim, tokens)
        table, lens = ints([[first + 7, first + 2, first + 5]]), ints([n])
        q.apr_kv8_append(cache, table, lens, k, v, row_start=ints([0, n]))
        q.apr_kv8_append(cache, table, lens, 2 * k[n - 40:], 2 * v[n - 40:], row_start=ints([0, 40]))  # raises the last page's scales
        kb, vb, out, w = torch.empty_like(k), torch.empty_like(v), torch.empty_like(x), torch.empty_like(weights)
        q.apr_kv8_read(cache, table, lens, kb, vb, row_start=ints([0, n]))
        q.apr_kv8_attention(cache, table, lens, x, out, heads, row_start=ints([0, 2]), weights=w)
        table_out, lens_out = torch.empty_like(table), torch.empty_like(lens)
        kept, wo = torch.empty((1, heads, 300), dtype=torch.int32, device="cuda"), torch.empty((1, heads, 300), device="cuda")
        q.apr_kv8_evict(cache, table, lens, weights, 300, 20, ints([[first + 6, first + 3]]), table_out, lens_out, wo, kept)
        q.apr_stream_status()
        ends = [a[first:].clone() for a in (cache.K, cache.V, cache.k_scale, cache.v_scale)]
        results.append(ends + [kb, vb, out, w, kept, wo, lens_out, table_out - first * (table_out >= 0).int()])
        assert all(bool(e[p].any()) for e in ends for p in (2, 3, 5, 6, 7))
        if first:  # nothing went anywhere else
            for a in (cache.K, cache.V):
                assert not any(bool(a[i:min(i + 512, first)].view(torch.int64).any()) for i in range(0, first, 512))
            assert not cache.k_scale[:first].any() and not cache.v_scale[:first].any()
    for big, small in zip(*results):
        assert torch.equal(big, small)


# ---------------------------------------------------------------- appends to many sequences
@pytest.mark.parametrize("tokens,before", [(32, 0), (64, 3), (32, 100)])
def test_append_to_many_ragged_sequences(q, tokens, before):
    # rows over up to four pages, sequences without rows or positions, packed rows ahead of the first sequence's
    rng = np.random.default_rng(tokens + before)
    lens = rng.integers(0, 200, 1500)
    rows = np.where(rng.random(1500) < 0.3, 0, np.minimum(rng.integers(0, 100, 1500), lens))
    rows[7] = lens[7] + 5  # more rows than positions
    c = Case(list(lens), 1, 64, tokens, seed=100).on_gpu(q)
    start = starts(rows) + np.int32(before)
    x = [c.rng.normal(size=(int(start[-1]) + 9, 64)).astype(np.float32) for _ in range(2)]
    q.apr_kv8_append(c.cache, c.gtable, c.glens, *(torch.from_numpy(a).cuda() for a in x), row_start=torch.from_numpy(start).cuda())
    q.apr_stream_status()
    c.assert_cache(oracle.kv8_append(c.host, c.table, c.lens, start, *x))


def test_the_time_of_an_append_does_not_grow_with_the_square_of_the_sequences(q):
    # 2 rows of each of 8000 sequences take no more than twice as long as one of each of 16000: 6 times where each CTA looks at all
    cache = q.Kv8Cache.allocate(16000, 8, 64, 32)
    table = torch.arange(16000, dtype=torch.int32, device="cuda").view(16000, 1)
    lens = torch.full((16000,), 20, dtype=torch.int32, device="cuda")
    x = torch.randn((16000, 8 * 64), device="cuda")
    start = torch.arange(0, 16001, 2, dtype=torch.int32, device="cuda")
    two = us_of(lambda: q.apr_kv8_append(cache, table[:8000], lens[:8000], x, x, row_start=start))
    one = us_of(lambda: q.apr_kv8_append(cache, table, lens, x, x))
    q.apr_stream_status()
    assert two <= 2 * one, (two, one)


@pytest.mark.parametrize("what", ["length", "row_start", "max_rows"])
def test_append_looks_at_every_sequence(q, what):
    # the last of 300 sequences, one without rows, says something that cannot be
    c = Case([10] * 300, 1, 64, 32, seed=101).on_gpu(q)
    start, more = torch.from_numpy(starts([2] * 299 + [0])).cuda(), {}
    if what == "length":
        c.glens[299] = 1 << 20
    elif what == "row_start":
        start[300] = 597
    else:
        more = {"max_rows": 1}
    x = torch.ones((598, 64), device="cuda")
    q.apr_kv8_append(c.cache, c.gtable, c.glens, x, x, row_start=start, **more)
    bad_index(q)


@pytest.mark.parametrize("heads,group,dim,rows", [(8, 4, 128, 1), (8, 2, 64, 3)])
def test_max_rows_left_out_costs_no_time(q, heads, group, dim, rows):
    # the same rows of each sequence: the tiles are those that max_rows gives (1.3 times as long with those for all rows)
    count, tokens = 48, 6000
    cache = q.Kv8Cache.allocate(count * 94, heads, dim, 64)
    table = torch.arange(count * 94, dtype=torch.int32, device="cuda").view(count, 94)
    lens = torch.full((count,), tokens, dtype=torch.int32, device="cuda")
    x = torch.randn((rows * count, heads * group * dim), device="cuda")
    start = torch.arange(0, rows * count + 1, rows, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(x) for _ in range(2)]
    given, left_out = (us_of(lambda: q.apr_kv8_attention(cache, table, lens, x, o, heads * group, row_start=start, max_rows=m), 15)
                       for o, m in zip(outs, (rows, 0)))
    q.apr_stream_status()
    assert left_out <= 1.15 * given, (left_out, given)
    assert torch.equal(*outs)


@pytest.mark.parametrize("accumulate", [False, True])
def test_tables_of_no_pages(q, accumulate):
    # two slots that hold nothing yet: every operator runs, rows read as zeros, weights stay or are zeros
    cache = q.Kv8Cache.allocate(4, 2, 64, 32)
    table, lens = torch.empty((2, 0), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    k, v, x = (torch.ones((2, n * 64), device="cuda") for n in (2, 2, 4))
    out, kb, vb, w = torch.ones_like(x), torch.ones_like(k), torch.ones_like(v), torch.full((2, 2, 7), 3.0, device="cuda")
    q.apr_kv8_append(cache, table, lens, k, v)
    q.apr_kv8_read(cache, table, lens, kb, vb)
    q.apr_kv8_attention(cache, table, lens, x, out, 4, weights=w, accumulate=accumulate)
    table_out, lens_out = torch.empty_like(table), torch.ones_like(lens)
    kept, wo = torch.ones((2, 2, 5), dtype=torch.int32, device="cuda"), torch.ones((2, 2, 5), device="cuda")
    q.apr_kv8_evict(cache, table, lens, w, 5, 2, torch.zeros((2, 1), dtype=torch.int32, device="cuda"), table_out, lens_out, wo, kept)
    q.apr_stream_status()
    assert not any(bool(t.any()) for t in (out, kb, vb, lens_out, wo, cache.K, cache.V, cache.k_scale, cache.v_scale))
    assert bool((kept == -1).all()) and bool((w == (3.0 if accumulate else 0.0)).all())
