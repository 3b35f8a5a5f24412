"""GPU parity of the 8-bit paged KV cache (include/apr_kv8.h) against its float64
oracle.

Append, read and eviction are bit for bit: codes, scales, positions and the
values read back are functions that both sides decide exactly.

Attention, per element, against the exact attention of the cache's values: with
R the largest sum of |scale q_c k_c| over a position that a row sees, a score is
off by at most d 2^-24 R (d float32 additions in any order; the split of q is
finer) and a weight by twice that relatively; 2^-17 more allows for the
exponentials (2^-21) and for a hundred float32 additions in a row. A mean of
values bounded by vmax moves by at most twice that of vmax. A 16-bit
output adds half a step of its type, finfo.eps / 2 relatively. Over all elements
a float32 result is held to the relative Frobenius bound of the library's exact
leg, 1e-5, where scores stay within the range of unit-variance rows.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EXACT_REL = 1e-5


def starts(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


class Case:
    """A cache of random codes whose tables name its pages in random order, on both sides."""

    def __init__(self, lens, heads=2, dim=128, tokens=64, seed=0, spare=2, extra_width=1):
        rng = self.rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        self.heads, self.dim, self.tokens = heads, dim, tokens
        width = max(-(-int(n) // tokens) for n in lens) + extra_width
        used = sum(-(-int(n) // tokens) for n in lens)
        pages = used + spare
        order = rng.permutation(pages)
        self.table = np.full((len(lens), width), -7, np.int32)  # entries past a length are never looked at
        at = 0
        for b, n in enumerate(lens):
            count = -(-int(n) // tokens)
            self.table[b, :count] = order[at:at + count]
            at += count
        self.free = order[at:]
        shape = (pages, heads, tokens, dim)
        self.host = {"K": np.clip(np.rint(rng.normal(0, 36, shape)), -127, 127).astype(np.int8),
                     "V": np.clip(np.rint(rng.normal(0, 36, shape)), -127, 127).astype(np.int8),
                     "k_scale": (np.exp(0.3 * rng.normal(size=shape[:2])) * 0.028).astype(np.float32),
                     "v_scale": (np.exp(0.3 * rng.normal(size=shape[:2])) * 0.028).astype(np.float32)}

    def on_gpu(self, q):
        self.cache = q.Kv8Cache(*(torch.from_numpy(self.host[n].copy()).cuda() for n in ("K", "V", "k_scale", "v_scale")))
        self.gtable, self.glens = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda()
        return self

    def assert_cache(self, want):
        for name in ("K", "V", "k_scale", "v_scale"):
            np.testing.assert_array_equal(getattr(self.cache, name).cpu().numpy(), want[name], err_msg=name)


def rows_tensor(x, dtype, pad=0):
    """[rows][width] of a type on the GPU, the rows `pad` elements further apart than dense."""
    wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, : x.shape[1]] = torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dtype)
    return wide[:, : x.shape[1]]


def as_f32(t):
    return t.float().cpu().numpy()


# ---------------------------------------------------------------- append and read
# (lens with the rows, rows; None: one row a sequence)
APPENDS = [
    ([1, 64, 65, 130, 0, 200], None),           # a fresh page, a page filled up, a page begun, an unused slot
    ([5, 64, 128, 300], [5, 64, 128, 300]),     # whole prompts
    ([70, 129, 40, 257], [6, 65, 0, 200]),      # rows that join a page, one sequence without rows
    ([3, 10], [5, 10]),                         # more rows than positions: the first are skipped
]


@pytest.mark.parametrize("lens,rows", APPENDS)
@pytest.mark.parametrize("type_,dim,tokens,heads,pad", [("f32", 128, 64, 2, 0), ("bf16", 64, 32, 3, 8), ("f16", 256, 128, 1, 24),
                                                        ("f32", 256, 256, 2, 4)])
def test_append_matches_oracle_bit_for_bit(q, lens, rows, type_, dim, tokens, heads, pad):
    c = Case(lens, heads, dim, tokens, seed=len(lens)).on_gpu(q)
    n = len(lens) if rows is None else sum(rows)
    scale = np.exp(c.rng.normal(size=(n, 1)))  # some rows raise their page's scale, some do not
    k = rows_tensor(c.rng.normal(size=(n, heads * dim)) * scale, TYPES[type_], pad)
    v = rows_tensor(c.rng.normal(size=(n, heads * dim)) * scale, TYPES[type_], pad)
    start = None if rows is None else starts(rows)
    gstart = None if rows is None else torch.from_numpy(start).cuda()
    q.apr_kv8_append(c.cache, c.gtable, c.glens, k, v, row_start=gstart)
    q.apr_stream_status()
    want = oracle.kv8_append(c.host, c.table, c.lens, start, as_f32(k), as_f32(v))
    c.assert_cache(want)
    # and back, into strided rows of the same type
    kb, vb = (rows_tensor(np.full((n, heads * dim), 7.0), TYPES[type_], 2 * pad) for _ in range(2))
    q.apr_kv8_read(c.cache, c.gtable, c.glens, kb, vb, row_start=gstart, max_rows=0 if rows is None else max(rows))
    q.apr_stream_status()
    wk, wv = oracle.kv8_read(want, c.table, c.lens, start, n)
    for got, w in ((kb, wk), (vb, wv)):
        assert torch.equal(got.cpu(), torch.from_numpy(w.reshape(n, -1)).to(TYPES[type_]))
        assert bool(torch.isnan(got.as_strided((n, 2 * pad), (got.stride(0), 1), got.shape[1])).all()) if pad and n > 1 else True
    # appending the same rows once more changes nothing
    q.apr_kv8_append(c.cache, c.gtable, c.glens, k, v, row_start=gstart)
    c.assert_cache(want)


def test_append_step_by_step_follows_the_oracle(q):
    c = Case([0, 0], 2, 64, 32, seed=3, spare=8, extra_width=3).on_gpu(q)
    c.table[:, :3] = c.free[:6].reshape(2, 3)
    c.gtable.copy_(torch.from_numpy(c.table))
    want = c.host
    for n in range(1, 71):
        c.lens[:] = (n, max(0, n - 40))
        c.glens.copy_(torch.from_numpy(c.lens))
        x = c.rng.normal(size=(2, 2, 2 * 64)).astype(np.float32) * (1 + n / 10)
        q.apr_kv8_append(c.cache, c.gtable, c.glens, torch.from_numpy(x[0]).cuda(), torch.from_numpy(x[1]).cuda())
        want = oracle.kv8_append(want, c.table, c.lens, None, x[0], x[1])
    q.apr_stream_status()
    c.assert_cache(want)


def test_append_of_special_values(q):
    c = Case([6, 40], 1, 64, 32, seed=4).on_gpu(q)
    x = np.zeros((8, 64), np.float32)
    x[0] = np.arange(64) - 31.5           # ties at scale 0.25: amax 31.75
    x[0, 0], x[0, 1:8] = 31.75, [0.125, 0.375, -0.125, -0.375, 0.625, np.nan, np.inf]
    x[1, 3], x[1, 4] = -np.inf, 1e-30
    x[2:6] = c.rng.normal(size=(4, 64)) * 1e-3
    y = np.zeros((8, 64), np.float32)     # all zeros; the other sequence: the smallest numbers
    y[6:] = c.rng.integers(-5, 6, (2, 64)) * 1e-45
    x[6], x[7] = np.nan, 1e38
    start = np.array([0, 6, 8], np.int32)
    q.apr_kv8_append(c.cache, c.gtable, c.glens, torch.from_numpy(x).cuda(), torch.from_numpy(y).cuda(),
                     row_start=torch.from_numpy(start).cuda())
    q.apr_stream_status()
    c.assert_cache(oracle.kv8_append(c.host, c.table, c.lens, start, x, y))


def test_append_decides_values_next_to_the_halves_exactly(q):
    c = Case([64], 1, 256, 64, seed=5).on_gpu(q)
    s = oracle.kv8_scale(np.float32(5.3))
    half = ((c.rng.integers(-126, 126, 64 * 256) + 0.5) * float(s)).astype(np.float32)
    step = c.rng.integers(-2, 3, half.shape)
    x = half.copy()
    for k in (1, 2):
        x = np.where(step >= k, np.nextafter(x, np.float32(9)), np.where(step <= -k, np.nextafter(x, np.float32(-9)), x))
    x = x.reshape(64, 256)
    x[5, 7] = 5.3
    q.apr_kv8_append(c.cache, c.gtable, c.glens, torch.from_numpy(x).cuda(), torch.from_numpy(-x).cuda(),
                     row_start=torch.tensor([0, 64], dtype=torch.int32, device="cuda"))
    q.apr_stream_status()
    assert c.cache.k_scale[c.table[0, 0], 0].item() == s
    c.assert_cache(oracle.kv8_append(c.host, c.table, c.lens, [0, 64], x, -x))


# ---------------------------------------------------------------- attention
def attend(q, c, num_heads, rows=None, type_="f32", pad=0, scale=0.0, weights=False, qh=None, **more):
    n = len(c.lens) if rows is None else sum(rows)
    qh = c.rng.normal(size=(n, num_heads * c.dim)) if qh is None else qh
    qt = rows_tensor(qh, TYPES[type_], pad)
    out = rows_tensor(np.full((n, num_heads * c.dim), np.nan), TYPES[type_], 2 * pad)
    start = None if rows is None else starts(rows)
    gstart = None if rows is None else torch.from_numpy(start).cuda()
    wide = c.table.shape[1] * c.tokens + 5
    w = torch.full((len(c.lens), c.heads, wide), 3.0, device="cuda") if weights else None
    q.apr_kv8_attention(c.cache, c.gtable, c.glens, qt, out, num_heads, row_start=gstart, scale=scale, weights=w, **more)
    q.apr_stream_status()
    if pad and n > 1:
        assert bool(torch.isnan(out.as_strided((n - 1, 2 * pad), (out.stride(0), 1), out.shape[1])).all())
    ref = oracle.kv8_attention(c.host, c.table, c.lens, start, as_f32(qt), num_heads, scale)
    return out, w, ref


def assert_attention(c, out, ref, type_="f32", frobenius=True):
    want, _, reach = ref
    y = as_f32(out).astype(np.float64).reshape(want.shape)
    vmax = float((np.abs(c.host["V"].astype(np.float64)) * c.host["v_scale"][..., None, None]).max())
    half = torch.finfo(TYPES[type_]).eps / 2
    tol = (2 * c.dim * 2.0 ** -24 * reach + 2.0 ** -17)[..., None] * 2 * vmax + half * np.abs(want)
    assert np.isfinite(y).all()
    assert (np.abs(y - want) <= tol).all(), float((np.abs(y - want) / tol).max())
    if frobenius and np.linalg.norm(want):
        rel = np.linalg.norm(y - want) / np.linalg.norm(want)
        assert rel <= EXACT_REL + (half if type_ != "f32" else 0), rel


def assert_weights(c, w, ref, before=0.0):
    want, reach = ref[1], float(ref[2].max()) if ref[2].size else 0.0
    got = w.cpu().numpy().astype(np.float64)
    for b, n in enumerate(c.lens):
        x = want[b, :, :n] + before
        np.testing.assert_allclose(got[b, :, :n], x, rtol=0, atol=(4 * c.dim * 2.0 ** -24 * reach + 2.0 ** -20) * max(1.0, x.max() if n else 1))


# one token a sequence: no positions, one, around a tile's, a page's and several units' ends, long ones
LENS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 200, 511, 1000]


@pytest.mark.parametrize("dim,heads,group,tokens,type_", [
    (64, 2, 1, 32, "f32"), (64, 1, 8, 64, "bf16"), (128, 2, 4, 64, "f32"), (128, 3, 7, 32, "f16"), (128, 1, 16, 128, "f32"),
    (256, 2, 4, 64, "f32"), (256, 1, 5, 256, "bf16"), (64, 1, 33, 32, "f32"), (256, 1, 20, 32, "f16")])
def test_attention_of_single_rows(q, dim, heads, group, tokens, type_):
    c = Case(LENS, heads, dim, tokens, seed=dim + group).on_gpu(q)
    out, w, ref = attend(q, c, heads * group, type_=type_, pad=8, weights=True)
    assert_attention(c, out, ref, type_)
    assert_weights(c, w, ref)
    for b, n in enumerate(c.lens):  # positions past a length: zeros
        assert not w[b, :, n:].any()
    assert not out[0].any()         # a slot without positions


@pytest.mark.parametrize("dim,heads,group,tokens,rows,lens", [
    (128, 2, 4, 64, [3, 0, 7, 1], [50, 300, 70, 1]),
    (64, 1, 2, 32, [40, 17, 64], [40, 400, 64]),           # whole prompts and a chunk behind a prefix
    (256, 1, 4, 64, [9, 2], [9, 130]),
    (128, 1, 1, 128, [130], [1000]),
    (64, 2, 12, 32, [5, 6], [3, 6])])                      # a row before the sequence's start sees nothing
def test_attention_of_several_rows(q, dim, heads, group, tokens, rows, lens):
    c = Case(lens, heads, dim, tokens, seed=7).on_gpu(q)
    out, w, ref = attend(q, c, heads * group, rows=rows, weights=True, pad=4)
    assert_attention(c, out, ref)
    assert_weights(c, w, ref)
    out16, _, ref16 = attend(q, c, heads * group, rows=rows, type_="bf16", max_rows=max(rows), max_len=max(lens))
    assert_attention(c, out16, ref16, "bf16")


def test_attention_of_long_sequences(q):
    # pieces of one sequence on every SM, beside short ones
    c = Case([20011, 3, 700], 1, 64, 64, seed=8).on_gpu(q)
    out, w, ref = attend(q, c, 2, weights=True)
    assert_attention(c, out, ref)
    assert_weights(c, w, ref)


def test_many_sequences(q):
    lens = list(np.random.default_rng(9).integers(0, 90, 700))
    c = Case(lens, 1, 64, 32, seed=9).on_gpu(q)
    out, _, ref = attend(q, c, 2)
    assert_attention(c, out, ref)


def test_every_operator_over_thousands_of_sequences(q):
    # more sequences than a CTA has threads: each thread counts several, some without rows, some without positions
    rng = np.random.default_rng(19)
    count = 3001
    lens = rng.integers(0, 70, count)
    rows = np.minimum(rng.integers(0, 4, count), lens)
    c = Case(list(lens), 1, 64, 32, seed=19, spare=2 * count).on_gpu(q)
    n, start = int(rows.sum()), starts(rows)
    gstart = torch.from_numpy(start).cuda()
    k, v = (torch.from_numpy(rng.normal(size=(n, 64)).astype(np.float32)).cuda() for _ in range(2))
    q.apr_kv8_append(c.cache, c.gtable, c.glens, k, v, row_start=gstart, max_rows=3)
    q.apr_stream_status()
    c.host = oracle.kv8_append(c.host, c.table, c.lens, start, as_f32(k), as_f32(v))
    c.assert_cache(c.host)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    q.apr_kv8_read(c.cache, c.gtable, c.glens, kb, vb, row_start=gstart, max_rows=3)
    wk, wv = oracle.kv8_read(c.host, c.table, c.lens, start, n)
    np.testing.assert_array_equal(as_f32(kb), wk.reshape(n, -1))
    np.testing.assert_array_equal(as_f32(vb), wv.reshape(n, -1))
    out, w, ref = attend(q, c, 2, rows=list(rows), weights=True, max_rows=3)
    assert_attention(c, out, ref)
    assert_weights(c, w, ref)
    evict(q, c, rng.random((count, 1, c.table.shape[1] * 32)).astype(np.float32), 40, 5)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_dominant_position_and_rising_scores(q, dim):
    # scores that rise from page to page by more than any reference is kept for, one position that takes all, and
    # pages whose scales differ by 2^20
    c = Case([500, 300, 400], 1, dim, 32, seed=10)
    c.host["K"][:] = c.rng.integers(-3, 4, c.host["K"].shape)
    for i in range(15):
        c.host["K"][c.table[0, i], 0, 5, 0] = 8 * (i + 1)
    c.host["K"][c.table[1, 4], 0, 3, 0] = 127
    c.host["v_scale"][c.table[2, ::2][:6]] = 2.0 ** -18
    c.host["v_scale"][c.table[2, 1::2][:6]] = 4.0
    c.host["k_scale"][c.table[0, :15]] = 0.5
    c.host["k_scale"][c.table[1, :9]] = 1.0
    c.on_gpu(q)
    qh = np.zeros((3, 2 * dim))
    qh[:, 0], qh[:, dim] = np.sqrt(dim), 3 * np.sqrt(dim)
    out, w, ref = attend(q, c, 2, qh=qh, weights=True)
    assert_attention(c, out, ref, frobenius=False)
    assert_weights(c, w, ref)


def test_small_weights_of_many_positions_add_up(q):
    # one weight of 1 beside 6000 of 2^-20 and less: what they carry together is kept
    c = Case([6000], 1, 64, 64, seed=11)
    c.host["K"][:], c.host["V"][:] = 0, 100
    c.host["k_scale"][:], c.host["v_scale"][:] = 1.0, 1.0
    c.host["K"][c.table[0, 50], 0, 9, 0] = 100
    c.host["V"][c.table[0, 50], 0, 9, :] = 0
    c.on_gpu(q)
    qh = np.zeros((1, 64))
    qh[0, 0] = 8.0 * 15.0 / 100.0  # a score of 15 against 0: weights of 3e-7
    out, _, ref = attend(q, c, 1, qh=qh)
    want = ref[0][0, 0]
    np.testing.assert_allclose(as_f32(out)[0], want, rtol=1e-4)


def test_custom_scale_and_zero_query(q):
    c = Case([300, 77], 2, 128, 64, seed=12).on_gpu(q)
    out, _, ref = attend(q, c, 4, scale=0.31)
    assert_attention(c, out, ref, frobenius=False)
    out, w, ref = attend(q, c, 4, qh=np.zeros((2, 4 * 128)), weights=True)
    assert_attention(c, out, ref)
    np.testing.assert_allclose(w[0, 0, :300].cpu().numpy(), 2 / 300, rtol=1e-5)


def test_tiny_and_huge_queries(q):
    c = Case([150, 150, 150], 1, 64, 32, seed=13)
    c.host["k_scale"][:] = 1e-12
    c.on_gpu(q)
    qh = c.rng.normal(size=(3, 64)) * np.array([[1e12], [1e-30], [1e10]])
    out, _, ref = attend(q, c, 1, qh=qh)
    assert_attention(c, out, ref)


def test_nan_and_infinite_queries_stay_in_their_row(q):
    c = Case([100, 100, 100], 1, 128, 64, seed=14).on_gpu(q)
    qh = c.rng.normal(size=(3, 4 * 128))
    clean, _, _ = attend(q, c, 4, qh=qh)
    qh[1, 5], qh[2, 128 * 2 + 9] = np.nan, np.inf
    qt, out = rows_tensor(qh, torch.float32), torch.zeros((3, 512), device="cuda")
    q.apr_kv8_attention(c.cache, c.gtable, c.glens, qt, out, 4)
    q.apr_stream_status()
    bad = torch.zeros((3, 4), dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 2] = True
    assert torch.equal(torch.isnan(out.view(3, 4, 128)).all(-1), bad)
    assert torch.equal(out.view(3, 4, 128)[~bad], clean.view(3, 4, 128)[~bad])


def test_what_lies_past_a_length_does_not_matter(q):
    c = Case([33, 70], 2, 128, 64, seed=15).on_gpu(q)
    qh = c.rng.normal(size=(2, 8 * 128))
    a, _, _ = attend(q, c, 8, qh=qh)
    for b, n in enumerate((33, 70)):  # other codes behind the last position, NaN scales in pages that are not theirs
        page = int(c.table[b, n // 64])
        c.cache.K[page, :, n % 64:] = -128
        c.cache.V[page, :, n % 64:] = 127
    used = {int(p) for b in range(2) for p in c.table[b, : -(-int(c.lens[b]) // 64)]}
    for p in range(c.cache.K.shape[0]):
        if p not in used:
            c.cache.k_scale[p] = float("nan")
            c.cache.v_scale[p] = float("nan")
    b, _, _ = attend(q, c, 8, qh=qh)
    assert torch.equal(a, b)


def test_weights_accumulate_over_steps(q):
    c = Case([40, 90, 10], 2, 64, 32, seed=16).on_gpu(q)
    wide = c.table.shape[1] * 32
    w = torch.full((3, 2, wide), float("nan"), device="cuda")
    want = np.zeros((3, 2, wide))
    for step, rows in enumerate(([40, 20, 1], [2, 0, 3], [1, 1, 1])):
        c.lens[:] = np.array([40, 90, 10]) - [[3, 1, 4], [1, 1, 1], [0, 0, 0]][step]
        c.glens.copy_(torch.from_numpy(c.lens))
        rows = [min(r, int(n)) for r, n in zip(rows, c.lens)]
        qt = torch.from_numpy(c.rng.normal(size=(sum(rows), 4 * 64)).astype(np.float32)).cuda()
        start = starts(rows)
        q.apr_kv8_attention(c.cache, c.gtable, c.glens, qt, torch.empty_like(qt), 4, row_start=torch.from_numpy(start).cuda(),
                            weights=w, accumulate=step > 0)
        _, add, _ = oracle.kv8_attention(c.host, c.table, c.lens, start, qt.cpu().numpy(), 4)
        want[:, :, : add.shape[2]] += add
        if step == 0:  # positions past a length are zeros after the first call; make them anything
            for b, n in enumerate(c.lens):
                w[b, :, n:] = 5.0
    q.apr_stream_status()
    got = w.cpu().numpy()
    for b, n in enumerate(c.lens):
        np.testing.assert_allclose(got[b, :, :n], want[b, :, :n], rtol=0, atol=4e-5)
        assert (got[b, :, n:] == 5.0).all()


@pytest.mark.parametrize("dim", [64, 256])
def test_weights_of_a_call_without_rows_are_zeros(q, dim):
    # no sequence has a row: every position received nothing, as where one sequence of several has none
    c = Case([40, 0, 700], 2, dim, 32, seed=24).on_gpu(q)
    out, w, ref = attend(q, c, 4, rows=[0, 0, 0], weights=True)
    assert out.shape[0] == 0 and not w.any() and not ref[1].any()
    w.fill_(3.0)
    attend_args = (c.cache, c.gtable, c.glens, out, out.clone(), 4)
    none = torch.zeros(4, dtype=torch.int32, device="cuda")
    q.apr_kv8_attention(*attend_args, row_start=none, weights=w, accumulate=True)
    assert bool((w == 3.0).all())
    q.apr_kv8_attention(*attend_args, row_start=none)
    q.apr_stream_status()


def test_repeats_are_bitwise_the_same(q):
    c = Case([5000, 40, 1300, 0, 77], 2, 128, 64, seed=17).on_gpu(q)
    qh = c.rng.normal(size=(5, 8 * 128))
    outs = [attend(q, c, 8, qh=qh, weights=True)[:2] for _ in range(3)]
    for out, w in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(w, outs[0][1])


# ---------------------------------------------------------------- eviction
def evict(q, c, weights, budget, recent, **more):
    wide = -(-budget // c.tokens)
    fresh = np.array(c.free[: wide * len(c.lens)], np.int32).reshape(len(c.lens), wide)
    table_out, lens_out = torch.full_like(c.gtable, 9), torch.full_like(c.glens, 9)
    wo = torch.full((len(c.lens), c.heads, budget + 3), 9.0, device="cuda")
    kept = torch.full((len(c.lens), c.heads, budget), 9, dtype=torch.int32, device="cuda")
    q.apr_kv8_evict(c.cache, c.gtable, c.glens, torch.from_numpy(weights).cuda(), budget, recent,
                    torch.from_numpy(fresh).cuda(), table_out, lens_out, wo, kept, **more)
    q.apr_stream_status()
    want, wt, wl, ww, wk = oracle.kv8_evict(c.host, c.table, c.lens, weights, budget, recent, fresh)
    np.testing.assert_array_equal(kept.cpu().numpy(), wk)
    np.testing.assert_array_equal(wo.cpu().numpy()[:, :, :budget], ww)
    assert not wo[:, :, budget:].any()
    np.testing.assert_array_equal(lens_out.cpu().numpy(), wl)
    np.testing.assert_array_equal(table_out.cpu().numpy(), wt)
    # the tail of a sequence's last page is not written; everything else is the same
    c.assert_cache(want)
    return table_out, lens_out, wo, kept


@pytest.mark.parametrize("budget,recent", [(64, 16), (65, 0), (100, 100), (1, 0), (1, 1), (700, 33), (4000, 7)])
@pytest.mark.parametrize("dim,heads,tokens", [(64, 3, 32), (128, 1, 64), (256, 2, 128)])
def test_eviction_matches_oracle_bit_for_bit(q, budget, recent, dim, heads, tokens):
    lens = [0, 1, 63, 64, 101, 330, 999]
    c = Case(lens, heads, dim, tokens, seed=budget, spare=len(lens) * -(-budget // tokens)).on_gpu(q)
    w = np.exp(3 * c.rng.normal(size=(len(lens), heads, c.table.shape[1] * tokens))).astype(np.float32)
    w[:, 0] = np.floor(w[:, 0])  # many equal ones, many zeros
    evict(q, c, w, budget, recent)


def test_eviction_of_special_weights(q):
    c = Case([300, 300, 300, 300], 1, 64, 32, seed=20, spare=16).on_gpu(q)
    w = np.zeros((4, 1, 320), np.float32)     # first: all equal
    w[1] = -c.rng.random((1, 320))            # negative ones
    w[1, 0, ::3] = -0.0
    w[2] = c.rng.normal(size=(1, 320))
    w[2, 0, [5, 50, 250]], w[2, 0, [7, 70]], w[2, 0, 9] = np.nan, np.inf, -np.inf
    w[3] = (c.rng.random((1, 320)) * 1e-42).astype(np.float32)   # subnormal
    w[:, :, 300:] = np.nan                    # past the lengths
    evict(q, c, w, 100, 20, max_len=300)


def test_eviction_of_a_long_sequence(q):
    c = Case([50000, 20], 1, 64, 256, seed=21, spare=48).on_gpu(q)
    w = np.exp(c.rng.normal(size=(2, 1, c.table.shape[1] * 256))).astype(np.float32)
    w[0, 0, 1000:30000] = 1.0
    evict(q, c, w, 6001, 1)


def test_eviction_of_more_positions_than_a_cluster_holds(q):
    # over 8 x 20480 positions: the keys are made from the weights again in each pass
    c = Case([170001], 1, 64, 256, seed=23, spare=36).on_gpu(q)
    w = np.exp(2 * c.rng.normal(size=(1, 1, c.table.shape[1] * 256))).astype(np.float32)
    w[0, 0, ::3] = 0
    w[0, 0, 5::7] = 9.0
    evict(q, c, w, 9000, 100)


def test_evicted_cache_is_read_and_appended_to(q):
    # the kept positions' attention is the attention over the rows read back, and the next token joins the fresh page
    c = Case([700, 90], 2, 128, 64, seed=22, spare=8).on_gpu(q)
    w = np.exp(2 * c.rng.normal(size=(2, 2, c.table.shape[1] * 64))).astype(np.float32)
    table, lens, _, _ = evict(q, c, w, 130, 30)
    lens += 1
    k, v = (torch.randn((2, 2 * 128), device="cuda") for _ in range(2))
    q.apr_kv8_append(c.cache, table, lens, k, v)
    qt = torch.randn((2, 8 * 128), device="cuda")
    out = torch.empty_like(qt)
    q.apr_kv8_attention(c.cache, table, lens, qt, out, 8)
    n = lens.tolist()
    kb, vb = (torch.empty((sum(n), 2 * 128), device="cuda") for _ in range(2))
    q.apr_kv8_read(c.cache, table, lens, kb, vb, row_start=torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda"))
    q.apr_stream_status()
    at = 0
    for b in range(2):
        K = kb[at:at + n[b]].double().view(n[b], 2, 128).repeat_interleave(4, 1)
        V = vb[at:at + n[b]].double().view(n[b], 2, 128).repeat_interleave(4, 1)
        p = torch.softmax(torch.einsum("hd,nhd->hn", qt[b].double().view(8, 128), K) / 128 ** 0.5, -1)
        want = torch.einsum("hn,nhd->hd", p, V)
        rel = (out[b].double().view(8, 128) - want).norm() / want.norm()
        assert rel <= EXACT_REL
        at += n[b]


# ---------------------------------------------------------------- streams, graphs, what the device arrays say
def test_two_streams_at_once(q):
    cases = [Case([900, 33], 2, 128, 64, seed=s).on_gpu(q) for s in (30, 31)]
    streams = [torch.cuda.Stream() for _ in cases]
    qs = [torch.from_numpy(c.rng.normal(size=(2, 8 * 128)).astype(np.float32)).cuda() for c in cases]
    outs = [torch.empty_like(x) for x in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, x, o in zip(cases, streams, qs, outs):
            q.apr_kv8_attention(c.cache, c.gtable, c.glens, x, o, 8, stream=s)
    for c, s, x, o in zip(cases, streams, qs, outs):
        q.apr_stream_status(s)
        assert_attention(c, o, oracle.kv8_attention(c.host, c.table, c.lens, None, x.cpu().numpy(), 8))


def test_a_captured_step_follows_the_lengths(q):
    # append, attention with weights, and the lengths' increment, captured once and replayed
    c = Case([70, 31, 0], 2, 64, 32, seed=32, spare=9, extra_width=3).on_gpu(q)
    c.table[:, -3:] = c.free[:9].reshape(3, 3)
    for b, n in enumerate(c.lens):
        count = -(-int(n) // 32)
        c.table[b, count:count + 3] = c.free[3 * b:3 * b + 3]
    c.gtable.copy_(torch.from_numpy(c.table))
    k, v = (torch.zeros((3, 2 * 64), device="cuda") for _ in range(2))
    qt, out = torch.zeros((3, 4 * 64), device="cuda"), torch.zeros((3, 4 * 64), device="cuda")
    w = torch.zeros((3, 2, c.table.shape[1] * 32), device="cuda")
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        c.glens.add_(1)
        q.apr_kv8_append(c.cache, c.gtable, c.glens, k, v, stream=s)
        q.apr_kv8_attention(c.cache, c.gtable, c.glens, qt, out, 4, weights=w, accumulate=True, stream=s)
    want, total = c.host, np.zeros(w.shape)
    for _ in range(40):
        x = c.rng.normal(size=(3, 8 * 64)).astype(np.float32)
        for t, part in ((k, x[:, :128]), (v, x[:, 128:256]), (qt, x[:, 256:])):
            t.copy_(torch.from_numpy(np.ascontiguousarray(part)))
        graph.replay()
        c.lens += 1
        want = oracle.kv8_append(want, c.table, c.lens, None, x[:, :128], x[:, 128:256])
        ref = oracle.kv8_attention(want, c.table, c.lens, None, x[:, 256:], 4)
        total[:, :, : ref[1].shape[2]] += ref[1]
    torch.cuda.synchronize()
    q.apr_stream_status(s)
    c.assert_cache(want)
    c.host = want
    assert_attention(c, out, ref)
    np.testing.assert_allclose(w.cpu().numpy(), total, rtol=0, atol=1e-4)


def bad_index(q):
    with pytest.raises(q.AprError) as e:
        q.apr_stream_status()
    assert e.value.status == -1 and "out of range" in str(e.value)
    q.apr_stream_status()  # cleared


@pytest.mark.parametrize("what", ["page", "negative page", "length", "row_start", "row_start past", "row_start falls", "max_rows"])
def test_bad_device_arrays_are_reported_and_touch_nothing(q, what):
    c = Case([100, 70], 1, 64, 32, seed=40, extra_width=0).on_gpu(q)
    rows, more = [3, 2], {}
    start = torch.from_numpy(starts(rows)).cuda()
    if what == "page":
        c.gtable[0, 3] = c.cache.K.shape[0]
    elif what == "negative page":
        c.gtable[0, 3] = -1
    elif what == "length":
        c.glens[0] = 129
    elif what == "row_start":
        start[1] = -2
    elif what == "row_start past":
        start[2] = 6
    elif what == "row_start falls":
        start[0], start[1] = 5, 0  # the first range ends before it begins, the second is the whole call
    else:
        more = {"max_rows": 2}
    k = torch.ones((5, 64), device="cuda")
    before = c.cache.K.clone()
    q.apr_kv8_append(c.cache, c.gtable, c.glens, k, k, row_start=start, **more)
    bad_index(q)
    assert torch.equal(c.cache.K[c.free], before[c.free])
    q.apr_kv8_read(c.cache, c.gtable, c.glens, torch.empty_like(k), torch.empty_like(k), row_start=start, **more)
    bad_index(q)
    q.apr_kv8_attention(c.cache, c.gtable, c.glens, torch.ones((5, 128), device="cuda"), torch.empty((5, 128), device="cuda"), 2,
                        row_start=start, **more)
    bad_index(q)


def test_bad_pages_of_an_eviction_are_reported(q):
    c = Case([100, 100], 1, 64, 32, seed=41, spare=4, extra_width=0).on_gpu(q)
    w = torch.rand((2, 1, 128), device="cuda")
    fresh = torch.tensor([[int(c.free[0])], [1 << 20]], dtype=torch.int32, device="cuda")
    args = (torch.empty_like(c.gtable), torch.empty_like(c.glens), torch.empty((2, 1, 30), device="cuda"),
            torch.empty((2, 1, 30), dtype=torch.int32, device="cuda"))
    q.apr_kv8_evict(c.cache, c.gtable, c.glens, w, 30, 30, fresh, *args)
    bad_index(q)
    fresh[1, 0] = int(c.free[1])
    c.gtable[1, 3] = -5  # holds the most recent positions, which are kept
    q.apr_kv8_evict(c.cache, c.gtable, c.glens, w, 30, 30, fresh, *args)
    bad_index(q)


def test_offsets_past_32_bits(q):
    # a cache of 2.4 GB of codes: the pages at its end
    pages, heads, tokens, dim = 4700, 8, 256, 256
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    cache = q.Kv8Cache.allocate(pages, heads, dim, tokens)
    n = 700
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((n, heads * dim), device="cuda") for _ in range(2))
    q.apr_kv8_append(cache, table, lens, k, v, row_start=start)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    q.apr_kv8_read(cache, table, lens, kb, vb, row_start=start)
    q.apr_stream_status()
    # half a step of the page's scale, of the largest value of 256 x 256
    assert float((k - kb).abs().max()) <= float(k.abs().max()) / 254 * 1.0001
    assert not cache.K[: pages - 3].view(torch.int64).any()
    qt = torch.randn((1, heads * dim), device="cuda")
    out = torch.empty_like(qt)
    q.apr_kv8_attention(cache, table, lens, qt, out, heads)
    K, V = kb.double().view(n, heads, dim), vb.double().view(n, heads, dim)
    p = torch.softmax(torch.einsum("hd,nhd->hn", qt.double().view(heads, dim), K) / dim ** 0.5, -1)
    want = torch.einsum("hn,nhd->hd", p, V)
    assert (out.double().view(heads, dim) - want).norm() / want.norm() <= EXACT_REL
