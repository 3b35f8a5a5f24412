"""The 8-bit KV cache without a GPU: its oracle against hand-made cases, its C
ABI's declarations and refusals (every refused call fails on the host before
any CUDA call; the addresses are made up and never read)."""

import ctypes
import math
import os
import re
from fractions import Fraction

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "apr_kv8.h")


# ---------------------------------------------------------------- the oracle
def one_page(heads=1, tokens=32, dim=64, pages=3):
    shape = (pages, heads, tokens, dim)
    return {"K": np.zeros(shape, np.int8), "V": np.zeros(shape, np.int8),
            "k_scale": np.zeros(shape[:2], np.float32), "v_scale": np.zeros(shape[:2], np.float32)}


def exact_code(x, s):
    """Nearest whole number to x / s in rational arithmetic, ties to even."""
    r = Fraction(float(x)) / Fraction(float(s))
    low = math.floor(r)
    up = r - low > Fraction(1, 2) or (r - low == Fraction(1, 2) and low % 2 == 1)
    return max(-127, min(127, low + up))


def test_codes_are_the_nearest_whole_number_exactly():
    rng = np.random.default_rng(0)
    s = oracle.kv8_scale(np.float32(3.7))
    x = rng.uniform(-3.7, 3.7, 300).astype(np.float32)
    # values on both sides of, and next to, the halves
    halves = np.array([(c + 0.5) * float(s) for c in range(-20, 20)], np.float32)
    x = np.concatenate([x, halves, np.nextafter(halves, np.float32(9)), np.nextafter(halves, np.float32(-9))])
    assert [int(c) for c in oracle.kv8_codes(x, s)] == [exact_code(v, s) for v in x]


def test_codes_at_ties_and_special_values():
    s = np.float32(0.25)
    x = np.array([0.125, 0.375, -0.125, -0.375, 31.75, 40.0, np.nan, np.inf, -np.inf], np.float32)
    assert oracle.kv8_codes(x, s).tolist() == [0, 2, 0, -2, 127, 127, 0, 127, -127]
    assert oracle.kv8_codes(x, np.float32(0)).tolist() == [0] * 9


def test_append_raises_the_scale_and_rounds_what_was_held():
    c = one_page()
    table = [[2, 0]]
    k1 = np.zeros((1, 64), np.float32)
    k1[0, :2] = 1.27, -0.5
    c = oracle.kv8_append(c, table, [1], None, k1, k1)
    s1 = oracle.kv8_scale(np.float32(1.27))
    assert c["k_scale"][2, 0] == s1 and c["K"][2, 0, 0, :3].tolist() == [127, -50, 0]
    k2 = np.zeros((1, 64), np.float32)
    k2[0, 0] = 2.54
    c = oracle.kv8_append(c, table, [2], None, k2, k2)
    s2 = oracle.kv8_scale(np.float32(2.54))
    assert c["k_scale"][2, 0] == s2
    assert c["K"][2, 0, 0, :2].tolist() == [exact_code(np.float32(127) * s1, s2), -25]
    assert c["K"][2, 0, 1, 0] == 127
    # a smaller row leaves the scale
    c2 = oracle.kv8_append(c, table, [3], None, k1, k1)
    assert c2["k_scale"][2, 0] == s2 and c2["K"][2, 0, 2, 1] == exact_code(np.float32(-0.5), s2)
    # the next page starts anew, whatever its scale was
    c2["k_scale"][0, 0] = 9.0
    c3 = oracle.kv8_append(c2, table, [33], None, k1, k1)
    assert c3["k_scale"][0, 0] == s1 and c3["K"][0, 0, 0, 0] == 127


def test_read_and_attention_of_hand_made_cache():
    c = one_page(heads=1)
    c["K"][1, 0, 0, 0], c["K"][1, 0, 1, 0] = 8, -4
    c["V"][1, 0, 0, 3], c["V"][1, 0, 1, 3] = 10, 20
    c["k_scale"][1, 0], c["v_scale"][1, 0] = 0.5, 2.0
    k, v = oracle.kv8_read(c, [[1]], [2], [0, 2], 2)
    assert k[:, 0, 0].tolist() == [4.0, -2.0] and v[:, 0, 3].tolist() == [20.0, 40.0]
    q = np.zeros((2, 2, 64))
    q[:, :, 0] = 8.0  # scores 4 and -2 at scale 1/8
    out, w, _ = oracle.kv8_attention(c, [[1]], [2], [0, 2], q, 2)
    e = math.exp(-6.0)
    assert out[0, :, 3].tolist() == [20.0, 20.0]
    np.testing.assert_allclose(out[1, :, 3], (20 + 40 * e) / (1 + e), rtol=1e-14)
    np.testing.assert_allclose(w[0, 0], [2 + 2 / (1 + e), 2 * e / (1 + e)], rtol=1e-14)
    out, w, _ = oracle.kv8_attention(c, [[1], [0]], [1, 0], None, q, 2)
    assert out[0, 0, 3] == 20.0 and not out[1].any() and w[0, 0].tolist() == [2.0]


def test_evict_keeps_the_largest_lowest_first_and_the_recent():
    c = one_page(pages=4)
    rng = np.random.default_rng(1)
    c["K"][:], c["V"][:] = rng.integers(-127, 128, c["K"].shape), rng.integers(-127, 128, c["V"].shape)
    c["k_scale"][:], c["v_scale"][:] = 0.5, 0.25
    w = np.zeros((1, 1, 40), np.float32)
    w[0, 0, [3, 7, 9, 12, 33]] = [1, 2, 2, 2, 5]
    new, table, lens, wo, kept = oracle.kv8_evict(c, [[0, 1]], [40], w, 5, 2, [[3]])
    assert kept[0, 0].tolist() == [7, 9, 33, 38, 39]  # of the three 2s the two lowest
    assert wo[0, 0].tolist() == [2, 2, 5, 0, 0] and table.tolist() == [[3, -1]] and lens.tolist() == [5]
    s = oracle.kv8_scale(np.abs(np.concatenate([c["K"][0, 0, [7, 9]], c["K"][1, 0, [1, 6, 7]]])).max() * np.float32(0.5))
    assert new["k_scale"][3, 0] == s
    assert new["K"][3, 0, 2].tolist() == [exact_code(np.float32(x) * np.float32(0.5), s) for x in c["K"][1, 0, 1]]
    # at or under the budget nothing moves
    new, table, lens, wo, kept = oracle.kv8_evict(c, [[0, 1]], [40], w, 40, 2, [[3, 2]])
    assert kept[0, 0].tolist() == list(range(40)) and table.tolist() == [[0, 1]] and np.array_equal(new["K"], c["K"])


# ---------------------------------------------------------------- the C ABI
def test_header_and_binding_agree(q):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^int (apr_kv8_\w+)\(", text, flags=re.M)
    assert sorted(names) == sorted(q.KV8_EXPORTS)
    for name in names:
        assert hasattr(q.library(), name)
    for name in ("APR_T_F32", "APR_T_F16", "APR_T_BF16"):
        assert int(re.search(rf"\b{name}\s*=\s*(\d+)", text).group(1)) == getattr(q, name)


A = 1 << 24  # a 16-byte aligned made-up address; the calls' arrays are smaller than A apart


def cache_and_rows(q, **change):
    from quantized_weight_prefill_q4_gb300 import kv8

    c = dict(K=A, V=2 * A, k_scale=3 * A, v_scale=4 * A, num_pages=8, num_kv_heads=2, page_tokens=64, head_dim=128)
    r = dict(page_table=5 * A, table_ld=4, lens=6 * A, row_start=7 * A, num_seqs=3, num_rows=10, max_rows=0, max_len=0)
    for name, value in change.items():
        (c if name in c else r)[name] = value
    return kv8._Cache(*c.values()), kv8._Rows(*r.values())


def refused(q, name, code, needle, change, args):
    c, r = cache_and_rows(q, **change)
    got = getattr(q.library(), name)(c, r, *args)
    assert got == code, (got, q.apr_last_error())
    assert needle in q.apr_last_error()


INVAL, ALIGN, ALIAS, DEVICE = -1, -3, -4, -5
CACHE_AND_ROWS = [
    (INVAL, "num_pages", dict(num_pages=0)),
    (INVAL, "num_kv_heads", dict(num_kv_heads=0)),
    (INVAL, "page_tokens", dict(page_tokens=48)),
    (INVAL, "page_tokens", dict(page_tokens=16)),
    (INVAL, "head_dim", dict(head_dim=96)),
    (INVAL, "num_seqs", dict(num_seqs=-1)),
    (INVAL, "table_ld", dict(table_ld=-1)),
    (INVAL, "table_ld", dict(table_ld=1 << 28)),
    (INVAL, "max_len", dict(max_len=257)),
    (INVAL, "null", dict(K=None)),
    (INVAL, "null", dict(v_scale=None)),
    (INVAL, "null", dict(lens=None)),
    (INVAL, "null", dict(page_table=None)),
    (ALIGN, "aligned", dict(V=2 * A + 8)),
    (ALIGN, "aligned", dict(k_scale=3 * A + 2)),
    (ALIGN, "aligned", dict(lens=6 * A + 1)),
    (ALIAS, "overlap", dict(V=A + 64)),
    (ALIAS, "overlap", dict(k_scale=A + 64)),
]
WITH_ROWS = [
    (INVAL, "num_rows", dict(num_rows=-1)),
    (INVAL, "max_rows", dict(max_rows=11)),
    (INVAL, "one row a sequence", dict(row_start=None)),
]
APPEND = (0, 8 * A, 9 * A, 256, None)
ATTEND = (0, 8 * A, 1024, 9 * A, 1024, 8, 0.0, None, 0, 0, None)
EVICT = (8 * A, 256, 100, 10, 9 * A, 10 * A, 11 * A, 12 * A, 100, 13 * A, None)


@pytest.mark.parametrize("code,needle,change", CACHE_AND_ROWS + WITH_ROWS)
def test_bad_caches_and_rows_are_refused(q, code, needle, change):
    refused(q, "apr_kv8_append", code, needle, change, APPEND)
    refused(q, "apr_kv8_read", code, needle, change, APPEND)
    refused(q, "apr_kv8_attention", code, needle, change, ATTEND)


@pytest.mark.parametrize("code,needle,change", CACHE_AND_ROWS)
def test_bad_caches_are_refused_by_the_eviction(q, code, needle, change):
    refused(q, "apr_kv8_evict", code, needle, change, EVICT)


def altered(args, change):
    args = list(args)
    for i, value in change.items():
        args[i] = value
    return tuple(args)


@pytest.mark.parametrize("code,needle,change", [
    (INVAL, "element type", {0: 2}),
    (INVAL, "ld=255", {3: 255}),
    (INVAL, "null", {1: None}),
    (INVAL, "null", {2: None}),
    (ALIGN, "16-byte", {1: 8 * A + 4}),
    (ALIGN, "16-byte", {3: 257}),
    (ALIGN, "16-byte", {0: 1, 3: 260}),
    (ALIAS, "overlaps", {1: A + 16}),
])
def test_bad_rows_are_refused(q, code, needle, change):
    refused(q, "apr_kv8_append", code, needle, {}, altered(APPEND, change))
    refused(q, "apr_kv8_read", code, needle, {}, altered(APPEND, change))


def test_read_refuses_outputs_that_overlap(q):
    refused(q, "apr_kv8_read", ALIAS, "k overlaps v", {}, (0, 8 * A, 8 * A + 512, 256, None))
    refused(q, "apr_kv8_read", ALIAS, "k overlaps v", {}, (0, 8 * A, 8 * A, 512, None))
    refused(q, "apr_kv8_read", ALIAS, "k overlaps v", {}, (0, 8 * A + 4 * 1024 + 16, 8 * A, 512, None))


@pytest.mark.parametrize("code,needle,change", [
    (INVAL, "element type", {0: 8}),
    (INVAL, "num_heads", {5: 7}),
    (INVAL, "num_heads", {5: 0}),
    (INVAL, "ldq", {2: 1020}),
    (INVAL, "ldo", {4: 1020}),
    (INVAL, "scale", {6: -1.0}),
    (INVAL, "scale", {6: math.inf}),
    (INVAL, "scale", {6: math.nan}),
    (INVAL, "weights_ld", {7: 14 * A, 8: 255}),
    (INVAL, "null", {1: None}),
    (INVAL, "null", {3: None}),
    (ALIGN, "16-byte", {2: 1026}),
    (ALIGN, "16-byte", {3: 9 * A + 4}),
    (ALIGN, "aligned", {7: 14 * A + 2, 8: 256}),
    (ALIAS, "out overlaps q", {3: 8 * A}),
    (ALIAS, "out overlaps V", {3: 2 * A}),
    (ALIAS, "weights overlaps", {7: 9 * A, 8: 256}),
    (ALIAS, "weights overlaps lens", {7: 6 * A, 8: 256}),
])
def test_bad_attention_is_refused(q, code, needle, change):
    refused(q, "apr_kv8_attention", code, needle, {}, altered(ATTEND, change))


@pytest.mark.parametrize("code,needle,change", [
    (INVAL, "weights_ld", {1: 255}),
    (INVAL, "budget", {2: 0}),
    (INVAL, "recent", {3: 101}),
    (INVAL, "recent", {3: -1}),
    (INVAL, "weights_out_ld", {8: 99}),
    (INVAL, "null", {0: None}),
    (INVAL, "null", {4: None}),
    (INVAL, "null", {9: None}),
    (ALIGN, "aligned", {6: 11 * A + 2}),
    (ALIAS, "table_out overlaps page_table", {5: 5 * A}),
    (ALIAS, "lens_out overlaps lens", {6: 6 * A}),
    (ALIAS, "weights_out overlaps weights", {7: 8 * A}),
    (ALIAS, "kept overlaps weights_out", {9: 12 * A}),
])
def test_bad_eviction_is_refused(q, code, needle, change):
    refused(q, "apr_kv8_evict", code, needle, {}, altered(EVICT, change))


def test_empty_calls_do_nothing(q):
    # no pointer is looked at, and no device is needed
    lib = q.library()
    none = dict(K=None, V=None, k_scale=None, v_scale=None, page_table=None, lens=None, row_start=None)
    for change in (dict(none, num_seqs=0, num_rows=0), dict(none, row_start=7 * A, num_rows=0)):
        c, r = cache_and_rows(q, **change)
        assert lib.apr_kv8_append(c, r, *APPEND) == 0
        assert lib.apr_kv8_read(c, r, *APPEND) == 0
        assert lib.apr_kv8_attention(c, r, *ATTEND) == 0
    c, r = cache_and_rows(q, num_seqs=0)
    assert lib.apr_kv8_evict(c, r, *EVICT) == 0
    assert q.library().apr_kv8_append(None, r, *APPEND) == INVAL
    assert q.library().apr_kv8_append(c, None, *APPEND) == INVAL


def test_weights_of_no_rows_are_an_output(q):
    # zeros to be written, so arguments are checked and the device is needed; with accumulate nothing changes
    import torch

    lib, none = q.library(), dict(num_rows=0, row_start=7 * A)
    sets = altered(ATTEND, {1: None, 3: None, 7: 10 * A, 8: 256})
    c, r = cache_and_rows(q, **none)
    assert lib.apr_kv8_attention(c, r, *altered(sets, {9: 1})) == 0
    refused(q, "apr_kv8_attention", INVAL, "weights_ld", none, altered(sets, {8: 255}))
    refused(q, "apr_kv8_attention", ALIGN, "weights", none, altered(sets, {7: 10 * A + 2}))
    refused(q, "apr_kv8_attention", ALIAS, "weights overlaps K", none, altered(sets, {7: A + 64}))
    refused(q, "apr_kv8_attention", INVAL, "null", dict(none, K=None), sets)
    if not torch.cuda.is_available():
        refused(q, "apr_kv8_attention", DEVICE, "", none, sets)
    c, r = cache_and_rows(q, **dict(none, num_seqs=0))
    assert lib.apr_kv8_attention(c, r, *sets) == 0


def test_good_arguments_reach_the_device_check(q):
    import torch

    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    for name, args in (("apr_kv8_append", APPEND), ("apr_kv8_read", APPEND), ("apr_kv8_attention", ATTEND),
                       ("apr_kv8_evict", EVICT)):
        c, r = cache_and_rows(q)
        assert getattr(q.library(), name)(c, r, *args) == DEVICE, (name, q.apr_last_error())
    c, r = cache_and_rows(q, row_start=None, num_rows=3)
    assert q.library().apr_kv8_append(c, r, *APPEND) == DEVICE


def test_binding_refuses_tensors_that_do_not_fit(q):
    import torch

    with pytest.raises(ValueError, match="device memory"):
        q.Kv8Cache.allocate(2, 1, 64, 32, device="cpu")
    with pytest.raises(TypeError, match="CUDA tensor"):
        q.Kv8Cache(1, 2, 3, 4)
    from quantized_weight_prefill_q4_gb300 import kv8

    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        kv8._matrix(torch.zeros(2, 64), "q", 64)
    with pytest.raises(ValueError, match="device memory"):
        kv8._array(torch.zeros(2), "lens", torch.float32, 1)
