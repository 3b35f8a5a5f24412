"""The rotations by position without a GPU: their oracle against hand-made cases and against differences, the C ABI's
declarations and refusals (every refused call fails on the host before any CUDA call; the addresses are made up and
never read), the binding's refusals."""

import math
import os
import re

import numpy as np
import pytest

import oracle
from test_kv8_binding import Unreached, cache_on, on
from test_kv8_host import ATTEND as DECODE
from test_kv8_host import A, ALIAS, ALIGN, CACHE_AND_ROWS, DEVICE, INVAL, WITH_ROWS, altered, cache_and_rows, refused

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "apr_rope.h")


# ---------------------------------------------------------------- the oracle
def test_rotation_by_hand():
    # a quarter turn, an eighth, none; dims past the rotation pass
    table = np.zeros((3, 4, 2), np.float32)
    table[0, :, 0] = 1
    table[1, :, 1] = 1
    table[2] = np.float32(math.sqrt(0.5))
    x = np.arange(1, 13, dtype=np.float32)[None]
    same = oracle.rope_rows(table, None, False, [[0]], x, 1)
    assert same.tolist() == x.tolist()
    halves = oracle.rope_rows(table, None, False, [[1]], x, 1)
    assert halves[0].tolist() == [-5, -6, -7, -8, 1, 2, 3, 4, 9, 10, 11, 12]
    pairs = oracle.rope_rows(table, None, True, [[1]], x, 1)
    assert pairs[0].tolist() == [-2, 1, -4, 3, -6, 5, -8, 7, 9, 10, 11, 12]
    axes = oracle.rope_rows(table, [0, 1, 0, 1], False, [[0], [1]], x, 1)
    assert axes[0].tolist() == [1, -6, 3, -8, 5, 2, 7, 4, 9, 10, 11, 12]
    eighth = oracle.rope_rows(table, None, False, [[2]], x, 1)
    np.testing.assert_allclose(eighth[0, :4], (x[0, :4] - x[0, 4:8]) * math.sqrt(0.5), rtol=1e-6)


def test_norm_by_hand():
    table = np.zeros((1, 4, 2), np.float32)
    table[..., 0] = 1
    x = np.array([[3, -4, 0, 0, 0, 0, 0, 0, 1, 1, 1, 1, 1, 1, 1, 1]], np.float32)  # means of squares 25 / 8 and 1
    got = oracle.rope_rows(table, None, True, [[0]], x, 2, norm=np.full(8, 2.0, np.float32))
    np.testing.assert_allclose(got[0, :2], np.array([6, -8]) / math.sqrt(25 / 8), rtol=1e-6)
    assert got[0, 8:].tolist() == [2] * 8
    with_eps = oracle.rope_rows(table, None, True, [[0]], x, 2, norm=np.ones(8, np.float32), eps=3.0)
    assert with_eps[0, 8:].tolist() == [0.5] * 8


def test_scores_depend_on_the_distance_alone():
    # the point of the rotation: q at p against k at p' is q at p + d against k at p' + d
    rng = np.random.default_rng(0)
    inv = (1.0 / 10000.0 ** (np.arange(16) / 16)).astype(np.float32)
    table = oracle.rope_table(inv, 0, 5000).astype(np.float32)
    q, k = rng.normal(size=(2, 1, 32)).astype(np.float32)
    at = lambda x, p: oracle.rope_rows(table, None, False, [[p]], x, 1).astype(np.float64)  # noqa: E731
    scores = [float((at(q, 40 + d) * at(k, 13 + d)).sum()) for d in (0, 1, 700, 4900)]
    np.testing.assert_allclose(scores, scores[0], atol=32 * 8 * 2.0 ** -24 * 9)  # roundings of 32 products of values up to 3


def test_table_of_far_positions():
    # whole turns taken off in rational arithmetic by hand: the angle of position 2^29 + 1 and frequency 1
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    at = 2 ** 29 + 1
    rest = Fraction(at) - (Fraction(at) // (2 * pi)) * 2 * pi
    got = oracle.rope_table(np.ones(1, np.float32), at, 1, 1.5)[0, 0]
    np.testing.assert_allclose(got, [1.5 * math.cos(float(rest)), 1.5 * math.sin(float(rest))], rtol=0, atol=1e-14)


# ---------------------------------------------------------------- the C ABI
def test_header_and_binding_agree(q):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^int (apr_\w+)\(", text, flags=re.M)
    assert sorted(names) == sorted(q.ROPE_EXPORTS)
    for name in names:
        assert hasattr(q.library(), name)


def rope(**change):
    from quantized_weight_prefill_q4_gb300 import rope as module

    r = dict(table=20 * A, num_positions=1000, rot_dim=128, interleaved=0, pair_axis=None, num_axes=1, positions=22 * A, positions_ld=0)
    r.update(change)
    return module._Rope(*r.values())


BAD_ROPES = [
    (INVAL, "rot_dim", dict(rot_dim=0)),
    (INVAL, "rot_dim", dict(rot_dim=12)),
    (INVAL, "rot_dim", dict(rot_dim=136)),
    (INVAL, "num_positions", dict(num_positions=0)),
    (INVAL, "num_axes", dict(num_axes=0)),
    (INVAL, "num_axes", dict(num_axes=17, pair_axis=23 * A)),
    (INVAL, "num_axes", dict(num_axes=2)),
    (INVAL, "positions_ld", dict(positions_ld=9)),
    (INVAL, "null", dict(table=None)),
    (ALIGN, "aligned", dict(table=20 * A + 8)),
    (ALIGN, "aligned", dict(positions=22 * A + 2)),
    (ALIGN, "aligned", dict(pair_axis=23 * A + 1)),
]
ROWS = (0, 8 * A, 1024, 9 * A, 1024, 10, 8, 128, None, 0.0, None)  # type, x, ldx, out, ldo, rows, heads, dim, norm, eps, stream


def rows_refused(q, code, needle, r, args):
    assert q.library().apr_rope_rows(r, *args) == code, q.apr_last_error()
    assert needle in q.apr_last_error()


@pytest.mark.parametrize("code,needle,change", BAD_ROPES + [(INVAL, "null", dict(positions=None))])
def test_bad_rotations_of_rows_are_refused(q, code, needle, change):
    rows_refused(q, code, needle, rope(**change), ROWS)


@pytest.mark.parametrize("code,needle,change", [
    (INVAL, "element type", {0: 2}),
    (INVAL, "null", {1: None}),
    (INVAL, "null", {3: None}),
    (INVAL, "strides", {2: 1023}),
    (INVAL, "strides", {4: 1 << 29}),
    (INVAL, "num_rows", {5: -1}),
    (INVAL, "num_rows", {5: (1 << 24) + 1}),
    (INVAL, "num_heads", {6: 0}),
    (INVAL, "head_dim", {7: 0}),
    (INVAL, "head_dim", {7: 132}),
    (INVAL, "head_dim", {7: 520}),
    (INVAL, "rot_dim", {7: 64}),
    (INVAL, "eps", {9: -1.0}),
    (INVAL, "eps", {9: math.nan}),
    (ALIGN, "norm", {8: 30 * A + 4}),
    (ALIGN, "16-byte", {1: 8 * A + 8}),
    (ALIGN, "16-byte", {2: 1025}),
    (ALIGN, "16-byte", {0: 1, 4: 1028}),
    (ALIAS, "out overlaps x", {3: 8 * A + 4096}),             # the next row
    (ALIAS, "out overlaps x", {3: 8 * A, 4: 2048}),           # x, but with other rows
    (ALIAS, "out overlaps x", {2: 2048, 3: 8 * A + 4080, 4: 2048}),
    (ALIAS, "out overlaps table", {3: 20 * A + 16}),
    (ALIAS, "out overlaps positions", {3: 22 * A}),
])
def test_bad_rows_to_rotate_are_refused(q, code, needle, change):
    rows_refused(q, code, needle, rope(), altered(ROWS, change))


@pytest.mark.parametrize("code,needle,change", [
    (INVAL, "pairs", {1: 0}),
    (INVAL, "pairs", {1: 257}),
    (INVAL, "beyond", {2: -1}),
    (INVAL, "beyond", {3: -1}),
    (INVAL, "beyond", {2: 1 << 30, 3: 1}),
    (INVAL, "beyond", {3: 1 << 28}),
    (INVAL, "scale", {4: math.inf}),
    (INVAL, "scale", {4: 1e39}),
    (INVAL, "scale", {4: math.nan}),
    (INVAL, "null", {0: None}),
    (INVAL, "null", {5: None}),
    (ALIGN, "aligned", {5: 9 * A + 8}),
    (ALIGN, "aligned", {0: 8 * A + 2}),
    (ALIAS, "overlaps", {5: 8 * A}),
])
def test_bad_tables_are_refused(q, code, needle, change):
    args = altered((8 * A, 64, 0, 100, 1.0, 9 * A, None), change)
    assert q.library().apr_rope_table(*args) == code, q.apr_last_error()
    assert needle in q.apr_last_error()


@pytest.mark.parametrize("scale", [2.0 ** -101, -(2.0 ** -101), 1e-300, 5e-324])
def test_tables_of_scales_whose_roundings_float32_does_not_hold_are_refused(q, scale):
    assert q.library().apr_rope_table(8 * A, 64, 0, 100, scale, 9 * A, None) == INVAL
    assert "scale" in q.apr_last_error()


# rope, type, k, v, ld, k_norm, q, ldq, q_out, ldqo, heads, q_norm, eps, stream
def append(**change):
    return (rope(**change), 0, 8 * A, 9 * A, 256, None, 10 * A, 1024, 11 * A, 1024, 8, None, 0.0, None)


@pytest.mark.parametrize("code,needle,change", CACHE_AND_ROWS + WITH_ROWS)
def test_bad_caches_are_refused_by_the_rotating_append(q, code, needle, change):
    refused(q, "apr_rope_kv8_append", code, needle, change, append())


@pytest.mark.parametrize("code,needle,change", BAD_ROPES + [(INVAL, "null", dict(positions=None, num_axes=2, pair_axis=23 * A))])
def test_bad_rotations_are_refused_by_the_append(q, code, needle, change):
    refused(q, "apr_rope_kv8_append", code, needle, {}, append(**change))


@pytest.mark.parametrize("code,needle,change", [
    (INVAL, "element type", {1: 8}),
    (INVAL, "ld=255", {4: 255}),
    (INVAL, "null", {2: None}),
    (ALIGN, "16-byte", {3: 9 * A + 4}),
    (ALIGN, "norm", {5: 30 * A + 8}),
    (ALIGN, "norm", {11: 30 * A + 8}),
    (INVAL, "without", {6: None}),
    (INVAL, "without", {8: None}),
    (INVAL, "strides", {7: 1020}),
    (INVAL, "num_heads", {10: 0}),
    (INVAL, "eps", {12: -1.0}),
    (ALIAS, "q_out overlaps q", {8: 10 * A + 16}),
    (ALIAS, "q_out overlaps k", {8: 8 * A}),
    (ALIAS, "q_out overlaps V", {8: 2 * A}),
    (ALIAS, "q_out overlaps lens", {8: 6 * A}),
    (ALIAS, "K overlaps k", {2: A + 64}),
    (ALIAS, "V overlaps q", {6: 2 * A + 64}),
    (ALIAS, "overlaps table", {8: 20 * A}),
])
def test_bad_arguments_of_the_rotating_append_are_refused(q, code, needle, change):
    refused(q, "apr_rope_kv8_append", code, needle, {}, altered(append(), change))


PREFILL = DECODE[:7] + (None,)  # type, q, ldq, out, ldo, heads, scale, stream


@pytest.mark.parametrize("code,needle,change", CACHE_AND_ROWS + WITH_ROWS)
def test_bad_caches_are_refused_by_the_prefill_attention(q, code, needle, change):
    refused(q, "apr_kv8_prefill_attention", code, needle, change, PREFILL)


@pytest.mark.parametrize("code,needle,change", [
    (INVAL, "element type", {0: 8}),
    (INVAL, "num_heads", {5: 7}),
    (INVAL, "num_heads", {5: 0}),
    (INVAL, "ldq", {2: 1020}),
    (INVAL, "ldo", {4: 1020}),
    (INVAL, "scale", {6: -1.0}),
    (INVAL, "scale", {6: math.nan}),
    (INVAL, "null", {1: None}),
    (INVAL, "null", {3: None}),
    (ALIGN, "16-byte", {2: 1026}),
    (ALIGN, "16-byte", {3: 9 * A + 4}),
    (ALIAS, "out overlaps q", {3: 8 * A}),
    (ALIAS, "out overlaps V", {3: 2 * A}),
    (ALIAS, "out overlaps page_table", {3: 5 * A}),
])
def test_bad_prefill_attention_is_refused(q, code, needle, change):
    refused(q, "apr_kv8_prefill_attention", code, needle, {}, altered(PREFILL, change))


def test_sizes_that_no_64_bits_count_are_refused(q):
    refused(q, "apr_kv8_prefill_attention", INVAL, "beyond", dict(num_rows=1 << 24, table_ld=1 << 24, num_kv_heads=1),
            altered(PREFILL, {5: 65536, 1: 1 << 40, 3: 1 << 60, 2: 1 << 23, 4: 1 << 23}))


def test_empty_calls_do_nothing(q):
    lib, none = q.library(), dict(K=None, V=None, k_scale=None, v_scale=None, page_table=None, lens=None, row_start=None)
    for change in (dict(none, num_seqs=0, num_rows=0), dict(none, row_start=7 * A, num_rows=0)):
        c, r = cache_and_rows(q, **change)
        assert lib.apr_rope_kv8_append(c, r, *append()) == 0
        assert lib.apr_kv8_prefill_attention(c, r, *PREFILL) == 0
    assert lib.apr_rope_rows(rope(), *altered(ROWS, {5: 0, 1: None, 3: None})) == 0
    assert lib.apr_rope_table(None, 64, 0, 0, 1.0, None, None) == 0


def test_good_arguments_reach_the_device_check(q):
    import torch

    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    lib = q.library()
    c, r = cache_and_rows(q)
    assert lib.apr_kv8_prefill_attention(c, r, *PREFILL) == DEVICE
    assert lib.apr_rope_table(8 * A, 64, 0, 100, 1.0, 9 * A, None) == DEVICE
    for args in (ROWS, altered(ROWS, {3: 8 * A}), altered(ROWS, {2: 2048, 3: 8 * A + 4096, 4: 2048}), altered(ROWS, {7: 512, 2: 4096, 4: 4096})):
        assert lib.apr_rope_rows(rope(), *args) == DEVICE, q.apr_last_error()  # in place; another slice of wider rows
    slices = altered(append(), {2: 10 * A + 4096, 3: 10 * A + 5120, 4: 1536, 7: 1536, 8: 10 * A, 9: 1536})
    for args in (append(), slices, altered(append(positions=None), {6: None, 8: None, 10: 0})):
        assert lib.apr_rope_kv8_append(c, r, *args) == DEVICE, q.apr_last_error()


# ---------------------------------------------------------------- the binding
def devices(q):
    import torch

    I32, U8 = torch.int32, torch.uint8
    rows = dict(page_table=on(0, 2, 4, dtype=I32), lens=on(0, 2, dtype=I32), row_start=on(0, 3, dtype=I32))
    turn = q.Rope(on(0, 100, 32, 2), pair_axis=on(0, 32, dtype=U8))
    at = dict(positions=on(0, 2, 5, dtype=I32))
    norms = dict(k_norm=on(0, 64), q_norm=on(0, 64))
    more = dict(q=on(0, 5, 256), q_out=on(0, 5, 256))
    return [(lambda **t: q.apr_rope_table(t["inv_freq"], t["table"]), dict(inv_freq=on(0, 32), table=on(0, 100, 32, 2))),
            (lambda **t: q.apr_rope_rows(turn, t["positions"], t["x"], t["out"], 4, 64, norm=t["norm"]), dict(at, x=on(0, 5, 256), out=on(0, 5, 256), norm=on(0, 64))),
            (lambda **t: q.apr_rope_kv8_append(cache_on(q, 0), rope=turn, num_heads=4, **t), dict(rows, k=on(0, 5, 128), v=on(0, 5, 128), **at, **norms, **more)),
            (lambda **t: q.apr_kv8_prefill_attention(cache_on(q, 0), num_heads=4, **t), dict(rows, q=on(0, 5, 256), out=on(0, 5, 256)))]


@pytest.fixture
def bindings(q, monkeypatch):
    from quantized_weight_prefill_q4_gb300 import kv8, rope as module

    monkeypatch.setattr(kv8, "_lib", Unreached())
    monkeypatch.setattr(module, "_lib", Unreached())
    monkeypatch.setattr(kv8, "_current_device", lambda: 0)
    monkeypatch.setattr(kv8, "_raw_stream", lambda index: 0)
    return kv8


@pytest.mark.parametrize("which", range(4))
def test_tensors_of_another_device_are_refused(q, bindings, which):
    call, tensors = devices(q)[which]
    with pytest.raises(AssertionError, match="was called"):  # all on one device: the library is reached
        call(**tensors)
    for name, t in tensors.items():
        if which == 0 and name == "table":
            continue  # (the call's device is the table's)
        other = on(1, *t.shape, dtype=t.dtype)
        with pytest.raises(ValueError, match=f"{name}: tensor is on device 1"):
            call(**{**tensors, name: other})


@pytest.mark.parametrize("which", range(4))
def test_another_device_than_the_current_one_is_refused(q, bindings, which, monkeypatch):
    call, tensors = devices(q)[which]
    monkeypatch.setattr(bindings, "_current_device", lambda: 2)
    with pytest.raises(ValueError, match="device 0, the current device is 2"):
        call(**tensors)


def test_binding_refuses_tensors_that_do_not_fit(q, bindings):
    import torch

    I32 = torch.int32
    turn = q.Rope(on(0, 100, 32, 2))
    x, out = on(0, 5, 256), on(0, 5, 256)
    for positions in (on(0, 4, dtype=I32), on(0, 2, 4, dtype=I32), on(0, 5), None):
        with pytest.raises((ValueError, TypeError), match="positions"):
            q.apr_rope_rows(turn, positions, x, out, 4, 64)
    with pytest.raises(ValueError, match="norm"):
        q.apr_rope_rows(turn, on(0, 5, dtype=I32), x, out, 4, 64, norm=on(0, 63))
    with pytest.raises(ValueError, match="x: expected rows of 320"):
        q.apr_rope_rows(turn, on(0, 5, dtype=I32), x, out, 5, 64)
    with pytest.raises(ValueError, match="out: expected 5 rows"):
        q.apr_rope_rows(turn, on(0, 5, dtype=I32), x, on(0, 4, 256), 4, 64)
    with pytest.raises(ValueError, match="table"):
        q.Rope(on(0, 100, 32, 3))
    with pytest.raises(ValueError, match="pair_axis"):
        q.Rope(on(0, 100, 32, 2), pair_axis=on(0, 31, dtype=torch.uint8))
    with pytest.raises(ValueError, match="table"):
        q.apr_rope_table(on(0, 31), on(0, 100, 32, 2))
    rows = dict(page_table=on(0, 5, 4, dtype=I32), lens=on(0, 5, dtype=I32), rope=turn, k=on(0, 5, 128), v=on(0, 5, 128))
    with pytest.raises(ValueError, match="both or neither"):
        q.apr_rope_kv8_append(cache_on(q, 0), **rows, q=x)
    with pytest.raises(ValueError, match="q: expected"):
        q.apr_rope_kv8_append(cache_on(q, 0), **rows, q=on(0, 5, 255), q_out=out, num_heads=4)
    with pytest.raises(ValueError, match="q: expected 5 rows"):
        q.apr_rope_kv8_append(cache_on(q, 0), **rows, q=on(0, 4, 256), q_out=out, num_heads=4)
