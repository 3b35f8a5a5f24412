"""The decode example: prefill, 8-bit cache, decode steps and evictions run together.

A decode step over the 8-bit cache is the step of apr_prefill_layer over the float32 cache, but for the rounding of k and
v: each value within half a step of its page's scale, at most 1 / 254 of the page's largest magnitude. For rows of normal
values that is under 0.02 of their root mean square at the worst and a third of it on average, in V as it is and in K
through the scores, so the attention moves by a few hundredths; the row, to which the sublayers add, by less.
"""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("decode_kv8", os.path.join(ROOT, "examples", "decode_kv8.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_decode_steps_follow_the_float32_cache(q):
    e = example()
    decoder, X, (K, V) = e.start(seed=3)
    layer, steps = decoder.layer, 4
    caches = []  # the same sequences with float32 caches
    at = 0
    for n in e.PROMPTS:
        room = torch.zeros((2, n + steps, e.KV * e.DIM), device="cuda")
        room[0, :n], room[1, :n] = K[at:at + n], V[at:at + n]
        caches.append((n, room))
        at += n
    want = X.clone()
    for i in range(steps):
        before = want.clone()
        for b, (n, (kc, vc)) in enumerate(caches):
            q.apr_prefill_layer(q.APR_Q4_0, layer.qkv, layer.out, layer.gate, layer.up, layer.down, e.HIDDEN, e.INTER, e.HEADS,
                                e.KV, 1, n + i, layer.attn_norm, layer.ffn_norm, e.EPS, want[b:b + 1], kc, vc)
        decoder.step(X)
        q.apr_stream_status()
        rel = (X - want).norm() / (want - before).norm()
        assert rel <= 0.05, rel
        X.copy_(want)
    assert decoder.lens.tolist() == [n + steps for n in e.PROMPTS]
    # every position's weight: each step's row gives each KV head HEADS / KV in all
    total = decoder.weights.sum(-1)
    torch.testing.assert_close(total, torch.full_like(total, steps * e.HEADS / e.KV), rtol=1e-4, atol=0)


def test_evictions_keep_budget_and_recent_positions(q):
    e = example()
    decoder, X, _ = e.start(seed=4)
    for i in range(10):
        decoder.step(X)
    before = decoder.lens.tolist()
    kept = decoder.evict()
    q.apr_stream_status()
    assert decoder.lens.tolist() == [min(n, e.BUDGET) for n in before]
    for b, n in enumerate(before):
        if n > e.BUDGET:
            assert kept[b, :, -e.RECENT:].tolist() == [list(range(n - e.RECENT, n))] * e.KV
    pages = decoder.table.flatten().tolist()
    assert len(set(pages)) == len(pages) and not set(pages) & set(decoder.free)
    for i in range(20):
        decoder.step(X)
    q.apr_stream_status()
    assert torch.isfinite(X).all()


def test_example_runs(q, capsys):
    example().main(20)
    assert "after the eviction" in capsys.readouterr().out
