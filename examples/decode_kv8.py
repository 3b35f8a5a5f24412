"""Prefill, then decode over the 8-bit paged KV cache, one layer (random Q4_0 weights).

Three prompts of different lengths go through ``apr_prefill_layer``, which leaves their k and v rows in float32 caches.
``apr_kv8_append`` moves those into one paged 8-bit cache. Then the three sequences decode together, a row each: qkv
projection, append, attention (which adds up the weight that every position received), output projection, FFN; a
sequence that has grown past the budget is cut by ``apr_kv8_evict`` to its most recent positions and those that received
the most weight.

    python examples/decode_kv8.py [steps]
"""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import quantized_weight_prefill_q4_gb300 as q  # noqa: E402
import synth  # noqa: E402

HIDDEN, INTER, HEADS, KV, DIM, PAGE, EPS = 512, 1024, 8, 2, 256, 32, 1e-6
PROMPTS = (150, 37, 260)
BUDGET, RECENT = 128, 32


class Layer:
    """One layer's weights, as GGUF Q4_0 blocks on the GPU."""

    def __init__(self, seed=0):
        shapes = [((HEADS + 2 * KV) * DIM, HIDDEN), (HIDDEN, HEADS * DIM), (INTER, HIDDEN), (INTER, HIDDEN), (HIDDEN, INTER)]
        self.qkv, self.out, self.gate, self.up, self.down = (
            torch.from_numpy(synth.quantize(synth.Q4_0, synth.weight_f32(n, k, seed + i))).cuda() for i, (n, k) in enumerate(shapes))
        self.attn_norm, self.ffn_norm = torch.ones(HIDDEN, device="cuda"), torch.ones(HIDDEN, device="cuda")

    def prefill(self, X, K, V):
        """X [T][HIDDEN] in place; K and V [T][KV * DIM] take the rows' keys and values."""
        q.apr_prefill_layer(q.APR_Q4_0, self.qkv, self.out, self.gate, self.up, self.down, HIDDEN, INTER, HEADS, KV, X.shape[0], 0,
                            self.attn_norm, self.ffn_norm, EPS, X, K, V)


class Decoder:
    """The sequences' 8-bit cache, and what a decode step keeps from one token to the next."""

    def __init__(self, layer, prompts, most_tokens):
        self.layer, count = layer, len(prompts)
        self.width = -(-most_tokens // PAGE)
        self.cache = q.Kv8Cache.allocate(2 * count * self.width, KV, DIM, PAGE)
        self.free = list(range(2 * count * self.width))
        table = [[self.free.pop() for _ in range(self.width)] for _ in prompts]
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.lens = ints(table), ints(list(prompts))
        self.most = max(prompts)  # a bound on the lengths that needs no copy from the device
        self.weights = torch.zeros((count, KV, self.width * PAGE), device="cuda")
        self.qkv = torch.empty((count, (HEADS + 2 * KV) * DIM), device="cuda")
        self.attended = torch.empty((count, HEADS * DIM), device="cuda")

    def append_prompts(self, K, V, starts):
        """The prompts' packed k and v rows into the cache."""
        q.apr_kv8_append(self.cache, self.table, self.lens, K, V, row_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))

    def step(self, X):
        """One token of every sequence: X [sequences][HIDDEN] in place."""
        n, layer = X.shape[0], self.layer
        self.lens += 1
        self.most += 1
        q.apr_qgemm_rmsnorm(q.APR_Q4_0, layer.qkv, self.qkv.shape[1], HIDDEN, X, n, self.qkv, layer.attn_norm, EPS)
        rows, keys, values = self.qkv.split((HEADS * DIM, KV * DIM, KV * DIM), 1)
        q.apr_kv8_append(self.cache, self.table, self.lens, keys, values)
        q.apr_kv8_attention(self.cache, self.table, self.lens, rows, self.attended, HEADS, max_len=self.most,
                            weights=self.weights, accumulate=True)
        q.apr_qgemm(q.APR_Q4_0, layer.out, HIDDEN, HEADS * DIM, self.attended, n, X, X)
        q.apr_ffn_sublayer(q.APR_Q4_0, layer.gate, layer.up, layer.down, HIDDEN, INTER, n, layer.ffn_norm, EPS, X)

    def evict(self):
        """Cuts the sequences that are over the budget. Their old pages become free; the positions kept are returned."""
        count, fresh_width = self.lens.numel(), -(-BUDGET // PAGE)
        fresh = torch.tensor([[self.free.pop() for _ in range(fresh_width)] for _ in range(count)], dtype=torch.int32, device="cuda")
        table, lens = torch.empty_like(self.table), torch.empty_like(self.lens)
        weights = torch.zeros_like(self.weights)
        kept = torch.empty((count, KV, BUDGET), dtype=torch.int32, device="cuda")
        q.apr_kv8_evict(self.cache, self.table, self.lens, self.weights, BUDGET, RECENT, fresh, table, lens, weights, kept,
                        max_len=self.most)
        # the pages that no table names any more, on the host, and room for further tokens behind the kept ones
        named = set(table.flatten().tolist())
        pages = set(self.table.flatten().tolist()) | set(fresh.flatten().tolist())
        self.free += sorted(pages - named)
        rows = [[p if p >= 0 else self.free.pop() for p in row] for row in table.tolist()]
        self.table = torch.tensor(rows, dtype=torch.int32, device="cuda")
        self.lens, self.weights, self.most = lens, weights, min(self.most, BUDGET)
        return kept


def start(seed=0, most_tokens=max(PROMPTS) + 64):
    """Prompts prefilled and in the 8-bit cache: (decoder, the prompts' last rows, their float32 k and v rows)."""
    layer = Layer(seed)
    starts = [sum(PROMPTS[:i]) for i in range(len(PROMPTS) + 1)]
    X = torch.from_numpy(synth.activations(starts[-1], HIDDEN, seed + 9)).cuda()
    K, V = (torch.empty((starts[-1], KV * DIM), device="cuda") for _ in range(2))
    for a, b in zip(starts, starts[1:]):
        layer.prefill(X[a:b], K[a:b], V[a:b])
    decoder = Decoder(layer, PROMPTS, most_tokens)
    decoder.append_prompts(K, V, starts)
    return decoder, X[[b - 1 for b in starts[1:]]].contiguous(), (K, V)


def main(steps=40):
    decoder, X, _ = start()
    for i in range(steps):
        decoder.step(X)
        X.mul_(1.0 / X.pow(2).mean(1, keepdim=True).sqrt())  # (in place of the rest of a model)
        if i % 16 == 15:
            before = decoder.lens.tolist()
            decoder.evict()
            print(f"step {i + 1}: {before} tokens, {decoder.lens.tolist()} after the eviction")
    q.apr_stream_status()
    print("lengths", decoder.lens.tolist(), "rms of the rows", [round(x, 4) for x in X.pow(2).mean(1).sqrt().tolist()])


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
