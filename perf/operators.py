"""The operators of the 8-bit key/value cache, as they are measured.

The cache holds K and V in pages of ``page`` tokens: codes int8 [pages][kv_heads][page][head_dim] and one float32
scale for each page and head, value = code * scale. A page table lists each sequence's pages; ``lens`` counts the
tokens that a sequence holds, the rows of the call included, so a call's n rows are the last n positions.

  append  quantises new k and v rows into the cache (a raised scale re-rounds what the page held)
  read    gives rows of the cache back as numbers
  attend  attention of each sequence's last n rows over its cache, with the weight that each position received
  evict   keeps, for each head, the positions of the largest weights and the most recent ones, in fresh pages

``own`` false: the plain forms below; true: the framework's calls. The cache's contents come back as the values that
they stand for, through ``read``.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step's rows for a full batch of slots, the 9B layer's heads (4 KV heads of 256), float32 rows as
        # the projections write them
        dict(name="append_step_64", kind="append", type="f32", seqs=64, lo=300, hi=20000, rows=1, heads=16, kv=4, dim=256, page=64),
        # a batch of prompts of different lengths, one of them joining pages that are partly full, rows a slice of a fused qkv buffer
        dict(name="append_prompts", kind="append", type="bf16", seqs=9, lo=201, hi=4500, rows=0, heads=32, kv=8, dim=128, page=64),
        # one long prompt of small heads
        dict(name="append_long", kind="append", type="f16", seqs=1, lo=50001, hi=50001, rows=0, heads=16, kv=8, dim=64, page=128),
        # a cached prefix handed to the float32 prompt attention (16 query heads over 4 KV heads of 256)
        dict(name="read_prefix", kind="read", type="f32", seqs=1, lo=6007, hi=6007, rows=0, heads=16, kv=4, dim=256, page=64),
        # the caches of a batch moved out as 16-bit rows
        dict(name="read_batch", kind="read", type="bf16", seqs=12, lo=100, hi=16000, rows=0, heads=32, kv=8, dim=128, page=32),
        # one user's next token after a short prompt: latency counts
        dict(name="attend_one_short", kind="attend", type="f32", seqs=1, lo=700, hi=700, rows=1, heads=16, kv=4, dim=256, page=64, weights=False),
        # a serving batch of ragged lengths
        dict(name="attend_batch", kind="attend", type="bf16", seqs=48, lo=130, hi=9000, rows=1, heads=32, kv=8, dim=128, page=64, weights=False),
        # few users with long caches
        dict(name="attend_long", kind="attend", type="f16", seqs=3, lo=100003, hi=131000, rows=1, heads=16, kv=4, dim=256, page=64, weights=False),
        # a decode step that also keeps each position's weight for eviction
        dict(name="attend_weights", kind="attend", type="f32", seqs=16, lo=2000, hi=12000, rows=1, heads=32, kv=4, dim=128, page=64, weights=True),
        # the last rows of a prompt as the window that rates its positions (or a draft of several tokens), small heads
        dict(name="attend_window", kind="attend", type="bf16", seqs=4, lo=5000, hi=8200, rows=9, heads=16, kv=8, dim=64, page=32, weights=True),
        # one sequence over its budget
        dict(name="evict_one", kind="evict", type="f32", seqs=1, lo=4099, hi=4099, budget=2048, recent=64, heads=16, kv=4, dim=256, page=64),
        # a batch, most of it over its budget, some of it not
        dict(name="evict_batch", kind="evict", type="bf16", seqs=10, lo=3500, hi=33000, budget=4100, recent=300, heads=32, kv=8, dim=128, page=64),
    ]


def draw(rng):
    """One more case of the same ranges: at most about 2.5 million rows of one KV head, 128 bytes each."""
    kind = rng.choice(("append", "read", "attend", "attend", "evict"))
    dim = rng.choice((64, 128, 256))
    kv = rng.choice((1, 2, 4, 8))
    c = dict(kind=kind, type=rng.choice(("f32", "f16", "bf16")), dim=dim, kv=kv, heads=kv * rng.choice((1, 2, 4, 7, 8)),
             page=rng.choice((32, 64, 128)), seqs=int(2 ** rng.uniform(0, 6)))
    most = (2_500_000 if kind == "attend" else 600_000) * 128 // (dim * kv * c["seqs"])
    c["hi"] = max(40, int(2 ** rng.uniform(6, 17)))
    c["hi"] = min(c["hi"], most)
    c["lo"] = max(33, int(c["hi"] * rng.uniform(0.05, 1.0)))
    c["hi"] = max(c["hi"], c["lo"])
    if kind == "evict":
        c["budget"] = max(16, int(c["hi"] * rng.uniform(0.1, 0.9)))
        c["recent"] = int(c["budget"] * rng.uniform(0.0, 0.5))
    elif kind == "attend":
        c["rows"] = rng.choice((1, 1, 1, 2, 5, 8))
        c["weights"] = rng.random() < 0.4
    else:
        c["rows"] = rng.choice((0, 0, 1, 17))
    return c


def _lens(case):
    """The sequences' lengths, spread from lo to hi (evenly over their logarithm)."""
    lo, hi = case["lo"], case["hi"]
    return [round(lo * (hi / lo) ** ((0.5 + 0.6180339887498949 * b) % 1.0)) if case["seqs"] > 1 else hi for b in range(case["seqs"])]


def _rows(case):
    """The call's rows of each sequence: its last ones; 0 in the case: all, but for the first sequence's first 37 when tokens join a page."""
    lens = _lens(case)
    if case.get("rows", 0):
        return [min(case["rows"], n) for n in lens]
    if case["kind"] == "append":
        lens[0] -= min(37, lens[0] - 1) if len(lens) > 1 else 0
    return lens


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B, kv, dim, page, heads = case["seqs"], case["kv"], case["dim"], case["page"], case["heads"]
    lens, dtype = _lens(case), TYPES[case["type"]]
    width = -(-max(lens) // page)  # pages of the longest sequence
    used = sum(-(-n // page) for n in lens)
    fresh_width = -(-case["budget"] // page) if case["kind"] == "evict" else 0
    pages = used + fresh_width * B + 3
    order = torch.randperm(pages, device=dev, generator=gen).to(torch.int32).cpu().tolist()  # pages in no order, as a long-running server has them
    table = [[0] * width for _ in range(B)]
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[b][i] = order.pop()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"kind": case["kind"], "kv": kv, "dim": dim, "page": page, "heads": heads, "dtype": dtype, "max_len": max(lens),
         "page_table": ints(table), "lens": ints(lens)}
    for name in ("K", "V"):
        codes = torch.empty((pages, kv, page, dim), dtype=torch.int8, device=dev)
        for at in range(0, pages, 4096):
            part = codes[at:at + 4096]
            part.copy_(torch.randn(part.shape, generator=gen, device=dev, dtype=torch.float16).mul_(36.0).round_().clamp_(-127, 127))
        s[name] = codes
        s[name.lower() + "_scale"] = torch.exp(0.3 * torch.randn((pages, kv), generator=gen, device=dev)) * 0.028
    if case["kind"] in ("append", "read"):
        rows = _rows(case)
        s["rows"], s["max_rows"] = sum(rows), max(rows)
        s["row_start"] = None if max(rows) == 1 else ints(_starts(rows))
        if case["kind"] == "append":
            # the k and v rows: slices of one buffer of q, k and v
            qkv = torch.randn((s["rows"], (heads + 2 * kv) * dim), generator=gen, device=dev).to(dtype)
            s["k"], s["v"] = qkv[:, heads * dim:(heads + kv) * dim], qkv[:, (heads + kv) * dim:]
            # what comes back: every page that the call touched
            back = [n - (n - r) // page * page for n, r in zip(lens, rows)]
            s["back_rows"], s["back_max"], s["back_start"] = sum(back), max(back), ints(_starts(back))
    elif case["kind"] == "attend":
        rows = _rows(case)
        s["rows"], s["max_rows"] = sum(rows), max(rows)
        s["row_start"] = None if max(rows) == 1 else ints(_starts(rows))
        s["q"] = torch.randn((s["rows"], heads * dim), generator=gen, device=dev).to(dtype)
        s["weights"] = case["weights"]
    else:
        s["budget"], s["recent"] = case["budget"], case["recent"]
        # accumulated weights: a few large, most small, those that underflowed zero
        w = torch.exp(3.0 * torch.randn((B, kv, max(lens)), generator=gen, device=dev) - 4.0)
        s["acc"] = torch.where(w < 1e-4, torch.zeros_like(w), w)
        s["fresh"] = ints([[order.pop() for _ in range(fresh_width)] for _ in range(B)])
        kept = [min(n, case["budget"]) for n in lens]
        s["back_rows"], s["back_max"], s["back_start"] = sum(kept), max(kept), ints(_starts(kept))
    return s


# ---------------------------------------------------------------- plain forms
def _place(s, table, lens, row_start, rows):
    """(page, slot, first) of each row of the call: the rows are the last positions of their sequences."""
    at = torch.arange(rows, device=lens.device)
    if row_start is None:
        seq, first = at, lens.long() - 1
        pos = first
    else:
        seq = torch.bucketize(at, row_start[1:].long(), right=True)
        first = lens.long()[seq] - (row_start[1:] - row_start[:-1]).long()[seq]
        pos = first + at - row_start.long()[seq]
    return table.long()[seq, pos // s["page"]], pos % s["page"]


def _touched(s):
    """The pages that the call's rows go to, a sequence's last one as often as it has fewer than the others."""
    lens, n = s["lens"].long(), 1 if s["row_start"] is None else (s["row_start"][1:] - s["row_start"][:-1]).long()
    i = torch.arange(s["max_rows"] // s["page"] + 2, device=lens.device)
    i = torch.minimum(((lens - n) // s["page"])[:, None] + i, ((lens - 1) // s["page"])[:, None])
    return torch.gather(s["page_table"].long(), 1, i).reshape(-1)


def _quantise(x, scale):
    """Codes of float32 values: the nearest whole number to x / scale, ties to the even one, decided in 64 bits."""
    d = scale.double()
    return torch.where(d > 0, torch.round(x.double() / torch.where(d > 0, d, 1.0)), 0.0).clamp(-127, 127).to(torch.int8)


def _append_one(s, codes, scale, x, page, slot, touched):
    pages, kv = scale.shape
    x = x.float().reshape(-1, kv, s["dim"])
    where = page[:, None].expand(-1, kv)
    need = torch.full_like(scale, -1.0).scatter_reduce(0, where, x.abs().amax(-1), "amax")
    fresh = torch.zeros(pages, device=scale.device).scatter_reduce(0, page, (slot == 0).float(), "amax")[:, None] > 0
    old = torch.where(fresh, 0.0, scale)
    new = torch.where(need >= 0, torch.maximum(old, (need.double() / 127).float()), scale)
    before, after = old[touched][:, :, None, None], new[touched][:, :, None, None]
    codes[touched] = torch.where((after > before) & (before > 0), _quantise(codes[touched].float() * before, after), codes[touched])
    codes[page, :, slot] = _quantise(x, new[page][:, :, None])
    scale.copy_(new)


def _read_plain(s, table, lens, row_start, rows):
    page, slot = _place(s, table, lens, row_start, rows)
    return tuple((s[n][page, :, slot].float() * s[n.lower() + "_scale"][page][:, :, None]).to(s["dtype"]).reshape(rows, -1) for n in ("K", "V"))


def _whole(s, name, kv, dim):
    """[B][kv][positions][dim] of a cache in float32, every page of the tables."""
    t = s["page_table"].long()
    x = s[name][t].float() * s[name.lower() + "_scale"][t][..., None, None]
    return x.transpose(1, 2).reshape(t.shape[0], kv, -1, dim)


def _attend_plain(s):
    B, kv, dim, heads = s["lens"].numel(), s["kv"], s["dim"], s["heads"]
    group, N, lens = heads // kv, s["max_rows"], s["lens"].long()
    start = torch.arange(B + 1, device=lens.device) if s["row_start"] is None else s["row_start"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(N, device=lens.device)
    row = (start[:-1, None] + i).clamp(max=s["rows"] - 1)  # [B][N], rows past a sequence's n are dropped below
    q = s["q"].float().reshape(-1, kv, group, dim)[row].permute(0, 2, 1, 3, 4).reshape(B, kv, N * group, dim)
    scores = torch.matmul(q, _whole(s, "K", kv, dim).transpose(-1, -2)).reshape(B, kv, N, group, -1) * (1.0 / math.sqrt(dim))
    sees = torch.arange(scores.shape[-1], device=lens.device) < ((lens - n)[:, None] + i + 1)[..., None]  # [B][N][positions]
    sees = (sees & (i < n[:, None])[..., None])[:, None, :, None]
    scores = torch.where(sees, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    out = torch.matmul(p.reshape(B, kv, N * group, -1), _whole(s, "V", kv, dim)).reshape(B, kv, N, group, dim)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, N, heads * dim)
    at = torch.arange(s["rows"], device=lens.device)
    seq = torch.bucketize(at, start[1:], right=True)
    out = out[seq, at - start[seq]].to(s["dtype"])
    return {"out": out, "weights": p.sum((2, 3))[..., :s["max_len"]].contiguous()} if s["weights"] else {"out": out}


def _evict_plain(s):
    lens, budget, recent, kv, page, dim = s["lens"].long(), s["budget"], s["recent"], s["kv"], s["page"], s["dim"]
    B, L = lens.numel(), s["acc"].shape[-1]
    at = torch.arange(L, device=lens.device)
    over = lens > budget
    kept_len = lens.clamp(max=budget)
    rank = torch.where(at >= (lens - recent)[:, None, None], math.inf, s["acc"])
    rank = torch.where(over[:, None, None], rank, math.inf)
    rank = torch.where(at < lens[:, None, None], rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices  # equal weights: the lowest position first
    k = min(budget, L)
    live = torch.arange(k, device=lens.device) < kept_len[:, None, None]
    kept = torch.sort(torch.where(live, order[..., :k], L), dim=-1).values
    src = kept.clamp(max=L - 1)
    weights = torch.where(live, torch.gather(s["acc"], 2, src), 0.0)
    b = torch.arange(B, device=lens.device)[:, None, None]
    g = torch.arange(kv, device=lens.device)[None, :, None]
    src_page = s["page_table"].long()[b, src // page]
    wide = s["fresh"].shape[1]
    for name in ("K", "V"):
        scale = s[name.lower() + "_scale"]
        x = s[name][src_page, g, src % page].float() * scale[src_page, g][..., None]
        x = torch.where(live[..., None], x, 0.0)
        x = torch.nn.functional.pad(x, (0, 0, 0, wide * page - k)).reshape(B, kv, wide, page, dim)
        new = (x.abs().amax((3, 4)).double() / 127).float()
        to = s["fresh"].long()[over]
        s[name][to] = _quantise(x, new[..., None, None])[over].transpose(1, 2)
        scale[to] = new[over].transpose(1, 2)
    pad = budget - k
    kept = torch.nn.functional.pad(torch.where(live, kept, -1), (0, pad), value=-1).to(torch.int32)
    weights = torch.nn.functional.pad(weights, (0, pad))
    width = s["page_table"].shape[1]
    fresh = torch.nn.functional.pad(s["fresh"], (0, max(0, width - wide)))[:, :width]
    table = torch.where(over[:, None], fresh, s["page_table"])
    table = torch.where(torch.arange(width, device=lens.device) < ((kept_len + page - 1) // page)[:, None], table, -1)
    lens_out = kept_len.to(torch.int32)
    k_back, v_back = _read_plain(s, table, lens_out, s["back_start"], s["back_rows"])
    return {"kept": kept, "weights": weights, "table": table.to(torch.int32), "lens": lens_out, "k": k_back, "v": v_back}


def _run_plain(s):
    if s["kind"] == "append":
        page, slot = _place(s, s["page_table"], s["lens"], s["row_start"], s["rows"])
        touched = _touched(s)
        _append_one(s, s["K"], s["k_scale"], s["k"], page, slot, touched)
        _append_one(s, s["V"], s["v_scale"], s["v"], page, slot, touched)
        return _read_plain(s, s["page_table"], s["lens"], s["back_start"], s["back_rows"])
    if s["kind"] == "read":
        return _read_plain(s, s["page_table"], s["lens"], s["row_start"], s["rows"])
    return _attend_plain(s) if s["kind"] == "attend" else _evict_plain(s)


# ---------------------------------------------------------------- the framework's calls
def _run_own(s):
    import quantized_weight_prefill_q4_gb300 as q

    cache = q.Kv8Cache(s["K"], s["V"], s["k_scale"], s["v_scale"])
    table, lens, kind, wide = s["page_table"], s["lens"], s["kind"], s["kv"] * s["dim"]
    empty = lambda *shape, dtype=s["dtype"]: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if kind == "append":
        q.apr_kv8_append(cache, table, lens, s["k"], s["v"], row_start=s["row_start"], max_rows=s["max_rows"])
        k, v = empty(s["back_rows"], wide), empty(s["back_rows"], wide)
        q.apr_kv8_read(cache, table, lens, k, v, row_start=s["back_start"], max_rows=s["back_max"])
        return k, v
    if kind == "read":
        k, v = empty(s["rows"], wide), empty(s["rows"], wide)
        q.apr_kv8_read(cache, table, lens, k, v, row_start=s["row_start"], max_rows=s["max_rows"])
        return k, v
    if kind == "attend":
        out = torch.empty_like(s["q"])
        weights = empty(lens.numel(), s["kv"], s["max_len"], dtype=torch.float32) if s["weights"] else None
        q.apr_kv8_attention(cache, table, lens, s["q"], out, s["heads"], row_start=s["row_start"], max_rows=s["max_rows"],
                            max_len=s["max_len"], weights=weights)
        return {"out": out, "weights": weights} if s["weights"] else {"out": out}
    B, kv, budget, i32 = lens.numel(), s["kv"], s["budget"], torch.int32
    kept, weights = empty(B, kv, budget, dtype=i32), empty(B, kv, budget, dtype=torch.float32)
    table_out, lens_out = torch.empty_like(table), torch.empty_like(lens)
    q.apr_kv8_evict(cache, table, lens, s["acc"], budget, s["recent"], s["fresh"], table_out, lens_out, weights, kept, max_len=s["max_len"])
    k, v = empty(s["back_rows"], wide), empty(s["back_rows"], wide)
    q.apr_kv8_read(cache, table_out, lens_out, k, v, row_start=s["back_start"], max_rows=s["back_max"])
    return {"kept": kept, "weights": weights, "table": table_out, "lens": lens_out, "k": k, "v": v}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    lens, kv, dim, heads, page = _lens(case), case["kv"], case["dim"], case["heads"], case["page"]
    size = 4 if case["type"] == "f32" else 2
    rows = _rows(case) if case["kind"] != "evict" else []
    row = 2 * kv * dim  # codes of one token's k and v
    scales = lambda tokens: 8 * kv * (-(-tokens // page))  # noqa: E731
    if case["kind"] == "append":
        back = [n - (n - r) // page * page for n, r in zip(lens, rows)]
        # the new rows in, their codes out; then the touched pages' codes in and their values out
        return {"bytes": sum(rows) * row * (size + 1) + sum(back) * row * (1 + size) + sum(2 * scales(n) for n in back), "flops": 2 * row * (sum(rows) + sum(back))}
    if case["kind"] == "read":
        return {"bytes": sum(rows) * row * (1 + size) + sum(scales(n) for n in rows), "flops": row * sum(rows)}
    if case["kind"] == "attend":
        seen = sum(n * r - r * (r - 1) // 2 for n, r in zip(lens, rows))
        out = 4 * kv * case["seqs"] * max(lens) if case["weights"] else 0
        return {"bytes": sum(lens) * row + sum(scales(n) for n in lens) + 2 * sum(rows) * heads * dim * size + out, "flops": 4 * seen * heads * dim}
    kept = [min(n, case["budget"]) for n in lens]
    moved = sum(k for n, k in zip(lens, kept) if n > case["budget"])
    # the weights of every position in; of the kept, weights and positions out, codes in and out; then the values back
    return {"bytes": 4 * kv * sum(lens) + 8 * kv * case["seqs"] * case["budget"] + moved * row * 2 + 2 * scales(moved) + sum(kept) * row * (1 + size) + sum(scales(k) for k in kept),
            "flops": row * (3 * moved + sum(kept))}


# ---------------------------------------------------------------- the definition in 64 bits
def _pages_of(s, name, b, count):
    """The first `count` tokens of sequence b as [count][kv][dim] float64 codes, and each token's scale [count][kv]."""
    ids = s["page_table"][b, : -(-count // s["page"])].long()
    codes = s[name].index_select(0, ids).to(torch.float64).permute(0, 2, 1, 3).reshape(-1, s["kv"], s["dim"])[:count]
    return codes, s[name.lower() + "_scale"].index_select(0, ids).to(torch.float64).repeat_interleave(s["page"], 0)[:count]


def _round_to_codes(values, page):
    """Float32 values [tokens][kv][dim] from a page's first slot on, quantised page by page: (codes, scale of each token), float64."""
    tokens = values.shape[0]
    full = torch.zeros((-(-tokens // page) * page,) + values.shape[1:], dtype=torch.float64, device=values.device)
    full[:tokens] = values
    full = full.reshape(-1, page, *values.shape[1:])
    scale = (full.abs().amax((1, 3)) / 127).float().double()
    codes = torch.round(full / scale[:, None, :, None]).nan_to_num(0.0).clamp(-127, 127)
    return codes.reshape(-1, *values.shape[1:])[:tokens], scale.repeat_interleave(page, 0)[:tokens]


def exact(case, seed):
    s = prepare(case, seed)
    lens, page, kv, dim = _lens(case), case["page"], case["kv"], case["dim"]
    if case["kind"] == "append":
        rows, got = _rows(case), {"k": [], "v": []}
        at = _starts(rows)
        for b, (n, r) in enumerate(zip(lens, rows)):
            first = (n - r) // page * page  # the first touched page's first position
            held = n - r - first
            for name in ("K", "V"):
                x = s[name.lower()][at[b]:at[b + 1]].double().reshape(r, kv, dim)
                if held:
                    codes, scale = _pages_of(s, name, b, n - r)
                    codes, old = codes[first:], scale[first]
                    here = x[: page - held]
                    want = (here.abs().amax((0, 2)) / 127).float().double()
                    new = torch.maximum(old, want)
                    kept = (codes * old[:, None]).float().double()
                    codes = torch.cat([torch.round(kept / new[:, None]), torch.round(here / new[:, None])]).clamp(-127, 127)
                    values = [codes * new[:, None]]
                    x = x[page - held:]
                else:
                    values = []
                if x.shape[0]:
                    codes, scale = _round_to_codes(x, page)
                    values.append(codes * scale[..., None])
                got[name.lower()].append(torch.cat(values).reshape(-1, kv * dim))
        return torch.cat(got["k"]), torch.cat(got["v"])
    if case["kind"] == "read":
        rows, got = _rows(case), []
        for name in ("K", "V"):
            parts = []
            for b, (n, r) in enumerate(zip(lens, rows)):
                codes, scale = _pages_of(s, name, b, n)
                parts.append((codes[n - r:] * scale[n - r:][..., None]).reshape(r, kv * dim))
            got.append(torch.cat(parts))
        return tuple(got)
    if case["kind"] == "attend":
        rows, group = _rows(case), case["heads"] // kv
        at, outs = _starts(rows), []
        weights = torch.zeros((len(lens), kv, max(lens)), dtype=torch.float64, device="cuda") if case["weights"] else None
        for b, (n, r) in enumerate(zip(lens, rows)):
            (ck, sk), (cv, sv) = _pages_of(s, "K", b, n), _pages_of(s, "V", b, n)
            q = s["q"][at[b]:at[b + 1]].double().reshape(r, kv, group, dim)
            heads = []
            for g in range(kv):
                k, v = ck[:, g] * sk[:, g, None], cv[:, g] * sv[:, g, None]
                scores = q[:, g] @ k.T / math.sqrt(dim)  # [r][group][n]
                for i in range(r):
                    scores[i, :, n - r + i + 1:] = -math.inf
                p = torch.softmax(scores, -1)
                heads.append(p @ v)
                if weights is not None:
                    weights[b, g, :n] = p.sum((0, 1))
            outs.append(torch.stack(heads, 1).reshape(r, -1))
        return {"out": torch.cat(outs), "weights": weights} if case["weights"] else {"out": torch.cat(outs)}
    k_rows, v_rows, budget = [], [], case["budget"]
    weights = torch.zeros((len(lens), kv, budget), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        picks = []
        for g in range(kv):
            w = s["acc"][b, g, :n].double()
            if n > budget:
                old = n - case["recent"]
                # the weight above which positions are surely kept, then the first of the equal ones
                need = budget - case["recent"]
                border = torch.topk(w[:old], need).values[-1] if need else torch.tensor(math.inf, device=w.device)
                above, equal = w[:old] > border, w[:old] == border
                take = above | (equal & (torch.cumsum(equal, 0) <= need - above.sum()))
                pick = torch.cat([torch.nonzero(take)[:, 0], torch.arange(old, n, device=w.device)])
            else:
                pick = torch.arange(n, device=w.device)
            weights[b, g, : pick.numel()] = w[pick]
            picks.append(pick)
        for name, to in (("K", k_rows), ("V", v_rows)):
            codes, scale = _pages_of(s, name, b, n)
            x = (codes * scale[..., None]).float().double()
            x = torch.stack([x[picks[g], g] for g in range(kv)], 1)
            if n > budget:
                codes, scale = _round_to_codes(x, page)
                x = codes * scale[..., None]
            to.append(x.reshape(-1, kv * dim))
    return {"kept": None, "weights": weights, "table": None, "lens": None, "k": torch.cat(k_rows), "v": torch.cat(v_rows)}
