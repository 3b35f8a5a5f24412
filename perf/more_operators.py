"""The operators between a chunk's qkv projection and its attention over the 8-bit cache, as they are measured.

  table   cosines and sines of position times frequency, which the rotations read
  rope    rotates rows of heads by their positions (one axis or several), behind an optional norm of each head
  append  rotates k rows on their way into the 8-bit paged cache, appends v rows, and rotates the q rows beside them
  attend  causal attention of chunks of new rows over their sequences' 8-bit paged caches

A rotation turns pair i of a head, dims (i, i + rot / 2) or (2 i, 2 i + 1), by the angle position[axis of i] * inv_freq[i];
dims past ``rot`` pass. Roundings of a rotation: cosine and sine to float32 (the table), 1 / rms of a head to float32, every
product, sum and difference to float32, the result to the rows' type; what is appended are those rounded rows.

The cache holds K and V in pages of ``page`` tokens: codes int8 [pages][kv_heads][page][head_dim] and one float32 scale
for each page and head, value = code * scale. A page table lists each sequence's pages; ``lens`` counts the
tokens that a sequence holds, the rows of the call included, so a call's n rows are the last n positions. The appended
contents come back as the values that they stand for, through a read.

``own`` false: the plain forms below; true: the framework's calls.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # the table of a short context, built when a model is loaded
        dict(name="table_short", kind="table", first=0, positions=8192, pairs=32, scale=1.0, base=10000.0),
        # the table of a long context with the cosines and sines of a stretched rotation scaled
        dict(name="table_long", kind="table", first=1, positions=400003, pairs=128, scale=1.1386294, base=5000000.0),
        # one user's next token: 16 query heads of 256, a quarter of the dims rotated, float32 rows as the projections write them
        dict(name="rope_step", kind="rope", type="f32", rows=1, heads=16, dim=256, rot=64, layout="halves", axes=1, norm=True),
        # patches of a large image, two axes, heads of 72
        dict(name="rope_image", kind="rope", type="f16", rows=5329, heads=16, dim=72, rot=72, layout="pairs", axes=2, norm=False),
        # a long prompt with images in it: time, height and width, normed heads
        dict(name="rope_prompt", kind="rope", type="bf16", rows=16390, heads=32, dim=128, rot=128, layout="halves", axes=3, norm=True),
        # one decode step's rows for a full batch of slots, the 9B layer's heads (16 over 4 KV heads of 256)
        dict(name="append_step_64", kind="append", type="f32", seqs=64, lo=300, hi=20000, rows=1, heads=16, kv=4, dim=256, page=64, rot=64, layout="halves", axes=1, norm=True),
        # chunks of a batch of prompts, joining pages that are partly full, rows slices of a fused qkv buffer
        dict(name="append_chunks", kind="append", type="bf16", seqs=9, lo=701, hi=9000, rows=2048, heads=32, kv=8, dim=128, page=64, rot=128, layout="halves", axes=3, norm=True),
        # one long prompt of small heads
        dict(name="append_long", kind="append", type="f16", seqs=1, lo=50001, hi=50001, rows=50001, heads=16, kv=8, dim=64, page=128, rot=64, layout="pairs", axes=1, norm=False),
        # the end of a prompt whose beginning was cached: latency counts
        dict(name="attend_tail", kind="attend", type="f16", seqs=1, lo=731, hi=731, rows=37, mixed=False, heads=8, kv=2, dim=64, page=32),
        # one chunk of a prompt, the 9B layer's heads, float32 rows as the projections write them
        dict(name="attend_chunk", kind="attend", type="f32", seqs=1, lo=6007, hi=6007, rows=512, mixed=False, heads=16, kv=4, dim=256, page=64),
        # a server's step: chunks of some prompts beside single tokens of other sequences
        dict(name="attend_mixed", kind="attend", type="bf16", seqs=7, lo=900, hi=9000, rows=1024, mixed=True, heads=32, kv=8, dim=128, page=64),
        # a large chunk far into a long document
        dict(name="attend_long", kind="attend", type="bf16", seqs=1, lo=40011, hi=40011, rows=2048, mixed=False, heads=32, kv=8, dim=128, page=128),
    ]


def draw(rng):
    """One more case of the same ranges; none costs more than the largest listed of its kind."""
    kind = rng.choice(("table", "rope", "append", "attend", "attend"))
    log = lambda lo, hi: int(2 ** rng.uniform(math.log2(lo), math.log2(hi)))  # noqa: E731
    if kind == "table":
        pairs = 4 * rng.randint(2, 32)
        return dict(kind=kind, first=rng.choice((0, 1, log(2, 500000))), positions=log(100, 50_000_000 // pairs), pairs=pairs,
                    scale=rng.choice((1.0, rng.uniform(0.8, 1.4))), base=10.0 ** rng.uniform(4, 7))
    c = dict(kind=kind, type=rng.choice(("f32", "f16", "bf16")))
    if kind != "attend":
        c.update(layout=rng.choice(("halves", "pairs")), axes=rng.choice((1, 1, 2, 3, 4)), norm=rng.random() < 0.5)
    if kind == "rope":
        c.update(dim=8 * rng.randint(4, 32), heads=rng.choice((1, 2, 8, 12, 16, 28, 32)))
        c.update(rot=c["dim"] if rng.random() < 0.7 else 8 * rng.randint(1, c["dim"] // 8), rows=log(1, 60_000_000 // (c["dim"] * c["heads"])))
        return c
    kv = rng.choice((1, 2, 4, 8))
    c.update(dim=rng.choice((64, 128, 256)), kv=kv, heads=kv * rng.choice((1, 2, 4, 7, 8)), page=rng.choice((32, 64, 128, 256)), seqs=log(1, 20))
    if kind == "append":
        c["rot"] = c["dim"] if rng.random() < 0.7 else 8 * rng.randint(1, c["dim"] // 8)
        c["rows"] = log(1, max(2, 30_000_000 // (c["dim"] * (c["heads"] + 2 * kv) * c["seqs"])))
        c["hi"] = c["rows"] + log(1, 10_000)
        c["lo"] = max(1, int(c["hi"] * rng.uniform(0.1, 1.0)))
        return c
    c["mixed"] = rng.random() < 0.4
    c["rows"] = log(1, 2500)
    c["hi"] = c["rows"] + log(1, 30_000)
    # scores of the padded batch: 1.5e9; products: those of the largest case
    while c["seqs"] * c["heads"] * c["rows"] * c["hi"] > 1_500_000_000 or c["seqs"] * c["kv"] * c["hi"] * c["dim"] > 400_000_000:
        c["seqs"], c["rows"], c["hi"] = max(1, c["seqs"] // 2), max(1, int(c["rows"] * 0.8)), max(2, int(c["hi"] * 0.8))
    c["lo"] = max(1, int(c["hi"] * rng.uniform(0.1, 1.0)))
    return c


def _lens(case):
    """The sequences' lengths, spread from lo to hi (evenly over their logarithm)."""
    lo, hi = case["lo"], case["hi"]
    return [round(lo * (hi / lo) ** ((0.5 + 0.6180339887498949 * b) % 1.0)) if case["seqs"] > 1 else hi for b in range(case["seqs"])]


def _rows(case):
    """The call's rows of each sequence, its last ones: chunks of different lengths, in a mixed batch every third sequence's next token."""
    spread = lambda b: round(case["rows"] * (1.0 - 0.5 * ((0.381966 * b) % 1.0)))  # noqa: E731
    return [1 if case.get("mixed") and b % 3 == 2 else max(1, min(n, spread(b))) for b, n in enumerate(_lens(case))]


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _inv_freq(pairs, base, dev):
    return (1.0 / base ** (torch.arange(pairs, dtype=torch.float64, device=dev) / pairs)).float()


def _table(inv_freq, first, positions, scale):
    """[positions][pairs][2] cosines and sines in float32; far positions times a frequency need 64 bits."""
    at = torch.arange(first, first + positions, dtype=torch.float64, device=inv_freq.device)
    angle = at[:, None] * inv_freq.double()
    return torch.stack((torch.cos(angle) * scale, torch.sin(angle) * scale), -1).float()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    kind = case["kind"]
    if kind == "table":
        # frequencies of a base, each off by a little, as scaled or learned ones are
        off = torch.exp(0.05 * torch.randn(case["pairs"], generator=gen, device=dev))
        return {"kind": kind, "inv_freq": _inv_freq(case["pairs"], case["base"], dev) * off, "first": case["first"], "positions": case["positions"], "scale": case["scale"]}
    dtype, dim, heads = TYPES[case["type"]], case["dim"], case["heads"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"kind": kind, "dtype": dtype, "dim": dim, "heads": heads}
    if kind != "attend":
        pairs = case["rot"] // 2
        s["rot"], s["halves"], s["axes"] = case["rot"], case["layout"] == "halves", case["axes"]
        reach = max(case["rows"], case.get("hi", 0)) + 1
        s["table"] = _table(_inv_freq(pairs, 1000000.0, dev), 0, reach, 1.0)
        # the axes of the pairs: neighbouring pairs' in turn, or one block after the other
        turn = torch.arange(pairs, device=dev) % case["axes"] if case["axes"] % 2 else torch.arange(pairs, device=dev) * case["axes"] // pairs
        s["pair_axis"] = turn.to(torch.uint8) if case["axes"] > 1 else None
        s["q_norm"], s["k_norm"] = (1.0 + 0.2 * torch.randn(dim, generator=gen, device=dev) if case["norm"] else None for _ in range(2))
    if kind == "rope":
        rows = case["rows"]
        s["x"] = (1.5 * torch.randn((rows, (heads + 2) * dim), generator=gen, device=dev)).to(dtype)[:, :heads * dim]  # a slice of a wider buffer
        s["positions"] = torch.randint(0, reach, (case["axes"], rows), generator=gen, device=dev, dtype=torch.int32)
        return s
    B, kv, page = case["seqs"], case["kv"], case["page"]
    lens, rows = _lens(case), _rows(case)
    width = -(-max(lens) // page)  # pages of the longest sequence
    used = sum(-(-n // page) for n in lens)
    pages = used + 3
    order = torch.randperm(pages, device=dev, generator=gen).to(torch.int32).cpu().tolist()  # pages in no order, as a long-running server has them
    table = [[0] * width for _ in range(B)]
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[b][i] = order.pop()
    s.update(kv=kv, page=page, max_len=max(lens), page_table=ints(table), lens=ints(lens), rows=sum(rows), max_rows=max(rows),
             row_start=None if max(rows) == 1 else ints(_starts(rows)))
    for name in ("K", "V"):
        codes = torch.empty((pages, kv, page, dim), dtype=torch.int8, device=dev)
        for at in range(0, pages, 4096):
            part = codes[at:at + 4096]
            part.copy_(torch.randn(part.shape, generator=gen, device=dev, dtype=torch.float16).mul_(36.0).round_().clamp_(-127, 127))
        s[name] = codes
        s[name.lower() + "_scale"] = torch.exp(0.3 * torch.randn((pages, kv), generator=gen, device=dev)) * 0.028
    if kind == "attend":
        s["q"] = torch.randn((s["rows"], heads * dim), generator=gen, device=dev).to(dtype)
        return s
    # q, k and v rows: slices of one buffer
    qkv = torch.randn((s["rows"], (heads + 2 * kv) * dim), generator=gen, device=dev).to(dtype)
    s["q"], s["k"], s["v"] = qkv.split((heads * dim, kv * dim, kv * dim), 1)
    # positions on several axes: the tokens of images stand at rows and columns; one axis: where the row lies in the cache
    s["positions"] = None if case["axes"] == 1 else torch.randint(0, reach, (case["axes"], s["rows"]), generator=gen, device=dev, dtype=torch.int32)
    # what comes back: every page that the call touched
    back = [n - (n - r) // page * page for n, r in zip(lens, rows)]
    s["back_rows"], s["back_max"], s["back_start"] = sum(back), max(back), ints(_starts(back))
    return s


# ---------------------------------------------------------------- plain forms
def _rotate(s, x, heads, positions, norm):
    """Rows x [rows][heads * dim] normed and rotated, in their type."""
    dim, rot = s["dim"], s["rot"]
    y = x.float().reshape(-1, heads, dim)
    if norm is not None:
        r = (1.0 / torch.sqrt((y.double() * y.double()).mean(-1, keepdim=True) + EPS)).float()  # long sums in 64 bits
        y = y * r * norm
    if s["pair_axis"] is None:
        turn = s["table"][positions.reshape(-1).long()]  # [rows][pairs][2]
    else:
        turn = s["table"][positions.long()[s["pair_axis"].long()].T, torch.arange(rot // 2, device=x.device)]
    c, w = turn[:, None, :, 0], turn[:, None, :, 1]
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if s["halves"] else (y[..., 0:rot:2], y[..., 1:rot:2])
    a, b = a * c - b * w, b * c + a * w
    turned = torch.cat((a, b), -1) if s["halves"] else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype).reshape(x.shape)


def _place(s, row_start, rows):
    """(position, page, slot) of each row: the rows are the last positions of their sequences."""
    lens = s["lens"].long()
    at = torch.arange(rows, device=lens.device)
    if row_start is None:
        seq, pos = at, lens - 1
    else:
        seq = torch.bucketize(at, row_start[1:].long(), right=True)
        pos = lens[seq] - (row_start[1:] - row_start[:-1]).long()[seq] + at - row_start.long()[seq]
    return pos, s["page_table"].long()[seq, pos // s["page"]], pos % s["page"]


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


def _append_plain(s):
    pos, page, slot = _place(s, s["row_start"], s["rows"])
    positions = pos[None] if s["positions"] is None else s["positions"]
    q = _rotate(s, s["q"], s["heads"], positions, s["q_norm"])
    k = _rotate(s, s["k"], s["kv"], positions, s["k_norm"])
    touched = _touched(s)
    _append_one(s, s["K"], s["k_scale"], k, page, slot, touched)
    _append_one(s, s["V"], s["v_scale"], s["v"], page, slot, touched)
    _, page, slot = _place(s, s["back_start"], s["back_rows"])
    k, v = ((s[n][page, :, slot].float() * s[n.lower() + "_scale"][page][:, :, None]).to(s["dtype"]).reshape(s["back_rows"], -1) for n in ("K", "V"))
    return {"q": q, "k": k, "v": v}


def _whole(s, name):
    """[B][kv][positions][dim] of a cache in float32, every page of the tables."""
    t = s["page_table"].long()
    x = s[name][t].float() * s[name.lower() + "_scale"][t][..., None, None]
    return x.transpose(1, 2).reshape(t.shape[0], s["kv"], -1, s["dim"])


def _attend_plain(s):
    B, kv, dim, heads = s["lens"].numel(), s["kv"], s["dim"], s["heads"]
    group, N, lens = heads // kv, s["max_rows"], s["lens"].long()
    start = torch.arange(B + 1, device=lens.device) if s["row_start"] is None else s["row_start"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(N, device=lens.device)
    row = (start[:-1, None] + i).clamp(max=s["rows"] - 1)  # [B][N], rows past a sequence's n are dropped below
    q = s["q"].float().reshape(-1, kv, group, dim)[row].permute(0, 2, 1, 3, 4).reshape(B, kv, N * group, dim)
    p = torch.matmul(q, _whole(s, "K").transpose(-1, -2)).reshape(B, kv, N, group, -1)
    p *= 1.0 / math.sqrt(dim)
    sees = torch.arange(p.shape[-1], device=lens.device) < ((lens - n)[:, None] + i + 1)[..., None]  # [B][N][positions]
    sees = (sees & (i < n[:, None])[..., None])[:, None, :, None]
    p.masked_fill_(~sees, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total > 0, total, 1.0)
    out = torch.matmul(p.reshape(B, kv, N * group, -1), _whole(s, "V")).reshape(B, kv, N, group, dim)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, N, heads * dim)
    at = torch.arange(s["rows"], device=lens.device)
    seq = torch.bucketize(at, start[1:], right=True)
    return out[seq, at - start[seq]].to(s["dtype"])


def _run_plain(s):
    if s["kind"] == "table":
        return _table(s["inv_freq"], s["first"], s["positions"], s["scale"])
    if s["kind"] == "rope":
        return _rotate(s, s["x"], s["heads"], s["positions"], s["q_norm"])
    return _append_plain(s) if s["kind"] == "append" else _attend_plain(s)


# ---------------------------------------------------------------- the framework's calls
def _run_own(s):
    import quantized_weight_prefill_q4_gb300 as q

    empty = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if s["kind"] == "table":
        table = empty(s["positions"], s["inv_freq"].numel(), 2, dtype=torch.float32)
        q.apr_rope_table(s["inv_freq"], table, first=s["first"], scale=s["scale"])
        return table
    if s["kind"] == "attend":
        cache, out = q.Kv8Cache(s["K"], s["V"], s["k_scale"], s["v_scale"]), torch.empty_like(s["q"])
        q.apr_kv8_prefill_attention(cache, s["page_table"], s["lens"], s["q"], out, s["heads"], row_start=s["row_start"],
                                    max_rows=s["max_rows"], max_len=s["max_len"])
        return out
    rope = q.Rope(s["table"], interleaved=not s["halves"], pair_axis=s["pair_axis"])
    if s["kind"] == "rope":
        out = empty(*s["x"].shape, dtype=s["dtype"])
        q.apr_rope_rows(rope, s["positions"], s["x"], out, s["heads"], s["dim"], norm=s["q_norm"], eps=EPS)
        return out
    cache, wide = q.Kv8Cache(s["K"], s["V"], s["k_scale"], s["v_scale"]), s["kv"] * s["dim"]
    q_out, k, v = empty(*s["q"].shape, dtype=s["dtype"]), empty(s["back_rows"], wide, dtype=s["dtype"]), empty(s["back_rows"], wide, dtype=s["dtype"])
    q.apr_rope_kv8_append(cache, s["page_table"], s["lens"], rope, s["k"], s["v"], positions=s["positions"], k_norm=s["k_norm"],
                          q=s["q"], q_out=q_out, num_heads=s["heads"], q_norm=s["q_norm"], eps=EPS, row_start=s["row_start"], max_rows=s["max_rows"])
    q.apr_kv8_read(cache, s["page_table"], s["lens"], k, v, row_start=s["back_start"], max_rows=s["back_max"])
    return {"q": q_out, "k": k, "v": v}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    kind = case["kind"]
    if kind == "table":
        return {"bytes": 8 * case["positions"] * case["pairs"], "flops": 20 * case["positions"] * case["pairs"]}
    size, dim, heads = 4 if case["type"] == "f32" else 2, case["dim"], case["heads"]
    if kind == "rope":
        # rows in and out, their positions, and the cosines and sines of each position once
        return {"bytes": case["rows"] * (2 * heads * dim * size + 4 * case["axes"] + 4 * case["rot"]), "flops": case["rows"] * heads * (3 * case["rot"] + (4 * dim if case["norm"] else 0))}
    lens, rows, kv, page = _lens(case), _rows(case), case["kv"], case["page"]
    row = 2 * kv * dim  # codes of one token's k and v
    scales = lambda tokens: 8 * kv * (-(-tokens // page))  # noqa: E731
    if kind == "append":
        back = [n - (n - r) // page * page for n, r in zip(lens, rows)]
        # q in and out, k and v in, their codes out; then the touched pages' codes in and their values out
        return {"bytes": sum(rows) * (2 * heads * dim * size + 4 * case["rot"] + row * (size + 1)) + sum(back) * row * (1 + size) + sum(2 * scales(n) for n in back),
                "flops": sum(rows) * (heads + kv) * (3 * case["rot"] + (4 * dim if case["norm"] else 0)) + 2 * row * (sum(rows) + sum(back))}
    seen = sum(n * r - r * (r - 1) // 2 for n, r in zip(lens, rows))
    return {"bytes": sum(lens) * row + sum(scales(n) for n in lens) + 2 * sum(rows) * heads * dim * size, "flops": 4 * seen * heads * dim}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_rotation(case, s, x, heads, positions, norm):
    """Rows [rows][heads][dim] in float64, rounded where the definition rounds: every step a float64 one whose result is rounded to
    float32 (products and sums of two float32 numbers are exact or nearly so in 64 bits), the result not to the type."""
    f32 = lambda t: t.float().double()  # noqa: E731
    dim, rot = case["dim"], case["rot"]
    y = x.double().reshape(-1, heads, dim)
    if norm is not None:
        r = f32((y.square().sum(-1, keepdim=True) / dim + EPS).rsqrt())
        y = f32(f32(y * r) * norm.double())
    out = y.clone()
    table, half = s["table"].double(), rot // 2
    for i in range(half):
        a = 0 if s["pair_axis"] is None else int(s["pair_axis"][i])
        cos, sin = table[positions[a].long(), i].unbind(-1)
        lo, hi = (i, half + i) if case["layout"] == "halves" else (2 * i, 2 * i + 1)
        u, v = y[..., lo], y[..., hi]
        out[..., lo] = f32(f32(u * cos[:, None]) - f32(v * sin[:, None]))
        out[..., hi] = f32(f32(v * cos[:, None]) + f32(u * sin[:, None]))
    return out


def _pages_of(s, name, b, first, count):
    """Tokens first .. count - 1 of sequence b (first at a page's start) as [tokens][kv][dim] float64 codes, and each token's scale [tokens][kv]."""
    ids = s["page_table"][b, first // s["page"]: -(-count // s["page"])].long()
    codes = s[name].index_select(0, ids).to(torch.float64).permute(0, 2, 1, 3).reshape(-1, s["kv"], s["dim"])[:count - first]
    return codes, s[name.lower() + "_scale"].index_select(0, ids).to(torch.float64).repeat_interleave(s["page"], 0)[:count - first]


def _exact_append(s, name, b, first, held, length, x):
    """The values of sequence b's touched pages, tokens first .. length - 1, after rows x [rows][kv][dim] joined the `held` tokens from `first` on."""
    page, values = s["page"], []
    for at in range(first, length, page):
        here = min(length, at + page) - at
        old = held if at == first else 0
        new = x[max(0, at - first - held):][: here - old]
        need = (new.abs().amax((0, 2)) / 127).float().double()
        codes = new
        if old:
            kept, scale = _pages_of(s, name, b, at, at + old)
            need = torch.maximum(scale[0], need)
            codes = torch.cat([(kept * scale[0][:, None]).float().double(), new])
        codes = torch.round(codes / need[:, None]).nan_to_num(0.0).clamp(-127, 127)
        values.append(codes * need[:, None])
    return torch.cat(values)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "table":
        # points at that angle on a circle of the scale's radius
        at = torch.arange(case["positions"], device="cuda", dtype=torch.float64) + case["first"]
        angle = torch.outer(at, s["inv_freq"].double())
        return torch.view_as_real(torch.polar(torch.full_like(angle, case["scale"]), angle))
    if case["kind"] == "rope":
        return _exact_rotation(case, s, s["x"], case["heads"], s["positions"], s["q_norm"]).reshape(case["rows"], -1)
    lens, rows, page, kv, dim, heads = _lens(case), _rows(case), case["page"], case["kv"], case["dim"], case["heads"]
    at = _starts(rows)
    if case["kind"] == "append":
        positions = s["positions"]
        if positions is None:
            positions = torch.cat([torch.arange(n - r, n, device="cuda") for n, r in zip(lens, rows)])[None]
        q = _exact_rotation(case, s, s["q"], heads, positions, s["q_norm"])
        k = _exact_rotation(case, s, s["k"], kv, positions, s["k_norm"]).to(s["dtype"]).double()
        got = {"k": [], "v": []}
        for b, (n, r) in enumerate(zip(lens, rows)):
            first = (n - r) // page * page
            for name, x in (("K", k), ("V", s["v"].double().reshape(-1, kv, dim))):
                got[name.lower()].append(_exact_append(s, name, b, first, n - r - first, n, x[at[b]:at[b + 1]]).reshape(-1, kv * dim))
        return {"q": q.reshape(sum(rows), -1), "k": torch.cat(got["k"]), "v": torch.cat(got["v"])}
    group, outs = heads // kv, []
    for b, (n, r) in enumerate(zip(lens, rows)):
        (ck, sk), (cv, sv) = _pages_of(s, "K", b, 0, n), _pages_of(s, "V", b, 0, n)
        q = s["q"][at[b]:at[b + 1]].double().reshape(r, kv, group, dim)
        hidden = torch.arange(n, device="cuda") > torch.arange(n - r, n, device="cuda")[:, None]
        out = torch.empty((r, heads, dim), dtype=torch.float64, device="cuda")
        for h in range(heads):
            g = h // group
            scores = (q[:, g, h % group] @ (ck[:, g] * sk[:, g, None]).T) / math.sqrt(dim)
            out[:, h] = torch.softmax(scores.masked_fill_(hidden, -math.inf), -1) @ (cv[:, g] * sv[:, g, None])
        outs.append(out.reshape(r, -1))
    return torch.cat(outs)
