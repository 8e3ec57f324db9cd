"""Workloads of the 4-bit paged cache, sliding-window decode and batch-table operators.

Each case is one pass through an operator as a serving loop calls it.  ``run``
computes it with the framework's kernels when ``own`` is true, and in plain
torch operations otherwise; ``exact`` evaluates the definition in 64 bits.

Operators
---------
``q4_decode``  decode attention over a paged cache held in 4 bits, optionally
               with a sliding window and a few first tokens that stay visible
``window``     decode attention over a bf16 or fp32 paged cache with a sliding
               window and a few first tokens that stay visible
``q4_write``   new tokens quantised into their slots of the 4-bit cache, and
               read back from it
``tables``     block tables, slot maps and positions of a batch from its
               requests' lengths and flat block lists

The 4-bit cache.  A head row of ``head_dim`` values is cut into groups of
``group`` values.  Each group has a minimum m (its smallest value rounded down
to bf16) and a step s (a fifteenth of its largest value's distance from m,
rounded up to bf16), and a value x is held as the code
round((x - m) * (1 / s)), every operation in fp32; it stands for s * code + m.
A page of one (block, KV head) is block_size rows of head_dim / 2 bytes of
codes, then block_size x groups pairs (s, m) of bf16.  Within a row, the units
of four values are stored so that unit 16 w + 8 h + g is half-word h of word
g * (head_dim / 64) + w.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ---

def _decode(name, op, seqs, min_len, max_len, spread, q_heads, kv_heads, head_dim, block, dtype="bf16", group=0,
            window=0, sinks=0, empty=0):
    return dict(name=name, op=op, seqs=seqs, min_len=min_len, max_len=max_len, spread=spread, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, block=block, dtype=dtype, group=group, window=window,
                sinks=sinks, empty=empty)


def listed():
    return [
        # one interactive request: nothing to hide the latency behind
        _decode("q4_single", "q4_decode", 1, 777, 777, "uniform", 32, 8, 128, 16, group=64),
        # the GQA serving batch of the benchmark (lognormal lengths), its cache in 4 bits
        _decode("q4_gqa", "q4_decode", 32, 256, 32768, "lognormal", 64, 8, 128, 16, group=64),
        # a large continuous batch at moderate lengths, with requests that have not started yet
        _decode("q4_batch", "q4_decode", 256, 16, 8192, "uniform", 64, 8, 128, 32, group=64, empty=3),
        # few very long requests: the long axis has to be split
        _decode("q4_long", "q4_decode", 7, 60001, 131072, "uniform", 64, 8, 128, 32, group=32),
        # 4-bit cache with a window and sinks, head_dim 64, plain multi-head attention
        _decode("q4_window", "q4_decode", 96, 1, 30000, "uniform", 24, 24, 64, 16, group=32, window=2000, sinks=5),
        # one request past its window: the smallest windowed call
        _decode("window_single", "window", 1, 20000, 20000, "uniform", 32, 8, 128, 16, window=512, sinks=4),
        # a serving batch with a window of 4096 tokens, some requests still shorter than it
        _decode("window_batch", "window", 64, 100, 32768, "uniform", 64, 8, 128, 16, window=4096, sinks=4, empty=1),
        # fp32, multi-head, a window that is no multiple of a block, sinks that end inside one
        _decode("window_f32", "window", 32, 1, 9000, "uniform", 32, 32, 128, 32, dtype="f32", window=1000, sinks=37),
        # the cache write of one decode step
        dict(name="q4_write_step", op="q4_write", tokens=32, padding=0, kv_heads=8, head_dim=128, block=16, group=64,
             dtype="bf16"),
        # the cache write of a prefill chunk, padded as a captured graph pads it
        dict(name="q4_write_prefill", op="q4_write", tokens=30011, padding=2757, kv_heads=8, head_dim=128, block=32,
             group=32, dtype="bf16"),
        # tables and slots of a decode step: one new token for each request
        dict(name="tables_step", op="tables", seqs=64, min_len=128, max_len=2048, new=1, block=16, padding=0, empty=0),
        # tables and slots of a large mixed batch: chunks of prompts and single tokens
        dict(name="tables_mixed", op="tables", seqs=513, min_len=1, max_len=16384, new=1024, block=16, padding=999,
             empty=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["q4_decode", "q4_decode", "window", "window", "q4_write", "tables"])
    if op == "tables":
        seqs = _log(rng, 1, 600)
        max_len = _log(rng, 1, 16384)
        return dict(op=op, seqs=seqs, min_len=rng.randint(1, max_len), max_len=max_len, new=_log(rng, 1, 1024),
                    block=rng.choice([16, 32]), padding=rng.randint(0, 500), empty=rng.randint(0, seqs // 8))
    head_dim, block, kv_heads = rng.choice([64, 128]), rng.choice([16, 32]), rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "q4_write":
        return dict(op=op, tokens=_log(rng, 1, 30000 * 1024 // max(1024, kv_heads * head_dim)),
                    padding=rng.randint(0, 300), kv_heads=kv_heads, head_dim=head_dim, block=block,
                    group=rng.choice([32, 64]), dtype=dtype)
    group_heads = rng.choice([1, 1, 2, 4, 5, 7, 8, 8, 12, 16])
    if kv_heads * group_heads > 64:
        group_heads = max(1, 64 // kv_heads)
    seqs = _log(rng, 1, 256)
    # the plain form holds every visible token widened: keep that within the largest listed case's
    most = (1 << 20) * 1024 // (seqs * kv_heads * head_dim)
    windowed = op == "window" or rng.random() < 0.3
    if windowed:
        window = _log(rng, 1, max(1, min(5000, most // (2 if dtype == "f32" else 1))))
        sinks = rng.choice([0, 1, 4, 4, rng.randint(0, 100)])
        max_len = _log(rng, 1, 40000)
    else:
        window = sinks = 0
        max_len = _log(rng, 1, max(1, min(131072, most)))
    return dict(op=op, seqs=seqs, min_len=rng.randint(1, max_len), max_len=max_len,
                spread="uniform", q_heads=kv_heads * group_heads, kv_heads=kv_heads, head_dim=head_dim,
                block=block, dtype=dtype, group=rng.choice([32, 64]) if op == "q4_decode" else 0, window=window,
                sinks=sinks, empty=rng.randint(0, seqs // 8))


# ----------------------------------------------------------------- inputs ---

def _lengths(case):
    """The batch's context lengths: part of the case, whatever the seed."""
    rng = np.random.default_rng([case["seqs"], case["min_len"], case["max_len"], case["block"]])
    n = case["seqs"]
    if case.get("spread") == "lognormal":
        lens = np.clip(np.rint(4096.0 * np.exp(rng.standard_normal(n))), case["min_len"], case["max_len"])
    else:
        lens = rng.integers(case["min_len"], case["max_len"], size=n, endpoint=True)
    lens = lens.astype(np.int64)
    lens[0] = case["max_len"]
    if case["empty"]:
        lens[n - case["empty"]:] = 0
    return lens


def _new_lengths(case, lens):
    rng = np.random.default_rng([case["seqs"], case["new"], case["max_len"]])
    if case["new"] == 1:
        return np.minimum(lens, 1)
    chunk = rng.integers(2, case["new"], size=len(lens), endpoint=True)
    return np.minimum(lens, np.where(rng.random(len(lens)) < 0.5, 1, chunk))


def _seen(case, lens):
    """Tokens each sequence attends over."""
    if not case["window"]:
        return lens
    first = np.minimum(lens, case["sinks"])
    return first + (lens - np.maximum(first, lens - case["window"]))


def _page_bytes(case):
    return case["block"] * (case["head_dim"] // 2 + 4 * (case["head_dim"] // case["group"]))


def _values(gen, rows, heads, dim, dtype):
    """Rows of keys or values: unit normals whose channels differ in scale and offset."""
    x = torch.randn(rows, heads, dim, generator=gen, device="cuda")
    spread = torch.rand(1, heads, dim, generator=gen, device="cuda") * 1.5 + 0.25
    shift = torch.randn(1, heads, dim, generator=gen, device="cuda") * 0.5
    return x.mul_(spread).add_(shift).to(dtype)


def _place(case, lens, gen):
    """Block tables over a shuffled pool; blocks behind the window have been given back (-1)."""
    bs, w = case["block"], case["window"]
    width = max(1, -(-int(lens.max()) // bs))
    start = torch.arange(width, device="cuda") * bs
    n = torch.from_numpy(lens).cuda()[:, None]
    used = start[None] < n
    if w:
        used &= (start[None] < case["sinks"]) | (start[None] + bs > n - w)
    blocks = int(sum(_used_pages(case, int(v)) for v in lens))
    num_blocks = math.ceil(1.05 * blocks) + 1
    order = torch.randperm(num_blocks, generator=gen, device="cuda")
    rank = used.flatten().cumsum(0).view_as(used) - 1
    table = torch.where(used, order[rank.clamp(min=0)], -1).to(torch.int32)
    return table, num_blocks


def _used_pages(case, n):
    bs = case["block"]
    pages = -(-n // bs)
    if not case["window"] or n == 0:
        return pages
    behind = max(0, n - case["window"]) // bs
    return pages - max(0, behind - -(-case["sinks"] // bs))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "tables":
        return _prepare_tables(case, gen)
    heads, dim, bs, dtype = case["kv_heads"], case["head_dim"], case["block"], DTYPES[case["dtype"]]
    if case["op"] == "q4_write":
        total = case["tokens"] + case["padding"]
        num_blocks = -(-case["tokens"] // bs) + 3
        # the last block of the pool is nobody's
        slots = torch.randperm((num_blocks - 1) * bs, generator=gen, device="cuda")[:total]
        if len(slots) < total:
            slots = torch.cat([slots, slots.new_full((total - len(slots),), -1)])
        slots[case["tokens"]:] = -1
        pages = (num_blocks, heads, _page_bytes(case))
        return dict(case=case, slots=slots, num_blocks=num_blocks,
                    k=_values(gen, total, heads, dim, dtype), v=_values(gen, total, heads, dim, dtype),
                    k_cache=torch.zeros(pages, dtype=torch.uint8, device="cuda"),
                    v_cache=torch.zeros(pages, dtype=torch.uint8, device="cuda"),
                    k_out=torch.zeros(total, heads, dim, dtype=dtype, device="cuda"),
                    v_out=torch.zeros(total, heads, dim, dtype=dtype, device="cuda"))
    lens = _lengths(case)
    table, num_blocks = _place(case, lens, gen)
    caches = []
    for _ in range(2):
        if case["op"] == "window":
            rows = _values(gen, num_blocks * bs, heads, dim, dtype)
            caches.append(rows.view(num_blocks, bs, heads, dim).transpose(1, 2).contiguous())
        else:
            cache = torch.empty(num_blocks, heads, _page_bytes(case), dtype=torch.uint8, device="cuda")
            step = max(1, (1 << 27) // (heads * dim * bs))
            for b in range(0, num_blocks, step):
                part = cache[b:b + step]
                rows = _values(gen, len(part) * bs, heads, dim, torch.bfloat16).float()
                codes, params = _quantise(rows, case["group"])
                spots = torch.arange(len(part) * bs, device="cuda")
                _store(part, case, spots, codes, params)
            caches.append(cache)
    return dict(case=case, k_cache=caches[0], v_cache=caches[1], block_tables=table,
                q=torch.randn(case["seqs"], case["q_heads"], dim, generator=gen, device="cuda").to(dtype),
                context_lens=torch.from_numpy(lens).to(torch.int32).cuda(), scale=1.0 / math.sqrt(dim),
                max_context_len=int(lens.max()))


def _prepare_tables(case, gen):
    lens = _lengths(case)
    new = _new_lengths(case, lens)
    bs = case["block"]
    blocks = int((-(-lens // bs)).sum())
    num_blocks = math.ceil(1.05 * blocks) + 1
    tokens = int(new.sum()) + case["padding"]
    width = max(1, -(-int(lens.max()) // bs))
    return dict(case=case, num_blocks=num_blocks,
                block_ids=torch.randperm(num_blocks, generator=gen, device="cuda")[:blocks].to(torch.int32),
                context_lens=torch.from_numpy(lens).to(torch.int32).cuda(),
                new_lens=torch.from_numpy(new).to(torch.int32).cuda(),
                block_tables=torch.empty(case["seqs"], width, dtype=torch.int32, device="cuda"),
                slot_mapping=torch.empty(tokens, dtype=torch.int64, device="cuda"),
                positions=torch.empty(tokens, dtype=torch.int32, device="cuda"),
                query_start=torch.empty(case["seqs"] + 1, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------- runs ---

def run(state):
    op = state["case"]["op"]
    if own:
        return {"q4_decode": _own_q4_decode, "window": _own_window, "q4_write": _own_q4_write,
                "tables": _own_tables}[op](state)
    return {"q4_decode": _plain_q4_decode, "window": _plain_window, "q4_write": _plain_q4_write,
            "tables": _plain_tables}[op](state)


def _own_q4_decode(s):
    step = s.get("step")
    if step is None:     # a serving loop builds its step once and keeps it
        from paged_kv_cache_237_gb300.engine import Q4DecodeStep
        c = s["case"]
        step = s["step"] = Q4DecodeStep(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                                        s["scale"], s["max_context_len"], group_size=c["group"], window=c["window"],
                                        num_sinks=c["sinks"])
    return step.decode()


def _own_window(s):
    step = s.get("step")
    if step is None:
        from paged_kv_cache_237_gb300.engine import DecodeStep
        c = s["case"]
        step = s["step"] = DecodeStep(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                                      s["scale"], s["max_context_len"], window=c["window"], num_sinks=c["sinks"])
    return step.decode()


def _own_q4_write(s):
    from paged_kv_cache_237_gb300 import pa_gather_q4, pa_reshape_and_cache_q4
    group = s["case"]["group"]
    pa_reshape_and_cache_q4(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], group_size=group)
    pa_gather_q4(s["k_out"], s["v_out"], s["k_cache"], s["v_cache"], s["slots"], group_size=group)
    return s["k_out"], s["v_out"]


def _own_tables(s):
    from paged_kv_cache_237_gb300 import pa_build_tables
    pa_build_tables(s["block_tables"], s["slot_mapping"], s["positions"], s["query_start"], s["block_ids"],
                    s["context_lens"], s["new_lens"], block_size=s["case"]["block"], num_blocks=s["num_blocks"])
    return s["block_tables"], s["slot_mapping"], s["positions"], s["query_start"]


# ------------------------------------------------------------ plain forms ---

def _quantise(x, group):
    """Codes (uint8, one per value) and the (step, minimum) pairs in bf16 of fp32 rows [T, H, D].

    The divisor 15 is a tensor because torch divides by a plain number as a product with its reciprocal."""
    x = x.unflatten(-1, (-1, group))
    low, high = x.amin(-1), x.amax(-1)
    bad = ~(x.abs().amax(-1) < 2.0 ** 126)
    bits = low.view(torch.int32)
    m = ((bits & -65536) + 65536 * ((bits < 0) & ((bits & 65535) != 0)).int()).view(torch.float32)
    far = high - m
    s = (((far / torch.full_like(far, 15)).view(torch.int32) + 65535) & -65536).view(torch.float32)
    s = torch.where(far > 0, s.clamp(min=2.0 ** -126), 0.0)
    codes = ((x - m[..., None]) * torch.where(s > 0, 1 / s, 0.0)[..., None]).round()
    codes = torch.where(bad[..., None], 0.0, codes).to(torch.uint8).flatten(-2)
    params = torch.stack([torch.where(bad, 0.0, s), torch.where(bad, float("nan"), m)], -1).to(torch.bfloat16)
    return codes, params


def _parts(cache, case):
    """The codes [blocks, H, bs, D / 2] and (s, m) pairs [blocks, H, bs, groups, 2] of a cache, as views."""
    bs, dim = case["block"], case["head_dim"]
    cut = bs * dim // 2
    return (cache[..., :cut].unflatten(-1, (bs, dim // 2)),
            cache[..., cut:].view(torch.bfloat16).unflatten(-1, (bs, dim // case["group"], 2)))


def _store(cache, case, slots, codes, params):
    c = codes.unflatten(-1, (-1, 2, 8, 4)).movedim(-2, -4).flatten(-4).unflatten(-1, (-1, 2))
    held, pairs = _parts(cache, case)
    at, row = slots // case["block"], slots % case["block"]
    held[at, :, row] = c[..., 0] | (c[..., 1] << 4)
    pairs[at, :, row] = params


def _load(cache, case, at, row):
    """fp32 values [..., H, D] of the tokens in rows `row` of blocks `at`."""
    held, pairs = _parts(cache, case)
    b = held[at, :, row]
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2).unflatten(-1, (8, -1, 2, 4)).movedim(-4, -2).flatten(-4)
    p = pairs[at, :, row].float()
    return (c.unflatten(-1, (-1, case["group"])) * p[..., :1] + p[..., 1:]).flatten(-2)


def _attend(q, k, v, ok, scale):
    """softmax(scale q K^T) V in fp32: q [S, Hq, D], k, v [S, N, Hkv, D], ok [S, N]; an empty row gives zeros."""
    seqs, heads = q.shape[0], k.shape[2]
    qg = q.float().view(seqs, heads, -1, q.shape[-1])
    logits = torch.einsum("shgd,snhd->shgn", qg, k) * scale
    logits = logits.masked_fill(~ok[:, None, None], float("-inf"))
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top.isinf(), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("shgn,snhd->shgd", p, v * ok[..., None, None])
    return torch.where(total > 0, o / total, 0.0).flatten(1, 2).to(q.dtype)


def _visible(s):
    """Positions each sequence attends over [S, N], which of them are real, their blocks and rows."""
    case, n = s["case"], s["context_lens"].long()[:, None]
    if case["window"]:
        first = torch.arange(min(case["sinks"], s["max_context_len"]), device="cuda")
        last = n - torch.arange(min(case["window"], s["max_context_len"]), 0, -1, device="cuda")
        pos = torch.cat([first.expand(len(n), -1), last], 1)
        fresh = torch.arange(pos.shape[1], device="cuda") < len(first)
        ok = (pos < n) & (pos >= 0) & (fresh | (pos >= case["sinks"]))
    else:
        pos = torch.arange(s["max_context_len"], device="cuda").expand(len(n), -1)
        ok = pos < n
    pos = torch.where(ok, pos, 0)
    at = s["block_tables"].gather(1, pos // case["block"]).clamp(min=0).long()
    return ok, at, pos % case["block"]


def _plain_q4_decode(s):
    ok, at, row = _visible(s)
    return _attend(s["q"], _load(s["k_cache"], s["case"], at, row), _load(s["v_cache"], s["case"], at, row), ok,
                   s["scale"])


def _plain_window(s):
    ok, at, row = _visible(s)
    return _attend(s["q"], s["k_cache"][at, :, row].float(), s["v_cache"][at, :, row].float(), ok, s["scale"])


def _plain_q4_write(s):
    case, slots = s["case"], s["slots"]
    spots = torch.where(slots < 0, s["num_blocks"] * case["block"] - 1, slots)   # a row of the block that is nobody's
    out = []
    for x, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        codes, params = _quantise(x.float(), case["group"])
        _store(cache, case, spots, codes, params)
        y = _load(cache, case, spots // case["block"], spots % case["block"])
        out.append(torch.where((slots >= 0)[:, None, None], y, 0.0).to(x.dtype))
    return tuple(out)


def _plain_tables(s):
    bs, n, new, ids = s["case"]["block"], s["context_lens"].long(), s["new_lens"].long(), s["block_ids"]
    blocks = (n + bs - 1) // bs
    first = blocks.cumsum(0) - blocks
    query_start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    col = torch.arange(s["block_tables"].shape[1], device="cuda")
    tables = torch.where(col < blocks[:, None], ids[(first[:, None] + col).clamp(max=len(ids) - 1)], -1)
    t = torch.arange(len(s["slot_mapping"]), device="cuda")
    seq = torch.searchsorted(query_start[1:], t, right=True).clamp(max=len(n) - 1)
    pos = n[seq] - new[seq] + t - query_start[seq]
    real = t < query_start[-1]
    pos = torch.where(real, pos, 0)
    slot = ids[(first[seq] + pos // bs).clamp(max=len(ids) - 1)].long() * bs + pos % bs
    return tables.to(torch.int32), torch.where(real, slot, -1), pos.to(torch.int32), query_start.to(torch.int32)


# ------------------------------------------------------------------- work ---

def work(case):
    if case["op"] == "tables":
        lens = _lengths(case)
        new = int(_new_lengths(case, lens).sum())
        blocks = int((-(-lens // case["block"])).sum())
        width = max(1, -(-int(lens.max()) // case["block"]))
        tokens = new + case["padding"]
        read = 4 * blocks + 8 * case["seqs"]
        return {"bytes": read + 4 * case["seqs"] * width + 12 * tokens + 4 * (case["seqs"] + 1),
                "flops": 4 * tokens + 2 * case["seqs"]}
    e = DTYPES[case["dtype"]].itemsize
    row = case["head_dim"] * e
    if case["group"]:
        held = case["head_dim"] // 2 + 4 * (case["head_dim"] // case["group"])
    if case["op"] == "q4_write":
        rows = 2 * case["tokens"] * case["kv_heads"]
        # values in, codes out, codes in, values out; slots for both calls
        return {"bytes": rows * 2 * (row + held) + 16 * (case["tokens"] + case["padding"]),
                "flops": rows * case["head_dim"] * 8}
    lens = _lengths(case)
    seen = int(_seen(case, lens).sum())
    pages = sum(_used_pages(case, int(n)) for n in lens)
    cache = 2 * seen * case["kv_heads"] * (held if case["group"] else row)
    return {"bytes": cache + 2 * case["seqs"] * case["q_heads"] * row + 4 * pages + 4 * case["seqs"],
            "flops": 4 * seen * case["q_heads"] * case["head_dim"]}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "q4_write":
        return tuple(_exact_roundtrip(s[x], s["slots"], case) for x in "kv")
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    bs, per = case["block"], case["q_heads"] // case["kv_heads"]
    for i, n in enumerate(_lengths(case).tolist()):
        if not n:
            continue
        behind = max(0, n - case["window"]) if case["window"] else 0
        pages = [p for p in range(-(-n // bs)) if p * bs < case["sinks"] or p * bs + bs > behind]
        ids = s["block_tables"][i].long()[torch.tensor(pages, device="cuda")]
        pos = (torch.tensor(pages, device="cuda")[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
        keep = (pos < n) & ((pos >= behind) | (pos < case["sinks"]))
        for h in range(case["kv_heads"]):
            k = _exact_rows(s["k_cache"][ids, h], case)[keep]
            v = _exact_rows(s["v_cache"][ids, h], case)[keep]
            q = s["q"][i, h * per:(h + 1) * per].double()
            out[i, h * per:(h + 1) * per] = torch.softmax(q @ k.T * s["scale"], -1) @ v
    return out


def _exact_rows(pages, case):
    """The fp64 rows that the pages [P, ...] of one head hold, in order."""
    bs, dim = case["block"], case["head_dim"]
    if not case["group"]:
        return pages.reshape(-1, dim).double()
    pages = pages.contiguous()
    words = pages[:, :bs * dim // 2].contiguous().view(torch.int16).view(-1, dim // 4).int() & 65535
    pairs = pages[:, bs * dim // 2:].contiguous().view(torch.bfloat16).view(-1, dim // case["group"], 2).double()
    unit = torch.arange(dim, device=pages.device) // 4
    spot = ((unit % 8) * (dim // 64) + unit // 16) * 2 + unit // 8 % 2
    code = (words[:, spot] >> (torch.arange(dim, device=pages.device) % 4 * 4)) & 15
    of = torch.arange(dim, device=pages.device) // case["group"]
    return pairs[:, of, 0] * code.double() + pairs[:, of, 1]


def _exact_roundtrip(x, slots, case):
    """What rows come back as: each fp32 operation of the format's definition, taken in 64 bits and rounded."""
    def f32(y):
        return y.float().double()

    def bf16(y, up):
        near = y.bfloat16().double()
        lower = near > y if not up else near < y
        step = torch.nextafter(near.bfloat16(), torch.full_like(y, math.inf if up else -math.inf).bfloat16())
        return torch.where(lower, step.double(), near)

    x = x.double().view(*x.shape[:-1], -1, case["group"])
    m = bf16(x.min(-1).values, False)
    far = f32(x.max(-1).values - m)
    s = torch.where(far > 0, bf16(f32(far / torch.full_like(far, 15)), True).clamp(min=2.0 ** -126), 0.0)
    back = torch.where(s > 0, f32(1 / s), 0.0)
    codes = torch.round(f32(f32(x - m[..., None]) * back[..., None]))
    y = (codes * s[..., None] + m[..., None]).flatten(-2)
    return torch.where((slots >= 0)[:, None, None], y, 0.0)
