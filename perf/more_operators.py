"""Workloads of the operators in which a sequence has several queries over a paged cache.

Each case is one pass through an operator as a serving loop calls it.  ``run``
computes it with the framework's kernels when ``own`` is true, and in plain
torch operations otherwise; ``exact`` evaluates the definition in 64 bits.

Operators
---------
``tree``    attention of a tree of drafted tokens (or a chain of them) over the
            paged cache that holds the context and the drafted tokens' own rows
``cross``   attention of any number of queries per request over an encoder's
            states in a paged cache, of another length than the queries
``plan``    ancestor bits and positions of a batch of trees from their parents
``commit``  the end of a drafted step: its rows written to the cache, the path
            that the target model agrees with, and the move of that path's rows
            to the positions where the sequence goes on

Queries of all sequences lie end to end: sequence i has rows query_start[i] to
query_start[i + 1] - 1.  A sequence of n tokens whose last c are drafted holds
drafted token r at position n - c + r.  The token r sees every position below
n - c, and of the drafted ones those whose bit is set in its row of the tree's
mask (itself and its ancestors); without a mask it sees the drafted tokens up
to itself.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ---

def _attention(name, op, seqs, len_range, new_range, q_heads, kv_heads, head_dim, block, dtype="bf16",
               spread="uniform", chain=False, empty=0):
    """len_range: tokens before the drafted ones (tree), or encoder states (cross); new_range: queries."""
    return dict(name=name, op=op, seqs=seqs, min_len=len_range[0], max_len=len_range[1], min_new=new_range[0],
                max_new=new_range[1], q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, block=block, dtype=dtype,
                spread=spread, chain=chain, empty=empty)


def listed():
    return [
        # one interactive request that verifies a chain of five drafted tokens: nothing hides the latency
        _attention("tree_single", "tree", 1, (777, 777), (5, 5), 32, 8, 128, 16, chain=True),
        # the GQA serving batch of the benchmark (lognormal lengths), each request with a tree of its own size
        _attention("tree_gqa", "tree", 32, (256, 32768), (16, 64), 64, 8, 128, 16, spread="lognormal"),
        # few very long requests: the long axis has to be split
        _attention("tree_long", "tree", 7, (60001, 131072), (25, 25), 64, 8, 128, 32),
        # fp32, multi-head, small trees, requests that have not started
        _attention("tree_f32", "tree", 24, (1, 4000), (1, 12), 32, 32, 128, 32, dtype="f32", empty=2),
        # one step of a speech-like encoder-decoder: four beams a request share 1500 states
        _attention("cross_step", "cross", 16, (1500, 1500), (4, 4), 16, 16, 64, 16),
        # the decoders' prompts of a mixed batch, some of one token, over inputs of any length
        _attention("cross_prompt", "cross", 64, (1, 1500), (1, 448), 20, 20, 64, 16, empty=1),
        # long outputs over long documents: the products bound it
        _attention("cross_long", "cross", 8, (4000, 16384), (1900, 2048), 64, 8, 128, 32),
        # fp32, decoders' prompts
        _attention("cross_f32", "cross", 16, (100, 1200), (1, 300), 24, 24, 64, 16, dtype="f32"),
        # masks and positions of a small batch's trees
        dict(name="plan_step", op="plan", seqs=8, min_len=1, max_len=4096, min_new=5, max_new=32, empty=0),
        # the same of a large batch with deep trees
        dict(name="plan_batch", op="plan", seqs=500, min_len=0, max_len=16384, min_new=1, max_new=250, empty=9),
        # the end of a step of one small batch
        dict(name="commit_step", op="commit", seqs=4, min_len=1, max_len=500, min_new=8, max_new=24, most=8,
             kv_heads=8, head_dim=128, block=16, dtype="bf16", empty=0),
        # the same of a large batch, with requests that drafted nothing
        dict(name="commit_batch", op="commit", seqs=250, min_len=0, max_len=700, min_new=1, max_new=64, most=12,
             kv_heads=8, head_dim=128, block=32, dtype="bf16", empty=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "cross", "cross", "plan", "commit"])
    if op == "plan":
        seqs, most = _log(rng, 1, 500), _log(rng, 1, 250)
        return dict(op=op, seqs=seqs, min_len=0, max_len=_log(rng, 1, 16384), min_new=rng.randint(1, most),
                    max_new=most, empty=rng.randint(0, seqs // 8))
    kv_heads, head_dim, block = rng.choice([1, 2, 3, 4, 8, 8, 16, 32]), rng.choice([64, 128]), rng.choice([16, 32])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "commit":
        # the pool, and the rows that move, stay within the largest listed case's
        seqs = _log(rng, 1, max(1, min(250, 250 * 8 * 128 // (kv_heads * head_dim * DTYPES[dtype].itemsize // 2))))
        most = _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, min_len=0, max_len=_log(rng, 1, 700), min_new=rng.randint(1, most), max_new=most,
                    most=rng.randint(1, 16), kv_heads=kv_heads, head_dim=head_dim, block=block, dtype=dtype,
                    empty=rng.randint(0, seqs // 8))
    group = rng.choice([1, 1, 2, 4, 5, 7, 8, 8, 12, 16])
    if kv_heads * group > 64:
        group = max(1, 64 // kv_heads)
    seqs = _log(rng, 1, 200)
    chain = op == "tree" and rng.random() < 0.4
    max_new = _log(rng, 1, 2000 if op == "cross" else 500 if chain else 130)
    # bytes of the cache and products: no more than the largest listed cases of the type have
    size = 2 * kv_heads * head_dim * DTYPES[dtype].itemsize
    room = min(2_500_000_000 // size, (4_000_000_000_000 if dtype == "bf16" else 30_000_000_000) //
               (4 * kv_heads * group * head_dim * max_new)) // seqs
    max_len = _log(rng, 1, max(1, min(131072, room)))
    return dict(op=op, seqs=seqs, min_len=rng.randint(0 if op == "tree" else 1, max_len), max_len=max_len,
                min_new=rng.randint(1, max_new), max_new=max_new, q_heads=kv_heads * group, kv_heads=kv_heads,
                head_dim=head_dim, block=block, dtype=dtype, spread="uniform", chain=chain,
                empty=rng.randint(0, seqs // 8))


# ----------------------------------------------------------------- inputs ---

def _sizes(case):
    """Context lengths n and query counts c of the batch: part of the case, whatever the seed."""
    rng = np.random.default_rng([case["seqs"], case["min_len"], case["max_len"], case["max_new"]])
    seqs = case["seqs"]
    if case.get("spread") == "lognormal":
        lens = np.clip(np.rint(4096.0 * np.exp(rng.standard_normal(seqs))), case["min_len"], case["max_len"])
    else:
        lens = rng.integers(case["min_len"], case["max_len"], size=seqs, endpoint=True)
    lens = lens.astype(np.int64)
    new = rng.integers(case["min_new"], case["max_new"], size=seqs, endpoint=True)
    lens[0], new[0] = case["max_len"], case["max_new"]
    if case["op"] == "cross":
        if case["empty"]:       # requests without an encoder input, or without a query in this step
            lens[seqs - case["empty"]:] = 0
            new[seqs - case["empty"]:seqs:2] = 0
        return lens, new
    lens += new
    if case["empty"]:           # requests that have not started, or that draft nothing in this step
        lens[seqs - case["empty"]:seqs:2] = 0
        new[seqs - case["empty"]:] = 0
    return lens, new


def _parents(case, new):
    """Parent of every drafted token within its sequence's tree, -1 for the first: part of the case."""
    if case.get("chain"):
        return np.concatenate([np.arange(-1, c - 1) for c in new] + [np.zeros(0, np.int64)]).astype(np.int64)
    rng = np.random.default_rng([case["seqs"], case["max_new"], 7])
    out = []
    for c in new.tolist():
        r = np.arange(c)
        # a child of one of the few tokens before it, or of any
        near = np.maximum(r - 1 - rng.integers(0, 4, size=c), 0)
        far = np.floor(rng.random(c) * r).astype(np.int64)
        p = np.where(rng.random(c) < 0.6, near, far)
        p[:1] = -1
        out.append(p)
    return np.concatenate(out + [np.zeros(0, np.int64)]).astype(np.int64)


def _mask_rows(new, parents, words):
    """Every drafted token's ancestors and itself, as words of 64 bits."""
    rows, at = [], 0
    for c in new.tolist():
        first = len(rows)
        for r in range(c):
            p = int(parents[at + r])
            rows.append((rows[first + p] if p >= 0 else 0) | 1 << r)
        at += c
    return rows, np.array([[(x >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for x in rows],
                          dtype=np.uint64).reshape(-1, words).view(np.int64)


def _words(case):
    return -(-case["max_new"] // 64)


def _place(lens, block, gen):
    """Block tables over a shuffled pool."""
    per = -(-lens // block)
    width = max(1, int(per.max()))
    num_blocks = math.ceil(1.05 * int(per.sum())) + 1
    order = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    first = torch.from_numpy(per.cumsum() - per).cuda()
    col = torch.arange(width, device="cuda")
    used = col < torch.from_numpy(per).cuda()[:, None]
    return torch.where(used, order[(first[:, None] + col).clamp(max=num_blocks - 1)], -1), num_blocks


def _starts(new):
    return np.concatenate([[0], new.cumsum()]).astype(np.int64)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).cuda()


def _rows(gen, shape, dtype):
    """Rows of keys or values: normals whose channels differ in scale and offset."""
    x = torch.randn(shape, generator=gen, device="cuda")
    spread = torch.rand(shape[-1], generator=gen, device="cuda") * 1.2 + 0.4
    return x.mul_(spread).add_(torch.randn(shape[-1], generator=gen, device="cuda") * 0.3).to(dtype)


def _cache(gen, num_blocks, heads, block, dim, dtype):
    cache = torch.empty(num_blocks, heads, block, dim, dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // (heads * block * dim))
    for b in range(0, num_blocks, step):
        cache[b:b + step] = _rows(gen, cache[b:b + step].shape, dtype)
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, new = _sizes(case)
    starts, tokens = _starts(new), int(new.sum())
    state = dict(case=case, lens=lens.tolist(), new=new.tolist(), starts=starts.tolist(), context_lens=_i32(lens),
                 query_start=_i32(starts))
    if case["op"] == "plan":
        # trees and lengths differ from step to step: the seed shifts where a token's parent lies, and the lengths
        parents, rng = _parents(case, new), np.random.default_rng(seed)
        parents = np.where(parents > 0, parents - rng.integers(0, 2, size=tokens), parents)
        return dict(state, parents=_i32(parents), context_lens=_i32(lens + rng.integers(0, 4096, size=len(lens))),
                    tree_mask=torch.empty(tokens, _words(case), dtype=torch.int64, device="cuda"),
                    positions=torch.empty(tokens, dtype=torch.int32, device="cuda"))
    heads, dim, bs, dtype = case["kv_heads"], case["head_dim"], case["block"], DTYPES[case["dtype"]]
    table, num_blocks = _place(lens, bs, gen)
    state.update(block_tables=table, num_blocks=num_blocks, k_cache=_cache(gen, num_blocks, heads, bs, dim, dtype),
                 v_cache=_cache(gen, num_blocks, heads, bs, dim, dtype))
    if case["op"] == "commit":
        return _prepare_commit(case, seed, state, gen, lens, new, tokens)
    mask = None
    if case["op"] == "tree" and not case["chain"]:
        mask = torch.from_numpy(_mask_rows(new, _parents(case, new), _words(case))[1]).cuda()
    return dict(state, q=torch.randn(tokens, case["q_heads"], dim, generator=gen, device="cuda").to(dtype),
                tree_mask=mask, scale=1.0 / math.sqrt(dim), max_context_len=max(1, int(lens.max())))


def _prepare_commit(case, seed, state, gen, lens, new, tokens):
    rng = np.random.default_rng(seed)
    parents, starts = _parents(case, new), _starts(new)
    draft = rng.integers(0, 32000, size=tokens)
    target = rng.integers(0, 32000, size=tokens)
    # the target model agrees with one of a token's drafted continuations more often than not
    for i, c in enumerate(new.tolist()):
        for r in rng.permutation(c).tolist():
            p = int(parents[starts[i] + r])
            if p >= 0 and rng.random() < 0.75:
                target[starts[i] + p] = draft[starts[i] + r]
    seqs, most = case["seqs"], case["most"]
    seq = np.repeat(np.arange(seqs), new)
    pos = torch.from_numpy(np.arange(tokens) - starts[seq] + (lens - new)[seq]).cuda()
    block = state["block_tables"][torch.from_numpy(seq).cuda(), pos // case["block"]].long()
    shape = (tokens, case["kv_heads"], case["head_dim"])
    empty = dict(dtype=torch.int32, device="cuda")
    return dict(state, parents=_i32(parents), draft_tokens=_i32(draft), target_tokens=_i32(target),
                k_new=_rows(gen, shape, DTYPES[case["dtype"]]), v_new=_rows(gen, shape, DTYPES[case["dtype"]]),
                slots=block * case["block"] + pos % case["block"], accepted_lens=torch.empty(seqs, **empty),
                accepted_nodes=torch.empty(seqs, most, **empty), next_tokens=torch.empty(seqs, **empty),
                new_lens=torch.empty(seqs, **empty),
                slot_pairs=torch.empty(seqs, most, 2, dtype=torch.int64, device="cuda"))


# ------------------------------------------------------------------- runs ---

def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "cross": _own_cross, "plan": _own_plan, "commit": _own_commit}[op](state)
    return {"tree": _plain_attention, "cross": _plain_attention, "plan": _plain_plan,
            "commit": _plain_commit}[op](state)


def _own_tree(s):
    step = s.get("step")
    if step is None:     # a serving loop builds its step once and keeps it
        from paged_kv_cache_237_gb300.engine import TreeDecodeStep
        step = s["step"] = TreeDecodeStep(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                                          s["query_start"], s["scale"], s["max_context_len"],
                                          tree_mask=s["tree_mask"])
    return step.decode()


def _own_cross(s):
    step = s.get("step")
    if step is None:
        from paged_kv_cache_237_gb300.engine import CrossDecodeStep
        step = s["step"] = CrossDecodeStep(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                                           s["query_start"], s["scale"], s["max_context_len"])
    return step.decode()


def _own_plan(s):
    from paged_kv_cache_237_gb300 import pa_build_tree
    pa_build_tree(s["tree_mask"], s["positions"], s["parents"], s["query_start"], s["context_lens"])
    return s["tree_mask"], s["positions"]


def _own_commit(s):
    from paged_kv_cache_237_gb300 import pa_accept_tree, pa_move_rows, pa_reshape_and_cache
    case = s["case"]
    pa_reshape_and_cache(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["slots"])
    pa_accept_tree(s["accepted_lens"], s["accepted_nodes"], s["next_tokens"], s["new_lens"], s["slot_pairs"],
                   s["draft_tokens"], s["target_tokens"], s["parents"], s["query_start"], s["context_lens"],
                   s["block_tables"], block_size=case["block"], num_blocks=s["num_blocks"])
    pa_move_rows(s["k_cache"], s["v_cache"], s["slot_pairs"])
    return (s["accepted_lens"], s["accepted_nodes"], s["next_tokens"], s["new_lens"], s["slot_pairs"], s["k_cache"],
            s["v_cache"])


# ------------------------------------------------------------ plain forms ---

def _visible(s, i, c, n):
    """Which of its n positions each of sequence i's c queries sees, [c, n], or None for all of them."""
    case = s["case"]
    if case["op"] == "cross":
        return None
    pos, row = torch.arange(n, device="cuda") - (n - c), torch.arange(c, device="cuda")
    if case["chain"]:
        return pos <= row[:, None]
    words = s["tree_mask"][s["starts"][i]:s["starts"][i] + c]
    at = pos.clamp(min=0)
    return ((words[:, at // 64] >> (at % 64)) & 1).bool() | (pos < 0)


def _plain_attention(s):
    """softmax(scale q K^T) V in fp32, sequence by sequence; a row that sees nothing gives zeros."""
    case, q = s["case"], s["q"]
    out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    for i, (n, c) in enumerate(zip(s["lens"], s["new"])):
        if not n or not c:
            continue
        rows = slice(s["starts"][i], s["starts"][i] + c)
        pages = s["block_tables"][i, :-(-n // case["block"])].long()
        k, v = (cache[pages].transpose(1, 2).flatten(0, 1)[:n].float() for cache in (s["k_cache"], s["v_cache"]))
        qg = q[rows].float().unflatten(1, (case["kv_heads"], -1))
        logits = torch.einsum("chgd,nhd->hgcn", qg, k) * s["scale"]
        seen = _visible(s, i, c, n)
        if seen is not None:
            logits = logits.masked_fill(~seen, float("-inf"))
        top = logits.amax(-1, keepdim=True)
        p = torch.exp(logits - torch.where(top.isinf(), 0.0, top))
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
        out[rows] = torch.einsum("hgcn,nhd->chgd", p, v).flatten(1, 2)
    return out.to(q.dtype)


def _sequence_of(s, tokens):
    """Sequence of each of the batch's rows, and the row's index within it."""
    row = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(s["query_start"][1:].long(), row, right=True)
    return seq, row - s["query_start"].long()[seq]


def _plain_plan(s):
    tokens = len(s["parents"])
    seq, node = _sequence_of(s, tokens)
    start, parents = s["query_start"].long()[seq], s["parents"].long()
    mask = torch.zeros_like(s["tree_mask"])
    depth = torch.zeros_like(node)
    at = node
    for _ in range(s["case"]["max_new"]):
        live = at >= 0
        bit = torch.where(live, 1 << (at.clamp(min=0) % 64), 0)
        mask.scatter_add_(1, (at.clamp(min=0) // 64)[:, None], bit[:, None])
        at = torch.where(live, parents[start + at.clamp(min=0)], -1)
        depth += at >= 0
    base = (s["context_lens"].long() - s["query_start"].long().diff())[seq]
    return mask, (base + depth).to(torch.int32)


def _plain_commit(s):
    case = s["case"]
    seqs, most, bs = case["seqs"], case["most"], case["block"]
    at, row = s["slots"] // bs, s["slots"] % bs
    for cache, rows in ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"])):
        cache[at, :, row] = rows
    tokens = len(s["parents"])
    seq, node = _sequence_of(s, tokens)
    start, new = s["query_start"].long()[:-1], s["query_start"].long().diff()
    parents, draft, target = s["parents"].long(), s["draft_tokens"].long(), s["target_tokens"].long()
    # first child whose drafted token is the target model's choice at its parent
    up = start[seq] + parents.clamp(min=0)
    agrees = (parents >= 0) & (draft == target[up])
    child = torch.full((tokens + 1,), tokens, device="cuda")
    child.scatter_reduce_(0, torch.where(agrees, up, tokens), torch.where(agrees, node, tokens), "amin")
    nodes = torch.full((seqs, most), -1, device="cuda")
    cur = torch.where(new > 0, 0, -1)
    last = cur
    for j in range(most):
        nodes[:, j] = cur
        last = torch.where(cur >= 0, cur, last)
        found = child[torch.where(cur >= 0, start + cur, tokens)]
        cur = torch.where((cur >= 0) & (found < tokens), found, -1)
    taken = (nodes >= 0).sum(1)
    following = torch.where(new > 0, target[(start + last).clamp(min=0, max=tokens - 1)], -1)
    base = s["context_lens"].long() - new

    def slot(pos):
        block = s["block_tables"].long().gather(1, (pos // bs).clamp(max=s["block_tables"].shape[1] - 1))
        return block * bs + pos % bs

    goal = torch.arange(most, device="cuda").expand(seqs, -1)
    moves = nodes > goal
    pairs = torch.stack([slot(base[:, None] + nodes.clamp(min=0)), slot(base[:, None] + goal)], -1)
    pairs = torch.where(moves[..., None], pairs, -1)
    src, dst = pairs[moves].unbind(-1)
    for cache in (s["k_cache"], s["v_cache"]):
        cache[dst // bs, :, dst % bs] = cache[src // bs, :, src % bs]
    return (taken.to(torch.int32), nodes.to(torch.int32), following.to(torch.int32), (base + taken).to(torch.int32),
            pairs, s["k_cache"], s["v_cache"])


# ------------------------------------------------------------------- work ---

def work(case):
    lens, new = _sizes(case)
    tokens, seqs = int(new.sum()), case["seqs"]
    if case["op"] == "plan":
        return {"bytes": tokens * (4 + 4 + 8 * _words(case)) + 4 * (2 * seqs + 1), "flops": 2 * tokens}
    row = case["head_dim"] * DTYPES[case["dtype"]].itemsize
    if case["op"] == "commit":
        # rows in and out once, the accepted path's read and written once more (half of its longest), the batch's lists
        moved = int(np.minimum(new, case["most"]).sum()) // 2
        lists = 12 * tokens + seqs * (4 * 4 + 20 * case["most"])
        return {"bytes": 2 * (2 * tokens + 2 * moved) * case["kv_heads"] * row + 8 * tokens + lists,
                "flops": 2 * tokens}
    live = np.where(new > 0, lens, 0)
    pages = int((-(-live // case["block"])).sum())
    pairs = int((new * (live - (0 if case["op"] == "cross" else new))).sum())
    if case["op"] == "tree":
        if case["chain"]:
            pairs += int((new * (new + 1) // 2).sum())
        else:
            pairs += sum(bin(x).count("1") for x in _mask_rows(new, _parents(case, new), 1)[0])
    masks = 8 * tokens * _words(case) if case["op"] == "tree" and not case["chain"] else 0
    return {"bytes": 2 * int(live.sum()) * case["kv_heads"] * row + 2 * tokens * case["q_heads"] * row + masks +
            4 * pages + 4 * (2 * seqs + 1), "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "commit":
        return _exact_commit(s)
    lens, new = _sizes(case)
    per, bs = case["q_heads"] // case["kv_heads"], case["block"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    parents, at = _parents(case, new), 0
    for i, (n, c) in enumerate(zip(lens.tolist(), new.tolist())):
        hidden = None
        if case["op"] == "tree" and c:
            sees = np.zeros((c, c), bool)
            for r in range(c):
                p = int(parents[at + r])
                if p >= 0:
                    sees[r] = sees[p]
                sees[r, r] = True
            hidden = torch.ones(c, n, dtype=torch.bool, device="cuda")
            hidden[:, :n - c] = False
            hidden[:, n - c:] = ~torch.from_numpy(sees).cuda()
        if n and c:
            token = torch.arange(n, device="cuda")
            where = s["block_tables"][i].long()[token // bs]
            for h in range(case["kv_heads"]):
                k = s["k_cache"][where, h, token % bs].double()
                v = s["v_cache"][where, h, token % bs].double()
                q = s["q"][at:at + c, h * per:(h + 1) * per].double()
                score = (q @ k.T) * s["scale"]
                if hidden is not None:
                    score.masked_fill_(hidden[:, None], -math.inf)
                out[at:at + c, h * per:(h + 1) * per] = torch.softmax(score, -1) @ v
        at += c
    return out


def _exact_commit(s):
    """Acceptance and moves, one sequence and one token after another."""
    case, bs = s["case"], s["case"]["block"]
    parents, draft, target, tables = (s[x].tolist() for x in ("parents", "draft_tokens", "target_tokens",
                                                              "block_tables"))
    k, v = s["k_cache"].double(), s["v_cache"].double()
    taken, paths, following, lens, pairs = [], [], [], [], []
    for i, (n, c, start) in enumerate(zip(s["lens"], s["new"], s["starts"])):
        slots = [tables[i][p // bs] * bs + p % bs for p in range(n - c, n)]
        path = [0] if c else []
        while path and len(path) < case["most"]:
            found = [r for r in range(c)
                     if parents[start + r] == path[-1] and draft[start + r] == target[start + path[-1]]]
            if not found:
                break
            path.append(found[0])
        for cache, rows in ((k, s["k_new"]), (v, s["v_new"])):
            where = torch.tensor(slots, dtype=torch.int64, device="cuda")
            cache[where // bs, :, where % bs] = rows[start:start + c].double()
            to = where[:len(path)]
            cache[to // bs, :, to % bs] = rows[[start + r for r in path]].double()
        rest = case["most"] - len(path)
        taken.append(len(path))
        paths.append(path + [-1] * rest)
        following.append(target[start + path[-1]] if path else -1)
        lens.append(n - c + len(path))
        pairs.append([[slots[r], slots[j]] if r != j else [-1, -1] for j, r in enumerate(path)] + [[-1, -1]] * rest)
    return (*(torch.tensor(x, device="cuda") for x in (taken, paths, following, lens, pairs)), k, v)
