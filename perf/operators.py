"""Workloads of the paged key/value cache operators, with their plain forms.

The operators serve a model whose answers are decoded over a catalog trie: every sequence's keys and values sit in
pages that sequences share; a step writes the keys of the new tokens (queries and keys normalised for each head and
rotated to their positions), attends from the new tokens (one token, a tree of drafted tokens, or a whole prompt) over
the cache, and keeps the rows of the drafted tokens that were accepted.

  attention   softmax(q k^T * scale) v of the new tokens of every sequence over its committed rows and over the new
              rows that a token sees: its ancestors in the tree of drafts (and itself), or all tokens up to itself
  write       the norm of queries and keys for each head, the rotation, the keys and values into their pages
  pages       sequences forked from others (pages shared by reference count), pages reserved for the drafted rows
              (the last page copied where it is shared), the drafted rows written, the accepted ones moved together
              and the pages past them given back

The head counts and widths are those of the hidden sizes 2048 (16 x 128), 4096 (32 x 128) and 256 (4 x 64) that the
decode workloads use, the batches 1, 64 and 256 theirs too.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------------------------------ cases

def _attention(name, dtype, heads, page, seqs, cached, new, tree):
    return {"name": name, "op": "attention", "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2],
            "page": page, "seqs": seqs, "cached_min": cached[0], "cached_max": cached[1], "new_min": new[0],
            "new_max": new[1], "tree": tree}


def _write(name, dtype, heads, page, seqs, cached, new, rotated, interleaved):
    return {"name": name, "op": "write", "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2],
            "page": page, "seqs": seqs, "cached_min": cached[0], "cached_max": cached[1], "new_min": new[0],
            "new_max": new[1], "rotated": rotated, "interleaved": interleaved}


def _pages(name, dtype, heads, page, layers, roots, seqs, cached, new):
    return {"name": name, "op": "pages", "dtype": dtype, "kv_heads": heads[1], "dim": heads[2], "page": page,
            "layers": layers, "roots": roots, "seqs": seqs, "cached_min": cached[0], "cached_max": cached[1],
            "new_min": new[0], "new_max": new[1]}


def listed():
    small, mid, big = (4, 2, 64), (16, 8, 128), (32, 8, 128)
    return [
        # the next token of one answer after a short prompt: nothing but latency
        _attention("attn_token_b1", "bf16", mid, 64, 1, (517, 517), (1, 1), False),
        # the next token of a batch of 64 with contexts of every length
        _attention("attn_token_b64_ragged", "bf16", big, 64, 64, (0, 8191), (1, 1), False),
        # drafts of the catalog's subtrees under 64 answers, verified in one pass
        _attention("attn_tree_b64", "bf16", mid, 64, 64, (1201, 2500), (5, 31), True),
        # a large tree of drafts over two very long contexts: few rows, a long axis
        _attention("attn_tree_long", "bf16", big, 64, 2, (90001, 120011), (63, 63), True),
        # whole prompts of different lengths packed into one pass, one of them behind a shared prefix
        _attention("attn_prompt", "bf16", big, 64, 3, (0, 1777), (2300, 4097), False),
        # fp32, as in the small test model: drafts in small pages
        _attention("attn_tree_f32", "f32", small, 16, 5, (0, 700), (1, 21), True),
        # one new token for each of 64 answers
        _write("write_token_b64", "bf16", big, 64, 64, (11, 8000), (1, 1), 128, False),
        # the tokens of whole prompts
        _write("write_prompt", "bf16", big, 64, 5, (0, 1000), (1801, 4100), 128, False),
        # fp32, adjacent pairs, half of the head rotated
        _write("write_draft_f32", "f32", small, 16, 9, (0, 333), (1, 37), 32, True),
        # a handful of branches from two prompts, one layer, small pages
        _pages("pages_b8", "f32", small, 16, 1, 2, 8, (19, 90), (1, 9)),
        # 64 answers of one product-sized model branch from one catalog prompt
        _pages("pages_b64", "bf16", mid, 64, 4, 1, 64, (1000, 1000), (3, 17)),
        # 256 answers from four prompts, drafts of up to 33 tokens, eight layers
        _pages("pages_b256", "bf16", big, 64, 8, 4, 256, (700, 2050), (0, 33)),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        heads = rng.choice([(4, 2, 64), (16, 8, 128), (32, 8, 128), (8, 1, 128), (6, 6, 64), (16, 4, 64), (8, 2, 256)])
        page = rng.choice([16, 32, 64, 128])
        op = rng.choice(["attention", "attention", "attention", "write", "pages"])
        if op == "attention":
            kind = rng.choice(["token", "tree", "tree", "prompt"])
            if kind == "token":
                seqs, new, top = _log(rng, 1, 256), (1, 1), _log(rng, 1, 60000)
            elif kind == "tree":
                hi = _log(rng, 2, 130)
                seqs, new, top = _log(rng, 1, 64), (rng.randint(0, hi), hi), _log(rng, 1, 100000)
            else:
                hi = _log(rng, 64, 4000)
                seqs, new, top = _log(rng, 1, 8), (rng.randint(1, hi), hi), rng.choice([0, _log(rng, 1, 4000)])
            case = _attention("", dtype, heads, page, seqs, (rng.randint(0, top), top), new, kind == "tree")
        elif op == "write":
            hi, top = rng.choice([1, _log(rng, 2, 4000)]), _log(rng, 1, 600 if dtype == "f32" else 60000)
            hi = min(hi, 300) if dtype == "f32" else hi
            case = _write("", dtype, heads, page, _log(rng, 1, 256), (rng.randint(0, top), top), (rng.randint(0, hi), hi),
                          rng.choice([0, 32, 64, heads[2]]), rng.random() < 0.5)
        else:
            hi, top, seqs = _log(rng, 1, 48), _log(rng, 1, 3000), _log(rng, 2, 256)
            case = _pages("", dtype, heads, page, rng.randint(1, 8), rng.randint(1, min(seqs - 1, 6)), seqs,
                          (rng.randint(1, top), top), (rng.randint(0, hi), hi))
        case.pop("name")
        rows = sum(sum(x) for x in zip(*_lengths(case)))
        cells = case["seqs"] * (case["cached_max"] + case["new_max"])  # what the plain form lays out, padded
        if 0 < rows < 400000 and sum(_lengths(case)[1]) and cells < 1500000 and 3072 not in case.values() \
                and _cost(case) <= most[op]:
            return case


# ----------------------------------------------------------------------------------------------------------- shapes

def _lengths(case):
    """Committed and new tokens of every sequence: part of the case, not of the seed."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["seqs"]
    cached = [_log(r, case["cached_min"], case["cached_max"]) if case["cached_max"] else 0 for _ in range(n)]
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(n)]
    cached[0], new[-1] = case["cached_max"], case["new_max"]
    if n > 1:
        cached[-1], new[0] = case["cached_min"], case["new_min"]
    if case["op"] == "pages":  # the sources keep their rows, the others are forked from them
        new = [0 if s < case["roots"] else new[s] for s in range(n)]
        cached = [c if s < case["roots"] else cached[s % case["roots"]] for s, c in enumerate(cached)]
    return cached, new


def _parents(case):
    """The tree of drafts: every token's parent among its sequence's new tokens, -1 where it follows the context."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + "tree")
    return [[-1 if i == 0 or r.random() < 0.05 else r.randint(max(0, i - 6), i - 1) for i in range(n)]
            for n in _lengths(case)[1]]


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _kept(case):
    """Accepted drafts of every sequence, ascending."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + "kept")
    return [sorted(r.sample(range(n), r.randint(0, n))) for n in _lengths(case)[1]]


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    cached, new = _lengths(case)
    row = 2 * case["kv_heads"] * case["dim"] * size  # keys and values of one token in one layer
    if case["op"] == "attention":
        q = case["q_heads"] * case["dim"]
        if case["tree"]:
            seen = sum(n * c + sum(d + 1 for d in _depths(p)) for c, n, p in zip(cached, new, _parents(case)))
        else:
            seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
        return {"bytes": sum(c + n for c, n in zip(cached, new) if n) * row + 2 * sum(new) * q * size, "flops": 4 * q * seen}
    if case["op"] == "write":
        values = sum(new) * (case["q_heads"] + 2 * case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * values * size + 8 * sum(new), "flops": 8 * values}
    page, layers = case["page"], case["layers"]
    shared = sum(c % page for c, n in zip(cached, new) if n)  # rows of the last page, where it is not full
    moved = sum(sum(i != j for j, i in enumerate(k)) for k in _kept(case))
    return {"bytes": 2 * layers * row * (shared + sum(new) + moved) + 8 * sum(-(-c // page) for c in cached), "flops": 0}


# ----------------------------------------------------------------------------------------------------------- inputs

def _offsets(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    order = random.Random(seed)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    cached, new = _lengths(case)
    page, dim, heads, seqs = case["page"], case["dim"], case["kv_heads"], case["seqs"]
    layers = case.get("layers", 1)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    # pages of every sequence in a random order of the pool; a few pages are nobody's
    width = max(max(-(-(c + n) // page) for c, n in zip(cached, new)), 1)
    if case["op"] == "pages":
        held = [-(-c // page) if s < case["roots"] else 0 for s, c in enumerate(cached)]
        spare = sum(1 + -(-n // page) for n in new if n) + 3
    else:
        held = [-(-(c + n) // page) for c, n in zip(cached, new)]
        spare = 3
    total = sum(held) + spare
    pool = list(range(total))
    order.shuffle(pool)
    table, refs = [[-1] * width for _ in range(seqs)], [0] * total
    for s, h in enumerate(held):
        for j in range(h):
            table[s][j] = pool.pop()
            refs[table[s][j]] = 1
    length = [c if h or case["op"] != "pages" else 0 for c, h in zip(cached, held)]
    kv = torch.empty((layers, total, 2, heads, page, dim), device=dev, dtype=dtype)
    for part in kv.view(layers * total, -1).split(256):
        part.copy_(normal(*part.shape))
    start = _offsets(new)
    tokens = start[-1]
    state = {"case": case, "kv": kv, "table": ints(table), "length": ints(length), "held": ints(held), "refs": ints(refs),
             "status": ints([0] * seqs), "start": ints(start), "max_new": max(new)}
    where = [s for s, n in enumerate(new) for _ in range(n)]
    if case["op"] == "attention":
        state["q"] = normal(tokens, case["q_heads"], dim)
        state["out"] = torch.empty_like(state["q"])
        state["scale"] = dim ** -0.5
        state["parent"] = ints([p for tree in _parents(case) for p in tree]) if case["tree"] else None
    elif case["op"] == "write":
        fused = normal(tokens, case["q_heads"] + 2 * heads, dim)  # the projection's rows: queries, keys, values
        state["q"], state["k"], state["v"] = fused.split([case["q_heads"], heads, heads], 1)
        state["q_out"] = torch.empty_like(state["q"], memory_format=torch.contiguous_format)
        state["q_weight"], state["k_weight"] = (1 + 0.2 * normal(dim).float()).to(dtype), (1 + 0.2 * normal(dim).float()).to(dtype)
        half = case["rotated"] // 2
        state["pos"] = ints([cached[s] + t - start[s] for t, s in enumerate(where)])
        state["inv_freq"] = (10000.0 ** -(torch.arange(half, device=dev, dtype=torch.float64) / max(half, 1))).float() if half else None
        state["eps"] = 1e-6
    else:
        state["src"] = ints([s if s < case["roots"] else s % case["roots"] for s in range(seqs)])
        state["n_new"] = ints(new)
        state["k"], state["v"] = normal(layers, tokens, heads, dim), normal(layers, tokens, heads, dim)
        kept = _kept(case)
        most = max(max(len(x) for x in kept), 1)
        state["n_keep"], state["keep"] = ints([len(x) for x in kept]), ints([x + [0] * (most - len(x)) for x in kept])
    return state


# ------------------------------------------------------------------------------------------------------ plain forms

def _places(s, row_of):
    """Page and slot of every new token: row_of[t] rows past the committed ones of its sequence."""
    start, page = s["start"].long(), s["kv"].shape[4]
    tokens = torch.arange(row_of.numel(), device=start.device)
    seq = torch.searchsorted(start, tokens, right=True) - 1
    row = s["length"].long()[seq] + row_of
    return s["table"].long()[seq, row // page], row % page


def _new_rows(s):
    """Which of its sequence's new tokens every token is."""
    start = s["start"].long()
    tokens = torch.arange(s["k"].shape[-3], device=start.device)
    return tokens - start[torch.searchsorted(start, tokens, right=True) - 1]


def _plain_attention(s):
    q, kv, start, length = s["q"], s["kv"], s["start"].long(), s["length"].long()
    tokens, q_heads, dim = q.shape
    heads, page = kv.shape[3], kv.shape[4]
    seqs, most = length.numel(), s["max_new"]
    rows = kv[0][s["table"].long().clamp(min=0)]                     # [seqs][pages][2][heads][page][dim]
    k, v = (rows[:, :, i].transpose(1, 2).reshape(seqs, heads, -1, dim).float() for i in (0, 1))
    count = start[1:] - start[:-1]
    i = torch.arange(most, device=q.device)
    at = (start[:-1, None] + i).clamp(max=tokens - 1)                # [seqs][most]
    x = q[at].float().view(seqs, most, heads, -1, dim).permute(0, 2, 3, 1, 4).reshape(seqs, heads, -1, dim)
    score = (x @ k.transpose(2, 3).contiguous()).view(seqs, heads, -1, most, k.shape[2]) * s["scale"]
    key = torch.arange(k.shape[2], device=q.device)
    new = key - length[:, None]                                      # [seqs][keys]: which new token a key is
    if s["parent"] is None:
        seen = new[:, None, :] <= i[:, None]
    else:
        # a token sees itself and whoever its parent sees: powers of (identity + parents)
        parent = s["parent"].long()[at]
        see = torch.eye(most, device=q.device) + (parent[:, :, None] == i).float()
        for _ in range(most.bit_length()):
            see = ((see @ see) > 0).float()
        among = see.gather(2, new.clamp(0, most - 1)[:, None, :].expand(-1, most, -1)) > 0
        seen = (new < 0)[:, None, :] | (among & (new < count[:, None])[:, None, :])
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    weight = torch.exp(score - score.amax(-1, keepdim=True))
    weight = weight / weight.sum(-1, keepdim=True)
    y = (weight.view(seqs, heads, -1, k.shape[2]) @ v).view(seqs, q_heads, most, dim).transpose(1, 2)
    s["out"].copy_(y[i < count[:, None]])
    return s["out"]


def _plain_head(x, weight, eps, angle, interleaved):
    """Norm of every head and rotation of its first 2 * angle.shape[-1] values."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()
    if angle is None:
        return x
    cos, sin, turn = angle.cos()[:, None], angle.sin()[:, None], 2 * angle.shape[-1]
    a, b = (x[..., 0:turn:2], x[..., 1:turn:2]) if interleaved else x[..., :turn].chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((head, x[..., turn:]), -1)


def _plain_write(s):
    angle = None if s["inv_freq"] is None else s["pos"].float()[:, None] * s["inv_freq"]
    turn = s["case"]["interleaved"]
    s["q_out"].copy_(_plain_head(s["q"], s["q_weight"], s["eps"], angle, turn))
    page, slot = _places(s, _new_rows(s))
    layer = s["kv"][0]
    layer[page, 0, :, slot] = _plain_head(s["k"], s["k_weight"], s["eps"], angle, turn).to(layer.dtype)
    layer[page, 1, :, slot] = s["v"]
    return {"q": s["q_out"], "kv": s["kv"]}


def _count(s):
    """Reference counts: how many sequences hold each page."""
    held = s["table"].long().flatten() + 1
    s["refs"].copy_(torch.zeros(s["refs"].numel() + 1, device=held.device, dtype=torch.int32)
                    .index_add_(0, held, torch.ones_like(held, dtype=torch.int32))[1:])


def _plain_fork(s):
    src, page = s["src"].long(), s["kv"].shape[4]
    me = torch.arange(src.numel(), device=src.device)
    of = src.clamp(min=0)
    pages = (s["length"].long()[of] + page - 1) // page
    j = torch.arange(s["table"].shape[1], device=src.device)
    table = torch.where((j < pages[:, None]) & (src >= 0)[:, None], s["table"][of], -1)
    stay = src == me
    s["table"].copy_(torch.where(stay[:, None], s["table"], table))
    s["held"].copy_(torch.where(stay, s["held"], torch.where(src < 0, 0, pages)))
    s["length"].copy_(torch.where(src < 0, 0, s["length"][of]))
    _count(s)


def _plain_reserve(s):
    kv, page = s["kv"], s["kv"].shape[4]
    length, held, n = s["length"].long(), s["held"].long(), s["n_new"].long()
    table, refs = s["table"].long(), s["refs"].long()
    last = (length // page).clamp(max=table.shape[1] - 1)            # the page of the first new row
    shared = table.gather(1, last[:, None])[:, 0]
    split = (n > 0) & (length % page > 0) & (refs[shared.clamp(min=0)] > 1)
    want = torch.where(n > 0, torch.maximum((length + n + page - 1) // page, held), held)
    more = want - held + split
    end = more.cumsum(0)
    free = torch.argsort((refs != 0).int(), stable=True)             # free pages first, lowest first
    fits = (end <= (refs == 0).sum()) | (more == 0)
    s["status"].copy_(torch.where(fits, s["status"], 9))
    split, want = split & fits, torch.where(fits, want, held)
    take = end - more
    j = torch.arange(table.shape[1], device=length.device)
    nth = (take + split)[:, None] + j - held[:, None]
    table = torch.where((j >= held[:, None]) & (j < want[:, None]), free[nth.clamp(0, free.numel() - 1)], table)
    copy = free[take.clamp(max=free.numel() - 1)]
    table = torch.where((j == last[:, None]) & split[:, None], copy[:, None], table)
    to, rows = torch.where(split, copy, shared), torch.where(split, length % page, 0)
    keep = torch.arange(page, device=length.device)[:, None] < rows[:, None, None, None, None]
    on = split.nonzero()[:, 0]
    kv[:, to[on]] = torch.where(keep[on], kv[:, shared[on]], kv[:, to[on]])
    s["table"].copy_(table)
    s["held"].copy_(want)
    _count(s)


def _plain_commit(s):
    kv, page, keep, n_keep = s["kv"], s["kv"].shape[4], s["keep"].long(), s["n_keep"].long()
    length, table = s["length"].long(), s["table"].long()
    j = torch.arange(keep.shape[1], device=kv.device)
    seq, j = ((j < n_keep[:, None]) & (keep != j)).nonzero().unbind(1)
    to, row = length[seq] + j, length[seq] + keep[seq, j]
    kv[:, table[seq, to // page], :, :, to % page] = kv[:, table[seq, row // page], :, :, row % page]
    s["length"].copy_(length + n_keep)
    pages = (s["length"] + page - 1) // page
    s["table"].masked_fill_(torch.arange(table.shape[1], device=kv.device) >= pages[:, None], -1)
    s["held"].copy_(pages)
    _count(s)


def _plain_pages(s):
    _plain_fork(s)
    _plain_reserve(s)
    page, slot = _places(s, _new_rows(s))
    s["kv"][:, page, 0, :, slot] = s["k"].transpose(0, 1)
    s["kv"][:, page, 1, :, slot] = s["v"].transpose(0, 1)
    _plain_commit(s)
    return {n: s[n] for n in ("kv", "table", "length", "held", "refs", "status")}


# -------------------------------------------------------------------------------------------------- the framework's

def _own(s):
    import trie_masked_sparse_amd as tms
    if "cache" not in s:  # the handle that a program keeps: it holds these tensors
        s["cache"] = tms.PagedCache(s["kv"], s["table"], s["length"], s["held"], s["refs"], s["status"])
    cache, op = s["cache"], s["case"]["op"]
    if op == "attention":
        tms.kv_attention(cache, 0, s["q"], s["start"], s["out"], s["scale"], parent=s["parent"], max_new=s["max_new"])
        return s["out"]
    if op == "write":
        tms.kv_write(cache, 0, s["k"], s["v"], s["start"], q=s["q"], q_out=s["q_out"], q_weight=s["q_weight"],
                     k_weight=s["k_weight"], eps=s["eps"], pos=s["pos"] if s["inv_freq"] is not None else None,
                     inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"])
        return {"q": s["q_out"], "kv": s["kv"]}
    tms.kv_fork(cache, s["src"], check=False)
    tms.kv_reserve(cache, s["n_new"], check=False)
    for layer in range(s["case"]["layers"]):
        tms.kv_write(cache, layer, s["k"][layer], s["v"][layer], s["start"])
    tms.kv_commit(cache, s["n_keep"], s["keep"], check=False)
    return {n: s[n] for n in ("kv", "table", "length", "held", "refs", "status")}


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "write": _plain_write, "pages": _plain_pages}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------------------ exact

def _exact_attention(case, s):
    cached, new = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, table, begin = case["q_heads"] // case["kv_heads"], s["table"].tolist(), 0
    for b, (c, n) in enumerate(zip(cached, new)):
        if not n:
            continue
        pages = [p for p in table[b] if p >= 0]
        sees = torch.zeros((n, c + n), dtype=torch.bool)
        sees[:, :c] = True
        if case["tree"]:
            for i, p in enumerate(_parents(case)[b]):
                if p >= 0:
                    sees[i] |= sees[p]
                sees[i, c + i] = True
        else:
            sees[:, c:] = torch.ones((n, n), dtype=torch.bool).tril()
        sees = sees.cuda()
        for h in range(case["kv_heads"]):
            k, v = (s["kv"][0, pages, i, h].reshape(-1, case["dim"])[:c + n].double() for i in (0, 1))
            for g in range(h * group, (h + 1) * group):
                score = (s["q"][begin:begin + n, g].double() @ k.T) / math.sqrt(case["dim"])
                score[~sees] = -math.inf
                out[begin:begin + n, g] = torch.softmax(score, -1) @ v
        begin += n
    return out


def _exact_write(case, s):
    cached, new = _lengths(case)
    q, kv, table, page = s["q"].double(), s["kv"].double(), s["table"].tolist(), case["page"]
    pos = torch.tensor([c + i for c, n in zip(cached, new) for i in range(n)], dtype=torch.float64, device="cuda")

    def head(x, w):
        x = x.double()
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["dim"] + 1e-6) * w.double()
        half = case["rotated"] // 2
        y = x.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            t = (pos * s["inv_freq"][i].double())[:, None]
            y[..., a] = x[..., a] * torch.cos(t) - x[..., b] * torch.sin(t)
            y[..., b] = x[..., a] * torch.sin(t) + x[..., b] * torch.cos(t)
        return y

    k, v = head(s["k"], s["k_weight"]), s["v"].double()
    rows = [(table[b][r // page], r % page) for b, (c, n) in enumerate(zip(cached, new)) for r in range(c, c + n)]
    p, r = torch.tensor(rows, device="cuda").unbind(1)
    for h in range(case["kv_heads"]):
        kv[0, p, 0, h, r] = k[:, h]
        kv[0, p, 1, h, r] = v[:, h]
    return {"q": head(q, s["q_weight"]), "kv": kv}


def _exact_pages(case, s):
    page, seqs, layers = case["page"], case["seqs"], case["layers"]
    cached, new = _lengths(case)
    kept, kv = _kept(case), s["kv"].clone()
    table = [[p for p in row if p >= 0] for row in s["table"].tolist()]
    of = [b if b < case["roots"] else b % case["roots"] for b in range(seqs)]
    table = [list(table[x]) for x in of]
    holders = {}
    for row in table:
        for p in row:
            holders[p] = holders.get(p, 0) + 1
    free = [p for p in range(kv.shape[1]) if p not in holders]
    begin, moves = 0, []
    for b in range(seqs):
        c, n = cached[b], new[b]
        if n and c % page and holders[table[b][-1]] > 1:
            p, table[b][-1] = table[b][-1], free.pop(0)
            kv[:, table[b][-1], :, :, :c % page] = kv[:, p, :, :, :c % page]
        while n and len(table[b]) * page < c + n:
            table[b].append(free.pop(0))
        at = [(table[b][r // page], r % page) for r in range(c, c + n)]
        moves += [(at[j], begin + i, i != j) for j, i in enumerate(kept[b])]
        if n:
            p, r = torch.tensor(at, device="cuda").unbind(1)
            kv[:, p, 0, :, r] = s["k"][:, begin:begin + n].transpose(0, 1)
            kv[:, p, 1, :, r] = s["v"][:, begin:begin + n].transpose(0, 1)
        table[b] = table[b][:-(-(c + len(kept[b])) // page)]
        begin += n
    moved = [(p, r, t) for (p, r), t, other in moves if other]
    if moved:
        p, r, t = torch.tensor(moved, device="cuda").unbind(1)
        kv[:, p, 0, :, r] = s["k"][:, t].transpose(0, 1)
        kv[:, p, 1, :, r] = s["v"][:, t].transpose(0, 1)
    refs = [0] * kv.shape[1]
    for row in table:
        for p in row:
            refs[p] += 1
    width = s["table"].shape[1]
    whole = {"table": [row + [-1] * (width - len(row)) for row in table], "refs": refs, "held": [len(row) for row in table],
             "length": [c + len(x) for c, x in zip(cached, kept)], "status": [0] * seqs}
    return {"kv": kv} | {n: torch.tensor(x, dtype=torch.int32) for n, x in whole.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "write": _exact_write, "pages": _exact_pages}[case["op"]](case, s)
