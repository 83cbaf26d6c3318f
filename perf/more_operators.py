"""Workloads of the operators that read long contexts of the paged key/value cache, with their plain forms.

Answers that are decoded over a catalog start from one long prompt (the catalog's entries, written out), so the sequences
of a batch hold the same pages, and of a long context a token needs few rows.

  shared   attention of the new tokens of a batch whose sequences share pages (one prompt, or several that begin with
           the same rows), over some layers: softmax(q k^T * scale) v over the committed rows and the new rows seen
  bounds   of every page that the last committed rows have made whole: the lowest and the highest key of each column
  select   the pages that a token reads: the first and the last whole ones and those with the highest bounds on q k
           (summed over the query heads of a key head), ascending; of equal scores the lower page
  pages    attention of the new tokens over their own choice of pages for each key head, the committed rows behind the
           last whole page, and the new rows seen

The head counts and widths are those of the hidden sizes 2048 (16 x 128), 4096 (32 x 128) and 256 (4 x 64) that the
decode workloads use, the batches 1, 64 and 256 theirs too.
"""
import math
import random
import zlib

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------------------------ cases

def _case(name, op, dtype, heads, page, seqs, new, **more):
    return {"name": name, "op": op, "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2],
            "page": page, "seqs": seqs, "new_min": new[0], "new_max": new[1], **more}


def _shared(name, dtype, heads, page, seqs, new, tree, layers, prompts, common, prompt, own_max):
    """`prompts` prompts whose first `common` pages are the same; sequence s goes on from prompt s % prompts with up to
    own_max committed rows of its own."""
    return _case(name, "shared", dtype, heads, page, seqs, new, tree=tree, layers=layers, prompts=prompts, common=common,
                 prompt_min=prompt[0], prompt_max=prompt[1], own_max=own_max)


def _bounds(name, dtype, heads, page, seqs, new, layers, cached):
    return _case(name, "bounds", dtype, heads, page, seqs, new, layers=layers, cached_min=cached[0], cached_max=cached[1])


def _select(name, dtype, heads, page, seqs, new, cached, pick, first, last):
    return _case(name, "select", dtype, heads, page, seqs, new, cached_min=cached[0], cached_max=cached[1], pick=pick,
                 first=first, last=last)


def _pages(name, dtype, heads, page, seqs, new, tree, cached, pick):
    return _case(name, "pages", dtype, heads, page, seqs, new, tree=tree, cached_min=cached[0], cached_max=cached[1],
                 pick=pick)


def listed():
    small, mid, big = (4, 2, 64), (16, 8, 128), (32, 8, 128)
    return [
        # four answers of the small test model behind one short prompt: nothing but latency
        _shared("shared_b4_f32", "f32", small, 16, 4, (1, 1), False, 1, 1, 0, (150, 150), 20),
        # the next token of 64 answers over one catalog prompt
        _shared("shared_b64_token", "bf16", big, 64, 64, (1, 1), False, 2, 1, 0, (9000, 9000), 400),
        # drafts of the catalog's subtrees under 64 answers, from four prompts with the same beginning
        _shared("shared_b64_tree", "bf16", mid, 64, 64, (5, 31), True, 2, 4, 10, (1201, 2500), 200),
        # 256 answers from four long prompts with the same beginning
        _shared("shared_b256_long", "bf16", big, 64, 256, (1, 1), False, 1, 4, 32, (9000, 24000), 1000),
        # after a step of 64 answers: a page in 64 tokens becomes whole
        _bounds("bounds_token_b64", "bf16", mid, 64, 64, (1, 1), 4, (11, 8000)),
        # after whole prompts, eight layers
        _bounds("bounds_prompt", "bf16", big, 64, 5, (1801, 4100), 8, (0, 1000)),
        # the next token of one answer behind a very long context
        _select("select_b1_long", "bf16", big, 64, 1, (1, 1), (120011, 120011), 64, 1, 2),
        # the next token of 64 answers with contexts of every length
        _select("select_b64_ragged", "bf16", big, 64, 64, (1, 1), (100, 60000), 32, 1, 1),
        # drafts over small pages, fp32
        _select("select_tree_f32", "f32", small, 16, 5, (1, 21), (0, 2000), 16, 0, 1),
        # the next token of one answer over its choice of pages: latency
        _pages("pages_b1", "bf16", mid, 64, 1, (1, 1), False, (60007, 60007), 32),
        # 64 answers, contexts of every length
        _pages("pages_b64_ragged", "bf16", big, 64, 64, (1, 1), False, (100, 60000), 64),
        # drafts under 16 answers, each with a choice of its own
        _pages("pages_tree_b16", "bf16", mid, 32, 16, (3, 13), True, (1000, 20000), 24),
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
        op = rng.choice(["shared", "shared", "bounds", "select", "select", "pages", "pages"])
        hi = rng.choice([1, 1, _log(rng, 2, 40)])
        new, tree = (rng.randint(0, hi) if hi > 1 else 1, hi), hi > 1 and rng.random() < 0.6
        if op == "shared":
            seqs, top = _log(rng, 2, 256), _log(rng, 20, 30000)
            prompts = rng.randint(1, min(seqs, 5))
            low = rng.randint(top // 3, top)
            case = _shared("", dtype, heads, page, seqs, new, tree, rng.randint(1, 3), prompts, rng.choice([0, low // page // 2]),
                           (low, top), rng.choice([0, _log(rng, 1, 1000)]))
        elif op == "bounds":
            hi, top = rng.choice([1, _log(rng, 2, 4000)]), _log(rng, 1, 20000)
            case = _bounds("", dtype, heads, page, _log(rng, 1, 256), (rng.randint(0, hi), hi), rng.randint(1, 8),
                           (rng.randint(0, top), top))
        else:
            top, seqs = _log(rng, 50, 120000), _log(rng, 1, 128)
            cached = (rng.randint(0, top), top)
            if op == "select":
                case = _select("", dtype, heads, page, seqs, new, cached, _log(rng, 4, 200), rng.randint(0, 2), rng.randint(0, 2))
            else:
                case = _pages("", dtype, heads, page, seqs, new, tree, cached, _log(rng, 1, 200))
        case.pop("name")
        cached, new = _lengths(case)
        row = 2 * case["kv_heads"] * case["dim"] * case.get("layers", 1) * (2 if dtype == "bf16" else 4)
        if sum(new) and (sum(cached) + sum(new)) * row < 24e9 and sum(new) < (1500 if op == "pages" else 6000) \
                and 0 < _cost(case) <= most[op]:
            return case


# ----------------------------------------------------------------------------------------------------------- shapes

def _random(case, what):
    """Random numbers that are part of the case, not of the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + what)


def _prompts(case):
    """Rows of every prompt: at least its common pages."""
    r = _random(case, "prompts")
    rows = [r.randint(case["prompt_min"], case["prompt_max"]) for _ in range(case["prompts"])]
    rows[-1] = case["prompt_max"]
    return [max(x, case["common"] * case["page"]) for x in rows]


def _lengths(case):
    """Committed and new tokens of every sequence."""
    r, n = _random(case, "lengths"), case["seqs"]
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(n)]
    new[-1] = case["new_max"]
    if case["op"] == "shared":
        prompts = _prompts(case)
        return [prompts[s % case["prompts"]] + r.randint(0, case["own_max"]) for s in range(n)], new
    cached = [_log(r, case["cached_min"], case["cached_max"]) if case["cached_max"] else 0 for _ in range(n)]
    cached[0] = case["cached_max"]
    if n > 1:
        cached[-1], new[0] = case["cached_min"], case["new_min"]
    return cached, new


def _parents(case):
    """The tree of drafts: every token's parent among its sequence's new tokens, -1 where it follows the context."""
    r = _random(case, "tree")
    return [[-1 if i == 0 or r.random() < 0.05 else r.randint(max(0, i - 6), i - 1) for i in range(n)]
            for n in _lengths(case)[1]]


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _chosen(case):
    """A choice of pages for every new token and key head: [tokens][kv_heads][pick], ascending, -1 past the whole pages.
    The drafts of a sequence have three quarters of theirs in common."""
    rng = np.random.default_rng(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))
    heads, pick = case["kv_heads"], case["pick"]
    out = []
    for c, n in zip(*_lengths(case)):
        whole = c // case["page"]
        x = np.full((n, heads, pick), -1, np.int32)
        k = min(whole, pick)
        for h in range(heads):
            same = rng.permutation(whole)[:k]
            for i in range(n):
                mine = same
                if whole > k and i:
                    fixed = same[:k - k // 4]
                    rest = rng.permutation(whole)
                    mine = np.concatenate([fixed, rest[~np.isin(rest, fixed)][:k // 4]])
                x[i, h, :k] = np.sort(mine)
        out.append(x)
    return np.concatenate(out)


def _seen(case, cached, new):
    """Rows that the new tokens see, in all, `cached` of every sequence among them."""
    if case["tree"]:
        return sum(n * c + sum(d + 1 for d in _depths(p)) for c, n, p in zip(cached, new, _parents(case)))
    return sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    cached, new = _lengths(case)
    page, dim, heads, op = case["page"], case["dim"], case["kv_heads"], case["op"]
    q = case["q_heads"] * dim
    if op == "shared":
        prompts, common = _prompts(case), case["common"] * page
        used = {s % len(prompts) for s, n in enumerate(new) if n}
        rows = common + sum(prompts[i] // page * page - common for i in used)
        rows += sum(c + n - prompts[s % len(prompts)] // page * page for s, (c, n) in enumerate(zip(cached, new)) if n)
        return {"bytes": case["layers"] * (rows * 2 * heads * dim + 2 * sum(new) * q) * size,
                "flops": case["layers"] * 4 * q * _seen(case, cached, new)}
    if op == "bounds":
        whole = sum(c // page - (c - n) // page for c, n in zip(_committed(case), new))
        return {"bytes": case["layers"] * whole * heads * (page + 2) * dim * size, "flops": case["layers"] * whole * heads * page * 2 * dim}
    if op == "select":
        free = [(max(c // page - case["first"] - case["last"], 0) if c // page > case["pick"] else 0) * (n > 0) for c, n in zip(cached, new)]
        return {"bytes": sum(free) * heads * 2 * dim * size + sum(new) * (q * size + 4 * heads * case["pick"]),
                "flops": sum(f * n for f, n in zip(free, new)) * heads * 4 * dim}
    chosen, at, rows = _chosen(case), 0, 0
    for c, n in zip(cached, new):
        if n:
            for h in range(heads):
                x = np.unique(chosen[at:at + n, h])
                rows += int((x >= 0).sum()) * page + c % page + n
        at += n
    picked = [min(c // page, case["pick"]) * page + c % page for c in cached]
    return {"bytes": rows * 2 * dim * size + 2 * sum(new) * q * size + chosen.size * 4, "flops": 4 * q * _seen(case, picked, new)}


def _committed(case):
    """Committed rows of the `bounds` cases: the last n of a sequence are what it has just committed."""
    cached, new = _lengths(case)
    return [c + n for c, n in zip(cached, new)]


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
    page, dim, heads, seqs, layers = case["page"], case["dim"], case["kv_heads"], case["seqs"], case.get("layers", 1)
    if case["op"] == "bounds":
        cached = _committed(case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    # pages of every sequence in a random order of the pool; a few pages are nobody's
    rows = [c + (n if case["op"] != "bounds" else 0) for c, n in zip(cached, new)]
    held = [-(-r // page) for r in rows]
    begin = [0] * seqs                                               # pages that a sequence shares
    total = sum(held) + 3
    if case["op"] == "shared":
        prompts = _prompts(case)
        begin = [prompts[s % len(prompts)] // page for s in range(seqs)]
        total = sum(h - b for h, b in zip(held, begin)) + sum(p // page for p in prompts) + 3
    pool = list(range(total))
    order.shuffle(pool)
    first = []                                                       # the pages of every prompt
    if case["op"] == "shared":
        same = [pool.pop() for _ in range(case["common"])]
        first = [same + [pool.pop() for _ in range(p // page - len(same))] for p in prompts]
    table, refs = [], [0] * total
    for s in range(seqs):
        table.append((list(first[s % len(first)]) if first else []) + [pool.pop() for _ in range(held[s] - begin[s])])
        for p in table[s]:
            refs[p] += 1
    width = max(max(held), 1)
    table = [x + [-1] * (width - len(x)) for x in table]
    kv = torch.empty((layers, total, 2, heads, page, dim), device=dev, dtype=dtype)
    for part in kv.view(layers * total, 2, heads, page, dim).split(128):
        part.copy_(normal(*part.shape))
        part[:, 0] += 0.5 * normal(part.shape[0], heads, 1, dim)     # keys of a page are alike
    start = _offsets(new)
    tokens = start[-1]
    state = {"case": case, "kv": kv, "table": ints(table), "length": ints(cached), "held": ints(held), "refs": ints(refs),
             "status": ints([0] * seqs), "start": ints(start), "max_new": max(new), "cached": cached, "new": new,
             "scale": dim ** -0.5}
    if case["op"] != "bounds":
        q = normal(layers, tokens, case["q_heads"], dim)
        state["q"] = q if case["op"] == "shared" else q[0]
    if case["op"] in ("shared", "pages"):
        state["out"] = torch.empty_like(state["q"])
        state["parent"] = ints([p for tree in _parents(case) for p in tree]) if case["tree"] else None
    if case["op"] in ("bounds", "select"):
        state["bounds"] = torch.zeros((layers, total, heads, 2, dim), device=dev, dtype=dtype)
    if case["op"] == "bounds":
        state["n_new"] = ints(new)
    if case["op"] == "select":
        for part, keys in zip(state["bounds"][0].split(128), kv[0].split(128)):
            part.copy_(torch.stack((keys[:, 0].amin(2), keys[:, 0].amax(2)), 2))
        state["chosen"] = torch.empty((tokens, heads, case["pick"]), device=dev, dtype=torch.int32)
    if case["op"] == "pages":
        state["chosen"] = torch.from_numpy(_chosen(case)).to(dev)
    return state


# ------------------------------------------------------------------------------------------------------ plain forms

def _tree(parent):
    """Who sees whom: powers of (identity + parents)."""
    n = parent.numel()
    i = torch.arange(n, device=parent.device)
    see = torch.eye(n, device=parent.device) + (parent[:, None] == i).float()
    for _ in range(n.bit_length()):
        see = ((see @ see) > 0).float()
    return see > 0


def _new_seen(s, b, at, n):
    """Which of its sequence's new rows each new token sees."""
    if s["parent"] is not None:
        return _tree(s["parent"][at:at + n].long())
    i = torch.arange(n, device=s["q"].device)
    return i[None, :] <= i[:, None]


def _softmax_product(q, k, v, seen, scale):
    """q [n][heads][group][D], k and v [heads][rows][D], seen [n][rows] or [heads][n][rows]."""
    n, heads, group, dim = q.shape
    x = q.permute(1, 0, 2, 3).reshape(heads, n * group, dim)
    score = (x @ k.transpose(1, 2).contiguous()).view(heads, n, group, -1) * scale
    score = score.masked_fill(~(seen if seen.dim() == 3 else seen[None])[:, :, None, :], float("-inf"))
    weight = torch.exp(score - score.amax(-1, keepdim=True))
    weight = weight / weight.sum(-1, keepdim=True)
    y = weight.view(heads, n * group, -1) @ v
    return y.view(heads, n, group, dim).permute(1, 0, 2, 3).reshape(n, heads * group, dim)


def _plain_shared(s):
    heads, page, dim = s["kv"].shape[3:]
    at = 0
    for b, (c, n) in enumerate(zip(s["cached"], s["new"])):
        if not n:
            continue
        pages = s["table"][b, :-(-(c + n) // page)].long()
        seen = _new_seen(s, b, at, n)
        seen = torch.cat((torch.ones((n, c), dtype=torch.bool, device=seen.device), seen), 1)
        for layer in range(s["kv"].shape[0]):
            rows = s["kv"][layer, pages].float()                     # [pages][2][heads][page][dim]
            k, v = (rows[:, i].transpose(0, 1).reshape(heads, -1, dim)[:, :c + n] for i in (0, 1))
            q = s["q"][layer, at:at + n].float().view(n, heads, -1, dim)
            s["out"][layer, at:at + n] = _softmax_product(q, k, v, seen, s["scale"]).to(s["out"].dtype)
        at += n
    return s["out"]


def _plain_bounds(s):
    page = s["kv"].shape[4]
    for b, (c, n) in enumerate(zip(s["cached"], s["new"])):
        first, last = (c - n) // page, c // page
        if first < last:
            pages = s["table"][b, first:last].long()
            for layer in range(s["kv"].shape[0]):
                keys = s["kv"][layer, pages, 0].float()
                s["bounds"][layer, pages] = torch.stack((keys.amin(2), keys.amax(2)), 2).to(s["bounds"].dtype)
    return s["bounds"]


def _plain_select(s):
    case, page = s["case"], s["kv"].shape[4]
    heads, dim, pick = case["kv_heads"], case["dim"], case["pick"]
    at = 0
    s["chosen"].fill_(-1)
    for b, (c, n) in enumerate(zip(s["cached"], s["new"])):
        whole = c // page
        if n and whole:
            q = s["q"][at:at + n].double().view(n, heads, -1, dim)
            over, under = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)   # [n][heads][dim]
            bound = s["bounds"][0, s["table"][b, :whole].long()].double()  # [whole][heads][2][dim]
            score = torch.empty((n, heads, whole), dtype=torch.float64, device=q.device)
            for i in range(n):
                score[i] = (over[i] * bound[:, :, 1] + under[i] * bound[:, :, 0]).sum(-1).T
            score[..., :case["first"]] = float("inf")
            score[..., max(whole - case["last"], 0):] = float("inf")
            best = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :pick]
            s["chosen"][at:at + n, :, :best.shape[-1]] = torch.sort(best, -1)[0].to(torch.int32)
        at += n
    return s["chosen"]


def _plain_pages(s):
    heads, page, dim = s["kv"].shape[3:]
    pick = s["chosen"].shape[2]
    at = 0
    for b, (c, n) in enumerate(zip(s["cached"], s["new"])):
        if not n:
            continue
        whole = c // page
        tail = s["kv"][0, s["table"][b, whole:-(-(c + n) // page)].long()]
        k1, v1 = (tail[:, i].transpose(0, 1).reshape(heads, -1, dim)[:, :c + n - whole * page].float() for i in (0, 1))
        among = torch.cat((torch.ones((n, c - whole * page), dtype=torch.bool, device=k1.device), _new_seen(s, b, at, n)), 1)
        head = torch.arange(heads, device=k1.device)[:, None]
        for i in range(n):
            chosen = s["chosen"][at + i].long()                      # [heads][pick]
            rows = s["kv"][0, s["table"][b].long()[chosen.clamp(min=0)], :, head].float()  # [heads][pick][2][page][dim]
            k, v = (torch.cat((rows[:, :, j].reshape(heads, -1, dim), x), 1) for j, x in ((0, k1), (1, v1)))
            seen = (chosen >= 0)[:, :, None].expand(heads, pick, page).reshape(heads, 1, -1)
            seen = torch.cat((seen, among[i].expand(heads, 1, -1)), 2)
            q = s["q"][at + i].float().view(1, heads, -1, dim)
            s["out"][at + i] = _softmax_product(q, k, v, seen, s["scale"])[0].to(s["out"].dtype)
        at += n
    return s["out"]


# -------------------------------------------------------------------------------------------------- the framework's

def _own(s):
    import trie_masked_sparse_amd as tms
    op = s["case"]["op"]
    if "cache" not in s:  # the handles that a program keeps: the cache holds these tensors, the others their work memory
        s["cache"] = tms.PagedCache(s["kv"], s["table"], s["length"], s["held"], s["refs"], s["status"])
        if op == "shared":
            s["plan"] = tms.SharedPlan(s["cache"], s["q"].shape[1], s["case"]["q_heads"])
        if op in ("bounds", "select"):
            s["index"] = tms.PageIndex(s["cache"], s["bounds"], tokens=s["q"].shape[0] if op == "select" else 1)
    cache = s["cache"]
    if op == "shared":
        tms.kv_share(cache, s["plan"], s["start"])
        for layer in range(s["kv"].shape[0]):
            tms.kv_attention_shared(cache, layer, s["q"][layer], s["start"], s["out"][layer], s["plan"], s["scale"],
                                    parent=s["parent"], max_new=s["max_new"])
        return s["out"]
    if op == "bounds":
        tms.kv_bounds(cache, s["index"], s["n_new"], max_new=s["max_new"])
        return s["bounds"]
    if op == "select":
        tms.kv_select(cache, 0, s["q"], s["start"], s["index"], s["chosen"], s["scale"], first=s["case"]["first"],
                      last=s["case"]["last"], max_new=s["max_new"])
        return s["chosen"]
    tms.kv_attention_pages(cache, 0, s["q"], s["start"], s["chosen"], s["out"], s["scale"], parent=s["parent"],
                           max_new=s["max_new"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"shared": _plain_shared, "bounds": _plain_bounds, "select": _plain_select, "pages": _plain_pages}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------------------ exact

def _sees(case, b, c, n):
    """Of c committed rows and the new ones of sequence b: who sees what, on the CPU."""
    sees = torch.zeros((n, c + n), dtype=torch.bool)
    sees[:, :c] = True
    if case["tree"]:
        for i, p in enumerate(_parents(case)[b]):
            if p >= 0:
                sees[i] |= sees[p]
            sees[i, c + i] = True
    else:
        sees[:, c:] = torch.ones((n, n), dtype=torch.bool).tril()
    return sees


def _exact_shared(case, s):
    cached, new = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, table, begin = case["q_heads"] // case["kv_heads"], s["table"].tolist(), 0
    for b, (c, n) in enumerate(zip(cached, new)):
        if not n:
            continue
        pages = torch.tensor([p for p in table[b] if p >= 0], device="cuda")
        hidden = ~_sees(case, b, c, n).cuda()
        for layer in range(case["layers"]):
            for h in range(case["kv_heads"]):
                k, v = (s["kv"][layer, pages, i, h].reshape(-1, case["dim"])[:c + n].double() for i in (0, 1))
                score = torch.einsum("tgd,rd->gtr", s["q"][layer, begin:begin + n, h * group:(h + 1) * group].double(), k)
                score = (score / math.sqrt(case["dim"])).masked_fill(hidden, -math.inf)
                out[layer, begin:begin + n, h * group:(h + 1) * group] = (torch.softmax(score, -1) @ v).transpose(0, 1)
        begin += n
    return out


def _exact_bounds(case, s):
    out = torch.zeros(s["bounds"].shape, dtype=torch.float64, device="cuda")
    table = s["table"].tolist()
    for b, (c, n) in enumerate(zip(_committed(case), _lengths(case)[1])):
        for j in range(c // case["page"]):
            if (j + 1) * case["page"] > c - n:
                keys = s["kv"][:, table[b][j], 0].double()
                out[:, table[b][j], :, 0] = keys.min(2)[0]
                out[:, table[b][j], :, 1] = keys.max(2)[0]
    return out


def _exact_select(case, s):
    cached, new = _lengths(case)
    table, q, bounds = s["table"].tolist(), s["q"].double().cpu().numpy(), s["bounds"][0].float().cpu().numpy()
    out = np.full((len(q), case["kv_heads"], case["pick"]), -1, np.int32)
    group, at = case["q_heads"] // case["kv_heads"], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        whole = c // case["page"]
        always = [j for j in range(whole) if j < case["first"] or j >= whole - case["last"]]
        for h in range(case["kv_heads"] if n and whole else 0):
            low, high = (bounds[table[b][:whole], h, i].astype(np.float64) for i in (0, 1))
            for t in range(at, at + n):
                rows = q[t, h * group:(h + 1) * group]
                total = high @ np.where(rows > 0, rows, 0).sum(0) + low @ np.where(rows < 0, rows, 0).sum(0)
                total[always] = np.inf
                best = np.argsort(-total, kind="stable")[:case["pick"]]
                out[t, h, :len(best)] = np.sort(best)
        at += n
    return torch.from_numpy(out)


def _exact_pages(case, s):
    cached, new = _lengths(case)
    if sum(new) * case["kv_heads"] > 6000:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    chosen, page, dim = s["chosen"].cpu().numpy(), case["page"], case["dim"]
    group, table, begin = case["q_heads"] // case["kv_heads"], s["table"].tolist(), 0
    for b, (c, n) in enumerate(zip(cached, new)):
        rest = c // page * page
        sees = _sees(case, b, c - rest, n) if n else None
        for t in range(begin, begin + n):
            mine = torch.nonzero(sees[t - begin])[:, 0] + rest
            for h in range(case["kv_heads"]):
                j = torch.from_numpy(chosen[t, h][chosen[t, h] >= 0]).long()
                row = torch.cat(((j[:, None] * page + torch.arange(page)).flatten(), mine))
                where = torch.tensor(table[b])[row // page].cuda(), (row % page).cuda()
                k, v = (s["kv"][0, where[0], i, h, where[1]].double() for i in (0, 1))
                score = k @ s["q"][t, h * group:(h + 1) * group].double().T / math.sqrt(dim)
                out[t, h * group:(h + 1) * group] = torch.softmax(score, 0).T @ v
        begin += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _exact_shared, "bounds": _exact_bounds, "select": _exact_select, "pages": _exact_pages}[case["op"]](case, s)
