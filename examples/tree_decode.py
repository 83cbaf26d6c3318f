"""Catalog answers over a paged cache, with the trie as the draft model.

A small model with random weights reads one shared prompt, every sequence forks
it and adds a question of its own; then all decode k catalog pointers.  The
legal continuations are known ahead, so one pass of the model takes the last
token and the trie's next nodes below it as a tree of drafts, decode_step_sparse
walks down the tree as long as the hidden state of the token that it chose is
among them, and the cache keeps the rows of that walk.

    python examples/tree_decode.py [--sequences 8] [--drafts 24]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import trie_masked_sparse_amd as tms  # noqa: E402
from synth import CONFIGS, catalog, embedding  # noqa: E402


class Model:
    """Attention blocks over the cache; the output head is the library's sparse one, tied to emb."""

    def __init__(self, emb, layers=2, q_heads=4, kv_heads=2, head_dim=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.emb, self.layers, self.q_heads, self.kv_heads, self.head_dim = emb, layers, q_heads, kv_heads, head_dim
        width = emb.shape[1]

        def weight(rows, columns):
            return (torch.randn(rows, columns, generator=g) / rows ** 0.5).to(emb)
        self.qkv = [weight(width, (q_heads + 2 * kv_heads) * head_dim) for _ in range(layers)]
        self.out = [weight(q_heads * head_dim, width) for _ in range(layers)]
        self.norm = torch.ones(head_dim).to(emb)
        self.inv_freq = (10000.0 ** (-torch.arange(0, head_dim, 2) / head_dim)).float().to(emb.device)

    def forward(self, cache, tokens, pos, start, max_new, parent=None):
        """Hidden states [T][H] of the packed new tokens, whose rows are reserved."""
        x, (hq, hkv, D) = self.emb[tokens.long()], (self.q_heads, self.kv_heads, self.head_dim)
        x = x / x.float().pow(2).mean(-1, keepdim=True).sqrt().to(x.dtype)
        for layer in range(self.layers):
            qkv = (x @ self.qkv[layer]).view(len(tokens), hq + 2 * hkv, D)
            q, out = torch.empty((2, len(tokens), hq, D), dtype=x.dtype, device=x.device)
            tms.kv_write(cache, layer, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], start, q=qkv[:, :hq], q_out=q,
                         q_weight=self.norm, k_weight=self.norm, pos=pos, inv_freq=self.inv_freq)
            tms.kv_attention(cache, layer, q, start, out, parent=parent, max_new=max_new)
            x = x + out.view(len(tokens), hq * D) @ self.out[layer]
        return x


def ints(values):
    return torch.tensor(np.asarray(values, np.int32), device="cuda")


def packed(lists):
    return [x for part in lists for x in part], np.concatenate([[0], np.cumsum([len(part) for part in lists])])


def draft_tree(csr, node, token, limit):
    """(tokens, parents, edges) of the last token and up to `limit` trie nodes
    below `node`, breadth first; edges[i]: {token: draft} of draft i."""
    tokens, parents, edges, queue = [token], [-1], [{}], [(0, node)]
    for at, n in queue:
        for e in range(csr["begin"][n], csr["begin"][n + 1]):
            if len(tokens) > limit:
                return tokens, parents, edges
            if csr["child"][e] == -2:  # stop: nothing comes after it
                continue
            edges[at][int(csr["tok"][e])] = len(tokens)
            tokens.append(int(csr["tok"][e]))
            parents.append(at)
            edges.append({})
            queue.append((len(tokens) - 1, max(int(csr["child"][e]), 0)))  # a separator leads to the root
    return tokens, parents, edges


def step(csr, node, token):
    """Node after `token`; None after stop."""
    for e in range(csr["begin"][node], csr["begin"][node + 1]):
        if csr["tok"][e] == token:
            return None if csr["child"][e] == -2 else max(int(csr["child"][e]), 0)
    raise ValueError(f"{token} is not an edge of node {node}")


def decode(trie, model, prompt, questions, k, drafts, page_tokens=16):
    """(tokens of every sequence, passes of the model)."""
    B, csr = len(questions), trie.csr()
    most = len(prompt) + max(map(len, questions)) + k * (trie.info["max_depth"] + 1) + drafts
    each = -(-most // page_tokens)
    cache = tms.PagedCache.empty(model.layers, B * each + each, model.kv_heads, page_tokens, model.head_dim, B, each,
                                 dtype=model.emb.dtype)
    state = tms.State(trie, B, k, model.emb)
    chosen = torch.empty(B, dtype=torch.int32, device="cuda")

    def run(lists, lengths, parents=None):
        tokens, start = packed(lists)
        # a draft's position is its depth in the tree
        at = []
        for s, part in enumerate(lists):
            depth = []
            for i in range(len(part)):
                depth.append(i if parents is None else 0 if parents[s][i] < 0 else depth[parents[s][i]] + 1)
            at += [lengths[s] + d for d in depth]
        tms.kv_reserve(cache, ints([len(part) for part in lists]))
        return model.forward(cache, ints(tokens), ints(at), ints(start), max(map(len, lists)),
                             None if parents is None else ints(packed(parents)[0])), start

    # the shared prompt once, in sequence 0; the others fork it
    run([prompt] + [[]] * (B - 1), [0] * B)
    tms.kv_commit(cache, ints([len(prompt)] + [0] * (B - 1)))
    tms.kv_fork(cache, ints([0] * B))
    lengths = [len(prompt)] * B
    x, start = run(questions, lengths)
    tms.kv_commit(cache, ints([len(part) for part in questions]))
    lengths = [a + len(part) for a, part in zip(lengths, questions)]

    answers, nodes, passes = [[] for _ in range(B)], [0] * B, 2
    tms.decode_step_sparse(state, x[ints(start[1:] - 1).long()].contiguous(), chosen)
    while True:
        for s, token in enumerate(chosen.tolist()):
            if nodes[s] is not None:
                answers[s].append(token)
                nodes[s] = step(csr, nodes[s], token)
        live = [s for s in range(B) if nodes[s] is not None]
        if not live:
            break
        trees = [draft_tree(csr, nodes[s], answers[s][-1], drafts) if s in live else ([], [], []) for s in range(B)]
        x, start = run([t[0] for t in trees], lengths, [t[1] for t in trees])
        passes += 1
        # down the trees, as long as every sequence's last token is among its drafts
        keep = [[0] if s in live else [] for s in range(B)]
        while True:
            rows = ints([start[s] + keep[s][-1] if keep[s] else 0 for s in range(B)])
            tms.decode_step_sparse(state, x[rows.long()].contiguous(), chosen)
            step_tokens = chosen.tolist()
            after = [trees[s][2][keep[s][-1]].get(step_tokens[s]) if nodes[s] is not None else None for s in range(B)]
            going = [s for s in live if nodes[s] is not None and step(csr, nodes[s], step_tokens[s]) is not None]
            if not going or any(after[s] is None for s in going):
                break
            for s in live:
                if nodes[s] is not None:
                    answers[s].append(step_tokens[s])
                    nodes[s] = step(csr, nodes[s], step_tokens[s])
                    if nodes[s] is not None:
                        keep[s].append(after[s])
        wide = max(map(len, keep))
        tms.kv_commit(cache, ints([len(part) for part in keep]), ints([part + [0] * (wide - len(part)) for part in keep]))
        lengths = [a + len(part) for a, part in zip(lengths, keep)]
    assert (state.status(check=True) == tms.OK).all() and cache.length.tolist() == lengths
    tms.kv_fork(cache, ints([-1] * B))  # all pages are free again
    assert not cache.refs.any()
    state.close()
    return answers, passes


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--sequences", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=24)
    args = ap.parse_args()
    c = CONFIGS["tiny"]
    rng = np.random.default_rng(1)
    trie = tms.Trie(catalog("tiny"), c.vocab, c.sep, c.stop)
    model = Model(torch.from_numpy(embedding("tiny").copy()).cuda())
    prompt = rng.integers(0, c.sep, 100).tolist()
    questions = [rng.integers(0, c.sep, int(n)).tolist() for n in rng.integers(1, 12, args.sequences)]
    plain, many = decode(trie, model, prompt, questions, c.k, 0)
    answers, passes = decode(trie, model, prompt, questions, c.k, args.drafts)
    if answers != plain:
        raise SystemExit("the answers with drafts differ from those without")
    print(f"{args.sequences} sequences, {sum(map(len, answers))} tokens: {passes} passes of the model with trees of up to "
          f"{args.drafts} drafts, {many} without, the same answers")
    trie.close()


if __name__ == "__main__":
    main()
