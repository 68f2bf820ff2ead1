"""Several answers to one prompt, drafted as trees: fork, shared-prefix attention, verification, compaction.

    python examples/shared_decode.py [--type q8_0|f16] [--answers N] [--steps N] [--nodes T]

The prompt is written once; every answer forks from it (full pages shared, the begun page's tokens copied).  Per step,
for all answers together and on one stream:
  kv_grow                       pages for the trees' nodes
  q|k|v, kv_append              as in examples/tree_decode.py, whose layer this uses
  attn_shared                   the prompt's pages attended once for all answers -> q8_0
  o and head projections        logits of every node
  softmax, verify_tree          the target's probabilities, each tree's accepted path and the token behind it
  kv_accept, kv_free            the path's nodes move up, pages behind them are given back
At the end every other answer is given up and the pages are moved to the front of the pool.  Random weights; a node's
drafted tokens are drawn from the distribution of the token above it in a table, in place of a draft model.
"""
import argparse
import importlib.util
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def tree_decode():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "tree_decode.py")
    spec = importlib.util.spec_from_file_location("tree_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Decoder:
    def __init__(self, mq, synth, ctype, answers, prompt, steps, nodes, vocab=2048, seed=3):
        import torch
        self.mq, self.td, self.vocab, self.nodes, self.answers = mq, tree_decode(), vocab, nodes, answers
        self.rng = np.random.default_rng(seed)
        self.layer = self.td.Layer(mq, synth, seed=seed)
        self.head = torch.from_numpy(synth.q4K_matrix(vocab, self.layer.H, seed + 9)).cuda()
        self.embedding = torch.randn((vocab, self.layer.H), generator=torch.Generator().manual_seed(seed)).cuda()
        # the draft's distribution behind each token
        z = torch.randn((vocab, vocab), generator=torch.Generator().manual_seed(seed + 1)).cuda() * 2.0
        self.draft = mq.softmax(z)
        most = prompt + (steps + 1) * nodes + nodes
        per = -(-most // mq.MQ_KV_PAGE_TOKENS)
        S = answers + 1  # sequence 0 is the prompt
        pages = -(-prompt // mq.MQ_KV_PAGE_TOKENS) + answers * (per - prompt // mq.MQ_KV_PAGE_TOKENS) + 2
        table = torch.zeros((S, per), dtype=torch.int32, device="cuda")
        self.cache = mq.KVCache.alloc(pages, table, ctype, self.layer.kv, self.layer.D)
        self.pool = mq.KVPool.alloc(self.cache)
        self.most = per * mq.MQ_KV_PAGE_TOKENS
        self.work = mq.attn_shared_workspace(self.cache, self.layer.heads, max(64, answers * nodes), 1)
        self.length = [0] * S
        self.tokens = [[] for _ in range(S)]
        self.last = [0] * S

    def i32(self, a):
        import torch
        return torch.from_numpy(np.asarray(a, np.int32)).cuda()

    def forward(self, new, depths, masks, shared_pages):
        """new: per sequence its tokens' ids; the trees' depths and masks; returns (y, q, attention, tok_start, ctx)."""
        import torch
        mq, layer = self.mq, self.layer
        start = np.concatenate([[0], np.cumsum([len(t) for t in new])])
        ids = [t for s in new for t in s]
        ctx = self.i32(self.length)
        mq.kv_grow(self.cache, self.pool, self.i32([c + len(t) for c, t in zip(self.length, new)]))
        x = self.embedding[torch.tensor(ids, device="cuda")]
        qkv = layer.project(layer.W_qkv, layer.rows, layer.H, x=x)
        q = mq.kv_append(self.cache, qkv, self.i32([c + d for c, ds in zip(self.length, depths) for d in ds]),
                         self.i32([s for s, t in enumerate(new) for _ in t]),
                         self.i32([c + i for c, t in zip(self.length, new) for i in range(len(t))]), layer.heads,
                         inv_freq=layer.inv_freq, q_norm=layer.q_norm, k_norm=layer.k_norm)
        m = torch.from_numpy(np.array([b for s in masks for b in s], np.uint64).view(np.int64)).cuda()
        tok_start = self.i32(start)
        # sequence 0 is in no group; all answers share the prompt's full pages
        att = mq.attn_shared(self.cache, q, tok_start, ctx, self.i32([1, self.answers + 1]), self.i32([shared_pages]), mask=m,
                             max_len=self.most, max_tokens=max(1, max(len(t) for t in new)), out_type="q8_0",
                             workspace=self.work)
        return layer.project(layer.W_o, layer.H, layer.heads * layer.D, xq=att), q, att, start, ctx

    def prompt(self, ids):
        for c in range(0, len(ids), 64):
            part = ids[c:c + 64]
            chain = [(2 << i) - 1 for i in range(len(part))]
            none = [[] for _ in range(self.answers)]
            self.forward([part] + none, [list(range(len(part)))] + none, [chain] + none, 0)
            self.length[0] += len(part)
        self.tokens[0] = list(ids)

    def fork(self):
        n = self.answers
        self.mq.kv_fork(self.cache, self.pool, self.i32([0] * n), self.i32(range(1, n + 1)), self.i32([self.length[0]] * n))
        for s in range(1, n + 1):
            self.length[s], self.tokens[s], self.last[s] = self.length[0], list(self.tokens[0]), s

    def step(self, live, on_step=None):
        """One tree per live answer; the others stay as they are."""
        import torch
        mq, T = self.mq, self.nodes
        trees = {s: self.td.draft_tree(self.rng, T) for s in live}
        S = self.answers + 1
        u = self.rng.random((S, T), dtype=np.float32)
        new = [[] for _ in range(S)]
        for s in live:  # a node's token is drawn from the draft's row of the token above it
            parent = trees[s][0]
            new[s] = [self.last[s]]
            for i in range(1, T):
                row = self.draft[new[s][parent[i]]].double().cumsum(0)
                new[s].append(min(self.vocab - 1, int(torch.searchsorted(row, self.rng.random() * float(row[-1])))))
        depths = [trees[s][1] if s in trees else [] for s in range(S)]
        masks = [trees[s][2] if s in trees else [] for s in range(S)]
        pages = self.length[0] // mq.MQ_KV_PAGE_TOKENS
        y, q, att, start, ctx = self.forward(new, depths, masks, pages)
        logits = self.layer.project(self.head, self.vocab, self.layer.H, x=y / y.abs().amax(-1, keepdim=True))
        target = mq.softmax(logits, scale=float(6.0 / logits.abs().amax()))
        ids = torch.tensor([t for s in new for t in s], device="cuda")
        parent = [max(p, 0) for s in range(S) if s in trees for p in trees[s][0]]
        path, n_path, last = mq.verify_tree(target, self.i32(start), ids.int(), self.i32(parent),
                                            u=torch.from_numpy(np.concatenate([u[s] for s in live])).cuda(),
                                            draft=self.draft[ids], path_ld=T)
        if on_step:
            on_step(self, dict(start=start, ctx=list(self.length), masks=masks, q=q, att=att, target=target, ids=ids,
                               parent=parent, path=path, n_path=n_path, last=last, u=u))
        mq.kv_accept(self.cache, ctx, path, n_path)
        got, paths, last = n_path.tolist(), path.tolist(), last.tolist()  # the host learns what was accepted
        for s in live:
            self.tokens[s] += [new[s][i] for i in paths[s][:got[s]]]
            self.length[s] += got[s]
            self.last[s] = last[s]
        P = mq.MQ_KV_PAGE_TOKENS
        mq.kv_free(self.cache, self.pool, self.i32(live), self.i32([-(-self.length[s] // P) for s in live]))
        return sum(got[s] for s in live)

    def drop(self, gone):
        self.mq.kv_free(self.cache, self.pool, self.i32(gone))
        self.mq.kv_compact(self.cache, self.pool)
        for s in gone:
            self.length[s] = 0


def run(mq, synth, ctype="q8_0", answers=5, steps=4, nodes=6, prompt=150, on_step=None):
    d = Decoder(mq, synth, ctype, answers, prompt, steps, nodes)
    d.prompt(d.rng.integers(0, d.vocab, prompt).tolist())
    d.fork()
    live = list(range(1, answers + 1))
    accepted = 0
    for _ in range(steps):
        accepted += d.step(live, on_step)
    gone = live[1::2]  # these have no tokens from now on, so the group may go on naming them
    d.drop(gone)
    live = live[::2]
    accepted += d.step(live, on_step)
    return d, live, accepted


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--type", default="q8_0", choices=["q8_0", "f16"])
    ap.add_argument("--answers", type=int, default=5)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--nodes", type=int, default=6)
    a = ap.parse_args()
    import torch
    from quantized_decode_matvec_gb300 import mq, synth
    mq.init(0)
    d, live, accepted = run(mq, synth, a.type, a.answers, a.steps, a.nodes)
    torch.cuda.synchronize()
    assert mq.mq_read_device_status(0) == 0
    used = d.cache.struct.n_pages - int(d.pool.n_free)
    print(f"{a.steps + 1} steps: {accepted} tokens accepted, {used} pages in use, lengths {[d.length[s] for s in live]}")


if __name__ == "__main__":
    main()
