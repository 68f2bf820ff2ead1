"""An attention layer in speculative decoding: prompt, draft trees, verification, acceptance.

    python examples/tree_decode.py [--type q8_0|f16] [--steps N] [--nodes T]

Per step and layer, on one stream and without a host synchronisation between the calls:
  q|k|v = W_qkv . q8_0(x)       mq_matvec_q4K_q8_0 (up to 8 tokens) or mq_mmq_q4K_q8_0
  kv_append                     norms and rotation; q as f16, K and V into the cache's pages
  attn_tree                     every node against its context and its ancestors -> q8_0
  y = W_o . attention           the projection reads the q8_0 output as it is
  kv_accept                     the accepted path's nodes move up behind the context
A prompt goes the same way, as chains of up to 64 tokens.  Random weights and inputs; the accepted path is the one
whose outputs' first value is largest at every branch, in place of a sampler.
"""
import argparse
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Layer:
    def __init__(self, mq, synth, hidden=1024, heads=8, kv_heads=2, head_dim=128, seed=11):
        import torch
        self.mq, self.H, self.heads, self.kv, self.D = mq, hidden, heads, kv_heads, head_dim
        self.rows = (heads + 2 * kv_heads) * head_dim
        self.W_qkv = torch.from_numpy(synth.q4K_matrix(self.rows, hidden, seed)).cuda()
        self.W_o = torch.from_numpy(synth.q4K_matrix(hidden, heads * head_dim, seed + 1)).cuda()
        rng = np.random.default_rng(seed)
        self.q_norm, self.k_norm = (torch.from_numpy(rng.uniform(0.5, 1.5, head_dim).astype(np.float32)).cuda()
                                    for _ in range(2))
        self.inv_freq = torch.from_numpy((1e6 ** (-np.arange(0, head_dim, 2) / head_dim)).astype(np.float32)).cuda()

    def project(self, W, rows, K, **act):
        n = next(iter(act.values())).shape[0]
        if n <= 8:
            return self.mq.matvec_q4K_q8_0(W, rows, K, **act)[0]
        return self.mq.mmq_q4K_q8_0(W, rows, K, **act)[0]

    def forward(self, cache, x, pos, seq, slot, tok_start, ctx, mask, max_len, workspace):
        """x fp32 [n, hidden], n <= 64 -> (y fp32 [n, hidden], q f16, attention's q8_0 columns)."""
        mq = self.mq
        qkv = self.project(self.W_qkv, self.rows, self.H, x=x)
        q = mq.kv_append(cache, qkv, pos, seq, slot, self.heads, inv_freq=self.inv_freq, q_norm=self.q_norm,
                         k_norm=self.k_norm)
        att = mq.attn_tree(cache, q, tok_start, ctx, mask=mask, max_len=max_len, out_type="q8_0", workspace=workspace)
        return self.project(self.W_o, self.H, self.heads * self.D, xq=att), q, att


def draft_tree(rng, T):
    """Parents (-1: the context's last token), depths and masks (bit j: node j is the node or its ancestor)."""
    parent = [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, T)]
    depth, mask = [], []
    for i, p in enumerate(parent):
        depth.append(0 if p < 0 else depth[p] + 1)
        mask.append((1 << i) | (0 if p < 0 else mask[p]))
    return parent, depth, mask


def pick_path(parent, score):
    path = [0]
    while True:
        next_ = [i for i, p in enumerate(parent) if p == path[-1]]
        if not next_:
            return path
        path.append(max(next_, key=lambda i: score[i]))


def run(mq, synth, ctype="q8_0", steps=4, nodes=12, prompts=(150, 37), seed=5, on_step=None):
    """Returns (cache, layer, context lengths, per sequence the accepted tokens' inputs).

    on_step(cache, layer, tree, q, att) is called after each verification, before the acceptance."""
    import torch
    rng = np.random.default_rng(seed)
    layer = Layer(mq, synth)
    S, most = len(prompts), max(prompts) + steps * nodes + nodes
    per = -(-most // mq.MQ_KV_PAGE_TOKENS)
    table = torch.from_numpy(rng.permutation(S * per).reshape(S, per).astype(np.int32)).cuda()
    cache = mq.KVCache.alloc(S * per, table, ctype, layer.kv, layer.D)
    work = mq.attn_workspace(cache, layer.heads)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()

    def feed(x, chunks, masks):
        """chunks: per sequence (context, depths) of its tokens in x."""
        start = np.concatenate([[0], np.cumsum([len(d) for _, d in chunks])])
        pos = [c + d for c, ds in chunks for d in ds]
        seq = [s for s, (_, ds) in enumerate(chunks) for _ in ds]
        slot = [c + i for c, ds in chunks for i in range(len(ds))]
        ctx = i32([c for c, _ in chunks])
        m = None
        if masks is not None:
            m = torch.from_numpy(np.array([b for s in masks for b in s], np.uint64).view(np.int64)).cuda()
        out = layer.forward(cache, torch.from_numpy(x).cuda(), i32(pos), i32(seq), i32(slot), i32(start), ctx, m, most, work)
        return out, start, ctx

    tokens = [rng.standard_normal((n, layer.H)).astype(np.float32) for n in prompts]
    for s in range(S):  # prompts in chains; the other sequences have no tokens meanwhile
        for c in range(0, prompts[s], 64):
            n = min(64, prompts[s] - c)
            feed(tokens[s][c:c + n], [(c, list(range(n))) if i == s else (0, []) for i in range(S)], None)
    length = list(prompts)
    for _ in range(steps):
        trees = [draft_tree(rng, nodes) for _ in range(S)]
        x = rng.standard_normal((S * nodes, layer.H)).astype(np.float32)
        (y, q, att), start, ctx = feed(x, [(length[s], trees[s][1]) for s in range(S)], [t[2] for t in trees])
        if on_step:
            on_step(cache, layer, (list(length), start, [t[2] for t in trees]), q, att)
        score = y[:, 0].cpu().numpy()  # the sampler's place: the host learns the accepted paths here
        paths = [pick_path(trees[s][0], score[start[s]:start[s + 1]]) for s in range(S)]
        padded = np.zeros((S, nodes), np.int32)
        for s, p in enumerate(paths):
            padded[s, :len(p)] = p
        mq.kv_accept(cache, ctx, i32(padded), i32([len(p) for p in paths]))
        for s, p in enumerate(paths):
            tokens[s] = np.concatenate([tokens[s], x[start[s]:start[s + 1]][p]])
            length[s] += len(p)
    return cache, layer, length, tokens


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--type", default="q8_0", choices=["q8_0", "f16"])
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--nodes", type=int, default=12)
    a = ap.parse_args()
    import torch
    from quantized_decode_matvec_gb300 import mq, synth
    mq.init(0)
    cache, layer, length, tokens = run(mq, synth, a.type, a.steps, a.nodes)
    seq = torch.zeros(length[0], dtype=torch.int32, device="cuda")
    slot = torch.arange(length[0], dtype=torch.int32, device="cuda")
    k, v = mq.kv_read(cache, seq, slot)
    torch.cuda.synchronize()
    assert mq.mq_read_device_status(0) == 0
    print(f"{a.steps} steps of {a.nodes} nodes: context lengths {length}; |k| {k.float().abs().mean():.4f}, "
          f"|v| {v.float().abs().mean():.4f}")


if __name__ == "__main__":
    main()
