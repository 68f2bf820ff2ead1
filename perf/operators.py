"""Cases for the key/value cache and the tree attention of the decode step.

Four operators stand between the q|k|v projection and the o projection:

* append: per-head norms of queries and keys, the position rotation and the
  write of keys and values into a paged cache (f16, or q8_0 codes);
* read: cached keys and values back as f16;
* accept: the accepted path of a verified tree moved to the front of the
  tree's slots;
* attention: every node of a tree of drafted tokens over its sequence's
  cache (a tree of one node is plain decoding).

The plain form computes them with elementary torch operations in 32 bits; the
cache's bytes are laid out as the library documents them (64-token pages, one
block per page and key/value head: K, V, then for q8_0 the scales of K and of
V; 16-byte chunks of a row permuted by the row number).  An element of a q8_0
cache stands for f16(scale * code).
"""
import math

import numpy as np
import torch

own = False

PAGE = 64  # tokens per page
EPS = 1e-6


# ---- cases ------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token of the 7B-class step (28 query heads, 4 key/value heads of 128): launch latency
        dict(name="append_one", op="append", seqs=1, lo=4095, hi=4095, tokens=1, heads=28, kv=4, dim=128, type="q8_0",
             norm=True, interleaved=False, rot=128),
        # a few sequences continued by ragged drafts, small heads, f16 cache, adjacent pairs, part of the head rotated
        dict(name="append_ragged_f16", op="append", seqs=5, lo=100, hi=901, tokens=37, heads=16, kv=8, dim=64, type="f16",
             norm=False, interleaved=True, rot=32),
        # a 2048-token prompt of the 7B-class step written at once (the prefill workload's length)
        dict(name="append_prompt", op="append", seqs=1, lo=0, hi=0, tokens=2048, heads=28, kv=4, dim=128, type="q8_0",
             norm=True, interleaved=False, rot=128),
        # three short sequences read back, e.g. to hand them to another engine
        dict(name="read_short_f16", op="read", seqs=3, lo=45, hi=301, heads=16, kv=8, dim=64, type="f16"),
        # one long context read back whole
        dict(name="read_long", op="read", seqs=1, lo=32768, hi=32768, heads=28, kv=4, dim=128, type="q8_0"),
        # one user: the accepted path of a 16-node tree
        dict(name="accept_one", op="accept", seqs=1, lo=1000, hi=1000, tokens=16, path=5, heads=28, kv=4, dim=128,
             type="q8_0"),
        # a batch of users with the largest trees
        dict(name="accept_batch_f16", op="accept", seqs=64, lo=77, hi=1900, tokens=64, path=11, heads=32, kv=8, dim=128,
             type="f16"),
        # one user, one token, a short context: latency
        dict(name="decode_one", op="attn", seqs=1, lo=1000, hi=1000, tokens=1, heads=28, kv=4, dim=128, type="q8_0",
             out="f16", chain=True),
        # a batch of 64 users at very different lengths, the result in the o projection's own input format
        dict(name="decode_batch", op="attn", seqs=64, lo=128, hi=8191, tokens=1, heads=28, kv=4, dim=128, type="q8_0",
             out="q8_0", chain=True),
        # one user at the library's longest row length, f16 cache: one head pair's work split over the whole chip
        dict(name="decode_long_f16", op="attn", seqs=1, lo=131071, hi=131071, tokens=1, heads=28, kv=4, dim=128, type="f16",
             out="f16", chain=True),
        # a few users with small ragged trees, small heads
        dict(name="tree_ragged_f16", op="attn", seqs=7, lo=0, hi=2000, tokens=13, heads=16, kv=8, dim=64, type="f16",
             out="f16", chain=False),
        # four users with the largest trees over long contexts: a real contraction
        dict(name="tree_large", op="attn", seqs=4, lo=8190, hi=32700, tokens=64, heads=28, kv=4, dim=128, type="q8_0",
             out="f16", chain=False),
    ]


def draw(rng):
    def log(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n + 1 if n == 3072 else n

    heads, kv, dim = rng.choice([(28, 4, 128), (16, 8, 64), (32, 8, 128), (12, 12, 64), (8, 1, 128), (10, 2, 64)])
    c = dict(op=rng.choice(["append", "read", "accept", "attn", "attn", "attn"]), heads=heads, kv=kv, dim=dim,
             type=rng.choice(["q8_0", "f16"]))
    c["seqs"] = log(1, 64)
    if c["op"] == "append":
        c["tokens"] = log(1, max(1, 2048 // c["seqs"]))
        c["lo"], c["norm"], c["interleaved"] = log(1, 8000) - 1, rng.random() < 0.5, rng.random() < 0.5
        c["hi"] = c["lo"] + log(1, 500) - 1
        c["rot"] = rng.choice([dim, dim, dim // 2, 0])
    elif c["op"] == "read":
        c["hi"] = log(16, 32768 // c["seqs"])
        c["lo"] = rng.randint(1, c["hi"])
    elif c["op"] == "accept":
        c["hi"] = log(1, 2000)
        c["lo"], c["tokens"] = rng.randint(0, c["hi"]), rng.randint(1, 64)
        c["path"] = rng.randint(1, min(12, c["tokens"]))
    else:
        c["tokens"], c["chain"] = rng.choice([1, log(1, 64), log(1, 64)]), rng.random() < 0.3
        # all sequences at the longest: at most the bytes of decode_batch and the contraction of tree_large
        most = min(131071, 2.9e8 / token_bytes(c) / c["seqs"], 5.5e10 / (4 * c["seqs"] * c["tokens"] * heads * dim))
        c["hi"] = log(16, int(most) - c["tokens"])
        c["lo"], c["out"] = rng.randint(0, c["hi"]), rng.choice(["f16", "f16", "q8_0"])
    return c


def token_bytes(case):
    """A token's bytes in the cache: keys and values of every head."""
    D = case["dim"]
    return 2 * case["kv"] * (D * 2 if case["type"] == "f16" else D + D // 16)


def lengths(case):
    """Context length and number of new tokens of each sequence: spread over the case's range, the same for every seed."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    at = [(i * 0.6180339887) % 1.0 for i in range(n)]
    ctx = [lo + int(round((hi - lo) * a)) for a in at]
    most = case.get("tokens", 0)
    # the first sequence brings the case's number of tokens, others of a ragged case fewer
    even = case["op"] == "attn" and case["chain"]
    new = [most if even or i % 3 == 0 else max(1, int(most * (1.0 - 0.8 * a))) if most else 0 for i, a in enumerate(at)]
    return ctx, new


def paths(case):
    """Accepted nodes of each sequence's tree (accept): increasing node numbers."""
    _, new = lengths(case)
    got = []
    for i, t in enumerate(new):
        k = min(t, max(1, case["path"] - i % 4))
        got.append([min(t - 1, int((j + 1) * t / k) - 1) if j else 0 for j in range(k)])
    return got


# ---- the cache's bytes ------------------------------------------------------------------------------
def layout(case):
    """Byte offsets within a block, for every token of a page and every element of a head: of K's element (V's
    follows at voff), and of K's scale; and the block's bytes."""
    D, row = case["dim"], torch.arange(PAGE, device="cuda")[:, None]
    d = torch.arange(case["dim"], device="cuda")[None, :]
    if case["type"] == "f16":
        at = (d // 64) * (PAGE * 128) + row * 128 + (((d % 64) // 8) ^ (row % 8)) * 16 + (d % 8) * 2
        return at, PAGE * D * 2, None, PAGE * D * 4
    swap = row % 8 if D == 128 else (row // 2) % 4
    at = row * D + ((d // 16) ^ swap) * 16 + d % 16
    b = torch.arange(D // 32, device="cuda")[None, :]
    return at, PAGE * D, 2 * PAGE * D + (row * (D // 32) + b) * 2, PAGE * (2 * D + D // 8)


def quantise(x):
    """fp32 [..., D] -> q8_0 codes and f16 scales [..., D/32]."""
    v = x.reshape(*x.shape[:-1], -1, 32)
    d = v.abs().amax(-1, keepdim=True) / 127.0
    q = v / torch.where(d == 0, torch.ones_like(d), d)
    q = torch.trunc(q + torch.copysign(torch.full_like(q, 0.5), q)).clamp(-127, 127)
    return q.reshape(x.shape), d.squeeze(-1).half()


def put(pages, case, page, head, at_row, x, is_v):
    """Writes fp32 rows x [n, D] at (page, head, row of the page) [n] of pages [n_pages, kv, block] in the cache's type."""
    at, voff, sc, _ = layout(case)
    soff = PAGE * (case["dim"] // 32) * 2
    if case["type"] == "f16":
        b = x.half().contiguous().view(torch.uint8).reshape(*x.shape, 2)
        where = (at[at_row] + (voff if is_v else 0))[..., None] + torch.arange(2, device=x.device)
        pages[page[:, None, None], head[:, None, None], where] = b
        return
    q, d = quantise(x)
    pages[page[:, None], head[:, None], at[at_row] + (voff if is_v else 0)] = (q + 128).to(torch.uint8)
    b = d.contiguous().view(torch.uint8).reshape(*d.shape, 2)
    where = (sc[at_row] + (soff if is_v else 0))[..., None] + torch.arange(2, device=x.device)
    pages[page[:, None, None], head[:, None, None], where] = b


def get(blocks, case, is_v):
    """The f16 values of every token of whole blocks: uint8 [..., block] -> f16 [..., 64, D]."""
    at, voff, sc, _ = layout(case)
    soff = PAGE * (case["dim"] // 32) * 2
    if case["type"] == "f16":
        w = blocks.view(torch.float16)
        return w[..., (at + (voff if is_v else 0)) // 2]
    q = blocks[..., at + (voff if is_v else 0)].to(torch.int16) - 128
    d = blocks.view(torch.float16)[..., (sc + (soff if is_v else 0)) // 2]
    return (q.float() * d.float().repeat_interleave(32, -1)).half()


def fill(case, gen, ctx, new):
    """A page pool and table that hold ctx + new tokens of every sequence, the pages in random order."""
    need = [max(1, -(-(c + t) // PAGE)) for c, t in zip(ctx, new)]
    total, kv, D = sum(need) + 3, case["kv"], case["dim"]
    at, voff, sc, size = layout(case)
    pages = torch.empty((total, kv, size), dtype=torch.uint8, device="cuda")
    offset = torch.zeros((kv, 1, D), device="cuda")  # keys have a few channels far from zero
    offset[:, :, torch.randint(0, D, (3,), generator=gen, device="cuda")] = 3.0
    for first in range(0, total, 256):
        n = min(256, total - first)
        part = pages[first:first + n]
        for is_v in (False, True):
            x = torch.randn((n, kv, PAGE, D), generator=gen, device="cuda")
            x = x if is_v else x + offset
            if case["type"] == "f16":
                part.view(torch.float16)[..., (at + (voff if is_v else 0)) // 2] = x.half()
            else:
                q, d = quantise(x)
                part[..., at + (voff if is_v else 0)] = (q + 128).to(torch.uint8)
                part.view(torch.float16)[..., (sc + (PAGE * (D // 32) * 2 if is_v else 0)) // 2] = d
    order = torch.randperm(total, generator=gen, device="cuda").int().cpu()
    table = torch.zeros((case["seqs"], max(need) + 1), dtype=torch.int32)
    done = 0
    for i, n in enumerate(need):
        table[i, :n] = order[done:done + n]
        done += n
    return pages, table.to("cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ctx, new = lengths(case)
    s = dict(case=case)
    s["pages"], s["table"] = fill(case, gen, ctx, new)
    Hq, Hkv, D = case["heads"], case["kv"], case["dim"]
    if case["op"] == "read":
        s["seq"] = ints([i for i, c in enumerate(ctx) for _ in range(c)])
        s["slot"] = ints([j for c in ctx for j in range(c)])
    elif case["op"] == "append":
        s["seq"] = ints([i for i, t in enumerate(new) for _ in range(t)])
        s["slot"] = ints([c + j for c, t in zip(ctx, new) for j in range(t)])
        s["pos"] = s["slot"].clone()
        s["qkv"] = torch.randn((sum(new), (Hq + 2 * Hkv) * D), generator=gen, device="cuda") * 1.7
        s["q_norm"] = 1 + 0.2 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None
        s["k_norm"] = 1 + 0.2 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None
        R = case["rot"]
        s["inv_freq"] = (1e6 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / max(R, 1))).float() if R else None
    elif case["op"] == "accept":
        got = paths(case)
        s["ctx"], s["n_path"] = ints(ctx), ints([len(p) for p in got])
        s["path"] = ints([p + [0] * (case["path"] - len(p)) for p in got])
        s["seq"] = ints([i for i, p in enumerate(got) for _ in p])
        s["slot"] = ints([ctx[i] + j for i, p in enumerate(got) for j in range(len(p))])
        s["from"] = ints([ctx[i] + j for i, p in enumerate(got) for j in p])
    else:
        s["q"] = torch.randn((sum(new), Hq * D), generator=gen, device="cuda").half()
        s["ctx"] = ints(ctx)
        s["start"] = ints([0] + list(np.cumsum(new)))
        s["mask"], s["scale"] = None, D ** -0.5
        if not case["chain"]:
            rng = np.random.default_rng(seed)
            bits = []
            for t in new:  # each node's parent is a random earlier one; it sees its ancestors and itself
                tree = []
                for i in range(t):
                    tree.append((tree[rng.integers(0, i)] if i else 0) | (1 << i))
                bits += [b - (1 << 64) if b >> 63 else b for b in tree]
            s["mask"] = torch.tensor(bits, dtype=torch.int64, device="cuda")
        s["longest"], s["most"] = max(c + t for c, t in zip(ctx, new)), max(new)
        # the same plan of rows that a scheduler keeps beside its batch: sequence of each token, its place in the tree
        s["seq"] = ints([i for i, t in enumerate(new) for _ in range(t)])
        s["node"] = ints([j for t in new for j in range(t)])
    return s


# ---- the passes --------------------------------------------------------------------------------------
def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(s):
    from quantized_decode_matvec_gb300 import mq
    case = s["case"]
    if "cache" not in s:  # the handle that a program keeps
        mq.init()
        s["cache"] = mq.KVCache(s["pages"], s["table"], case["type"], case["kv"], case["dim"])
        if case["op"] == "attn":
            s["work"] = mq.attn_workspace(s["cache"], case["heads"], s["most"])
    cache = s["cache"]
    if case["op"] == "append":
        q = mq.kv_append(cache, s["qkv"], s["pos"], s["seq"], s["slot"], case["heads"], inv_freq=s["inv_freq"],
                         interleaved=case["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return (q,) + mq.kv_read(cache, s["seq"], s["slot"])
    if case["op"] == "read":
        return mq.kv_read(cache, s["seq"], s["slot"])
    if case["op"] == "accept":
        mq.kv_accept(cache, s["ctx"], s["path"], s["n_path"])
        return mq.kv_read(cache, s["seq"], s["slot"])
    out = mq.attn_tree(cache, s["q"], s["start"], s["ctx"], mask=s["mask"], scale=s["scale"], max_len=s["longest"],
                       max_tokens=s["most"], out_type=case["out"], workspace=s["work"])
    if case["out"] == "q8_0":  # 34-byte blocks: f16 scale, 32 codes; the values they stand for
        n = out.shape[0]
        return out.view(torch.int8).view(n, -1, 34)[..., 2:] * out.view(torch.float16).view(n, -1, 17)[..., :1]
    return out


def where(s, slot):
    """Page and row of the page of (sequence, slot) pairs."""
    return s["table"][s["seq"].long(), slot.long() // PAGE].long(), slot.long() % PAGE


def read_plain(s):
    case = s["case"]
    at, voff, sc, _ = layout(case)
    soff = PAGE * (case["dim"] // 32) * 2
    page, row = where(s, s["slot"])
    n, kv = page.numel(), case["kv"]
    p, h = page[:, None, None], torch.arange(kv, device="cuda")[None, :, None]
    half = s["pages"].view(torch.float16)
    if case["type"] == "f16":
        a = (at[row] // 2)[:, None, :]
        return half[p, h, a], half[p, h, a + voff // 2]
    a, b = at[row][:, None, :], (sc[row] // 2)[:, None, :]
    k = (s["pages"][p, h, a].float() - 128) * half[p, h, b].float().repeat_interleave(32, -1)
    v = (s["pages"][p, h, a + voff].float() - 128) * half[p, h, b + soff // 2].float().repeat_interleave(32, -1)
    return k.half(), v.half()


def normed(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def rotated(x, angle, rot, interleaved):
    """x [n, heads, D] rotated by angle [n, rot/2] in its first rot elements."""
    c, s = angle.cos()[:, None, :], angle.sin()[:, None, :]
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)
    a, b = r[..., :rot // 2], r[..., rot // 2:]
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1)


def run_plain(s):
    case = s["case"]
    Hq, Hkv, D = case["heads"], case["kv"], case["dim"]
    if case["op"] == "read":
        return read_plain(s)
    if case["op"] == "accept":
        page, row = where(s, s["from"])
        at, voff, sc, _ = layout(case)
        w = [at, at + voff] if sc is None else [at, at + voff, sc, sc + PAGE * (D // 32) * 2]
        w = torch.cat([x if x is at and sc is not None or x.shape[1] == D and sc is not None
                       else torch.stack([x, x + 1], -1).flatten(1) for x in w], 1)
        h = torch.arange(Hkv, device="cuda")[None, :, None]
        moved = s["pages"][page[:, None, None], h, w[row][:, None, :]]
        page, row = where(s, s["slot"])
        s["pages"][page[:, None, None], h, w[row][:, None, :]] = moved
        return read_plain(s)
    if case["op"] == "append":
        n = s["qkv"].shape[0]
        x = s["qkv"].view(n, Hq + 2 * Hkv, D)
        q, k, v = normed(x[:, :Hq], s["q_norm"]), normed(x[:, Hq:Hq + Hkv], s["k_norm"]), x[:, Hq + Hkv:]
        if case["rot"]:
            angle = s["pos"].float()[:, None] * s["inv_freq"]
            q, k = (rotated(t, angle, case["rot"], case["interleaved"]) for t in (q, k))
        page, row = where(s, s["slot"])
        page, row = page.repeat_interleave(Hkv), row.repeat_interleave(Hkv)
        head = torch.arange(Hkv, device="cuda").repeat(n)
        put(s["pages"], case, page, head, row, k.reshape(-1, D), False)
        put(s["pages"], case, page, head, row, v.reshape(-1, D), True)
        return (q.reshape(n, -1).half(),) + read_plain(s)
    # attention: every sequence's cache padded to the longest, every tree to the largest
    B, G, T, L = case["seqs"], Hq // Hkv, s["most"], s["longest"]
    used = s["table"][:, :-(-L // PAGE)].long()
    blocks = s["pages"][used]  # [B, pages, kv, block]
    k, v = (get(blocks, case, w).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)[:, :, :L].float() for w in (False, True))
    q = torch.zeros((B, T, Hq, D), device="cuda")
    seq, node = s["seq"].long(), s["node"].long()
    q[seq, node] = s["q"].view(-1, Hq, D).float()
    q = q.view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    score = torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, T, G, L) * s["scale"]
    j = torch.arange(L, device="cuda") - s["ctx"].long()[:, None]  # [B, L]: the node that a key is, negative: context
    seen = torch.zeros((B, T), dtype=torch.int64, device="cuda")
    seen[seq, node] = s["mask"] if s["mask"] is not None else ((2 << node) - 1)
    bit = (seen[:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    ok = (j < 0)[:, None, :] | ((j >= 0) & (j < 64))[:, None, :] & (bit == 1)
    score = score.masked_fill(~ok[:, None, :, None, :], -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    # keys past a sequence's end hold whatever its pages hold: they weigh nothing
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p.view(B, Hkv, T * G, L), v).view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq * D)
    o = o[seq, node]
    if case["out"] == "q8_0":
        c, d = quantise(o)
        return (c.view(o.shape[0], -1, 32) * d.float()[..., None]).half()
    return o.half()


# ---- what a pass cannot do without -------------------------------------------------------------------
def work(case):
    ctx, new = lengths(case)
    D, Hq, Hkv = case["dim"], case["heads"], case["kv"]
    token = token_bytes(case)
    back = 2 * Hkv * D * 2  # a token read back as f16
    if case["op"] == "read":
        return dict(bytes=sum(ctx) * (token + back), flops=sum(ctx) * 2 * Hkv * D)
    if case["op"] == "accept":
        n = sum(len(p) for p in paths(case))
        return dict(bytes=n * (3 * token + back), flops=n * 2 * Hkv * D)
    n = sum(new)
    if case["op"] == "append":
        return dict(bytes=n * ((Hq + 2 * Hkv) * D * 4 + Hq * D * 2 + 2 * token + back), flops=n * (Hq + 2 * Hkv) * D * 8)
    out = Hq * D * (2 if case["out"] == "f16" else 34 / 32)
    return dict(bytes=sum((c + t) * token for c, t in zip(ctx, new)) + n * (Hq * D * 2 + out),
                flops=sum(4 * (c + t) * t * Hq * D for c, t in zip(ctx, new)))


# ---- the definition in 64 bits -----------------------------------------------------------------------
def cached64(s, seq, slots, head):
    """Keys and values (float64, [n, D]) of one head at slots of a sequence, byte by byte from the layout."""
    case = s["case"]
    D, size = case["dim"], s["pages"].shape[-1]
    slots = torch.as_tensor(slots, device="cuda", dtype=torch.int64)
    blocks = s["pages"][s["table"][seq].long()[slots // PAGE], head].reshape(-1, size)
    r = (slots % PAGE)[:, None]
    got = []
    for is_v in (0, 1):
        if case["type"] == "f16":
            e = torch.arange(D, device="cuda")[None, :]
            byte = is_v * PAGE * D * 2 + (e >> 6) * 8192 + r * 128 + ((((e & 63) >> 3) ^ (r & 7)) << 4) + 2 * (e & 7)
            got.append(torch.gather(blocks.view(torch.float16), 1, byte >> 1).double())
        else:
            e = torch.arange(D, device="cuda")[None, :]
            turn = (r & 7) if D == 128 else (r >> 1) & 3
            code = torch.gather(blocks, 1, is_v * PAGE * D + r * D + (((e >> 4) ^ turn) << 4) + (e & 15)).double() - 128
            place = 2 * PAGE * D + is_v * PAGE * (D >> 4) + 2 * (r * (D >> 5) + (e >> 5))
            got.append((torch.gather(blocks.view(torch.float16), 1, place >> 1).double() * code).half().double())
    return got


def exact(case, seed):
    s = prepare(case, seed)
    ctx, new = lengths(case)
    D, Hq, Hkv = case["dim"], case["heads"], case["kv"]
    if case["op"] in ("read", "accept"):
        each = [list(range(c)) for c in ctx] if case["op"] == "read" else [[c + j for j in p] for c, p in zip(ctx, paths(case))]
        per = [[cached64(s, i, w, h) for h in range(Hkv)] for i, w in enumerate(each) if w]
        return tuple(torch.cat([torch.stack([x[a] for x in hs], 1) for hs in per]) for a in (0, 1))
    if case["op"] == "append":
        # the values themselves: what the cache keeps of them is rounded to its type
        x = s["qkv"].double().view(-1, Hq + 2 * Hkv, D)
        parts = [x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]]
        for a, w in ((0, s["q_norm"]), (1, s["k_norm"])):
            y = parts[a]
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + EPS) * w.double()
            if case["rot"]:
                z, half = y.clone(), case["rot"] // 2
                t = s["pos"].double()[:, None, None] * s["inv_freq"].double()
                i = torch.arange(half, device="cuda")
                one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                z[..., one] = y[..., one] * torch.cos(t) - y[..., two] * torch.sin(t)
                z[..., two] = y[..., one] * torch.sin(t) + y[..., two] * torch.cos(t)
                y = z
            parts[a] = y
        return parts[0].reshape(x.shape[0], -1), parts[1], parts[2]
    if sum(4.0 * (c + t) * t * Hq * D for c, t in zip(ctx, new)) > 4e12:
        return None
    outs, first, G = [], 0, Hq // Hkv
    for i, (c, t) in enumerate(zip(ctx, new)):
        q = s["q"][first:first + t].double().view(t, Hq, D)
        o = torch.zeros((t, Hq, D), dtype=torch.float64, device="cuda")
        see = torch.ones((t, c + t), dtype=torch.bool, device="cuda")
        for a in range(t):
            bits = int(s["mask"][first + a]) if s["mask"] is not None else (2 << a) - 1
            see[a, c:] = torch.tensor([(bits >> b) & 1 == 1 for b in range(t)], device="cuda")
        for h in range(Hkv):
            k, v = cached64(s, i, list(range(c + t)), h)
            for g in range(h * G, h * G + G):
                w = (q[:, g] @ k.T * s["scale"]).masked_fill(~see, -math.inf)
                o[:, g] = torch.softmax(w, -1) @ v
        outs.append(o.view(t, Hq * D))
        first += t
    o = torch.cat(outs)
    return o.view(o.shape[0], -1, 32) if case["out"] == "q8_0" else o
