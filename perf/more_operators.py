"""Cases for serving several continuations of one prompt with drafted trees, over the paged key/value cache.

Five operators stand around the cache's append, read, accept and tree attention:

* attn_shared: attention of a batch whose sequences share the pages of a long prefix, which is attended once for all;
* softmax: the target's probabilities from the logits of every node;
* verify: drafted trees against those probabilities, from given random numbers: the accepted path of every sequence
  and the token behind it;
* fork: sequences that go on from a point of another one: full pages are shared, a begun page's tokens are copied;
* compact: sequences given up, and the pages that remain moved to the front of the pool.

The plain form computes them with elementary torch operations, in 32 bits, and in 64 where a sum over a vocabulary is
compared with a random number.  The cache's bytes are laid out as the library documents them.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64  # tokens per page


# ---- cases ------------------------------------------------------------------------------------------
def listed():
    return [
        # four answers to one prompt of ordinary length, one token each: latency
        dict(name="shared_small", op="attn", groups=1, each=4, prefix=1000, lo=1, hi=90, tokens=1, heads=28, kv=4, dim=128,
             type="q8_0", out="f16", chain=True),
        # 64 requests behind one long system prompt, one token each, the result in the o projection's input format
        dict(name="shared_batch", op="attn", groups=1, each=64, prefix=8192, lo=50, hi=900, tokens=1, heads=28, kv=4,
             dim=128, type="q8_0", out="q8_0", chain=True),
        # three documents of different lengths, 43 requests on each with trees of up to 7 nodes, f16 cache
        dict(name="shared_trees_f16", op="attn", groups=3, each=43, prefix=20011, lo=0, hi=700, tokens=7, heads=32, kv=8,
             dim=128, type="f16", out="f16", chain=False),
        # the nodes of one small tree, an odd vocabulary: latency
        dict(name="softmax_small", op="softmax", rows=7, vocab=50001, scale=1.25),
        # the nodes of 32 trees of 16
        dict(name="softmax_batch", op="softmax", rows=512, vocab=131072, scale=1.0),
        # one user's tree: latency
        dict(name="verify_one", op="verify", seqs=1, tokens=16, vocab=131072, mode="draft", near=0.7),
        # drafts looked up in the text so far: no distribution of their own; odd sizes, rows not aligned
        dict(name="verify_lookup", op="verify", seqs=17, tokens=7, vocab=50001, mode="lookup", near=0.0),
        # a batch of users
        dict(name="verify_batch", op="verify", seqs=64, tokens=16, vocab=131072, mode="draft", near=0.7),
        # three answers to one prompt: latency
        dict(name="fork_small", op="fork", seqs=1, each=3, lo=1000, hi=1000, kv=4, dim=128, type="q8_0"),
        # 16 prompts, eight answers each
        dict(name="fork_batch_f16", op="fork", seqs=16, each=8, lo=500, hi=9000, kv=8, dim=128, type="f16"),
        # one of five short sequences ends
        dict(name="compact_small", op="compact", seqs=5, every=5, lo=45, hi=301, kv=8, dim=64, type="f16"),
        # a quarter of a batch ends, its pages are scattered over the pool
        dict(name="compact_batch", op="compact", seqs=64, every=4, lo=500, hi=8191, kv=4, dim=128, type="q8_0"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["attn", "attn", "softmax", "verify", "verify", "fork", "compact"])
    if op == "softmax":
        rows = log(1, 512)
        return dict(op=op, rows=rows, vocab=log(1000, min(262144, 512 * 131072 // rows)), scale=rng.choice([1.0, 0.5, 1.6]))
    if op == "verify":
        c = dict(op=op, seqs=log(1, 64), tokens=rng.randint(2, 16), mode=rng.choice(["draft", "draft", "lookup", "greedy"]))
        c["vocab"] = log(1000, min(262144, 64 * 131072 // c["seqs"]))
        c["near"] = rng.choice([0.3, 0.7, 1.5]) if c["mode"] == "draft" else 0.0
        return c
    heads, kv, dim = rng.choice([(28, 4, 128), (16, 8, 64), (32, 8, 128), (12, 12, 64), (8, 1, 128), (10, 2, 64)])
    c = dict(op=op, kv=kv, dim=dim, type=rng.choice(["q8_0", "f16"]))
    if op == "attn":
        c.update(heads=heads, groups=log(1, 8), tokens=rng.choice([1, 1, log(1, 24)]), chain=rng.random() < 0.5)
        c["each"] = log(1, 128 // c["groups"])
        seqs = c["groups"] * c["each"]
        # at most the work of shared_trees_f16
        most = min(65536, 7e9 / token_bytes(c) / c["groups"] / 16, 8e10 / (4 * seqs * c["tokens"] * heads * dim))
        c["prefix"] = log(32, int(max(64, most)))
        c["hi"] = log(1, int(max(2, min(2000, most / 4))))
        c["lo"], c["out"] = rng.randint(0, c["hi"]), rng.choice(["f16", "f16", "q8_0"])
        return c
    if op == "fork":
        c.update(seqs=log(1, 16), each=rng.randint(1, 8))
        c["hi"] = log(1, 9000)
    else:
        c["seqs"] = log(2, 64)
        c.update(every=rng.randint(2, min(5, c["seqs"])))
        c["hi"] = log(16, 2.0e8 / token_bytes(c) / c["seqs"])
    c["lo"] = rng.randint(1, c["hi"])
    return c


def token_bytes(case):
    """A token's bytes in the cache: keys and values of every head."""
    D = case["dim"]
    return 2 * case["kv"] * (D * 2 if case["type"] == "f16" else D + D // 16)


def spread(n):
    return [(i * 0.6180339887) % 1.0 for i in range(n)]


def batch(case):
    """attn: every sequence's group, the groups' prefixes (tokens), the contexts and the numbers of new tokens."""
    G, each = case["groups"], case["each"]
    prefix = [max(1, int(case["prefix"] * (1.0 - 0.7 * a))) for a in spread(G)]
    group = [g for g in range(G) for _ in range(max(1, each - (g % 3)))]
    at = spread(len(group))
    ctx = [prefix[g] + case["lo"] + int(round((case["hi"] - case["lo"]) * a)) for g, a in zip(group, at)]
    new = [case["tokens"] if case["chain"] or i % 3 == 0 else max(1, int(case["tokens"] * (1.0 - 0.8 * a)))
           for i, a in enumerate(at)]
    return group, prefix, ctx, new


def lengths(case):
    """fork, compact: tokens of each sequence in the pool."""
    return [case["lo"] + int(round((case["hi"] - case["lo"]) * a)) for a in spread(case["seqs"])]


def forks(case):
    """fork: (source, tokens taken over) of every new sequence: all of a source, or up to a point before its end."""
    n = lengths(case)
    return [(s, n[s] if j % 2 == 0 else max(1, int(n[s] * a)))
            for s in range(case["seqs"]) for j, a in zip(range(case["each"]), spread(case["each"] + 1)[1:])]


def trees(case):
    """verify: parents of every tree's nodes (node 0 is the root, the token that the step before ended with)."""
    got = []
    for i in range(case["seqs"]):
        rng = np.random.default_rng(i)
        t = case["tokens"] if i % 3 == 0 else max(1, case["tokens"] - i % 5)
        got.append([0] + [int(rng.integers(max(0, j - 4), j)) for j in range(1, t)])
    return got


def depth(parents):
    d = [1]
    for p in parents[1:]:
        d.append(d[p] + 1)
    return max(d)


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


def get(blocks, case, is_v):
    """The f16 values of every token of whole blocks: uint8 [..., block] -> f16 [..., 64, D]."""
    at, voff, sc, _ = layout(case)
    soff = PAGE * (case["dim"] // 32) * 2
    if case["type"] == "f16":
        return blocks.view(torch.float16)[..., (at + (voff if is_v else 0)) // 2]
    q = blocks[..., at + (voff if is_v else 0)].to(torch.int16) - 128
    d = blocks.view(torch.float16)[..., (sc + (soff if is_v else 0)) // 2]
    return (q.float() * d.float().repeat_interleave(32, -1)).half()


def row_bytes(case, rows):
    """Byte offsets within a block of everything that its first `rows` tokens hold."""
    D = case["dim"]
    at, voff, sc, _ = layout(case)
    if case["type"] == "f16":
        a = torch.stack([at[:rows], at[:rows] + 1], -1).flatten()
        return torch.cat([a, a + voff])
    a, b = at[:rows].flatten(), torch.stack([sc[:rows], sc[:rows] + 1], -1).flatten()
    return torch.cat([a, a + voff, b, b + PAGE * (D // 32) * 2])


def new_pool(case, gen, total):
    """Pages filled with keys (a few channels far from zero) and values."""
    kv, D = case["kv"], case["dim"]
    at, voff, sc, size = layout(case)
    pages = torch.empty((total, kv, size), dtype=torch.uint8, device="cuda")
    offset = torch.zeros((kv, 1, D), device="cuda")
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
    return pages


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "softmax":
        x = torch.randn((case["rows"], case["vocab"]), generator=gen, device="cuda") * 2.5
        s["x"] = x + 6.0 * (torch.rand(x.shape, generator=gen, device="cuda") > 0.9998)
    elif case["op"] == "verify":
        prepare_verify(s, gen)
    elif case["op"] == "attn":
        prepare_attn(s, gen, seed)
    else:
        prepare_pool(s, gen)
    return s


def prepare_attn(s, gen, seed):
    case = s["case"]
    group, prefix, ctx, new = batch(case)
    Hq, D = case["heads"], case["dim"]
    shared = [p // PAGE for p in prefix]  # pages that a group's sequences have in common
    need = [-(-(c + t) // PAGE) - shared[g] for g, c, t in zip(group, ctx, new)]
    total = sum(shared) + sum(need) + 3
    s["pages"] = new_pool(case, gen, total)
    order = torch.randperm(total, generator=gen, device="cuda").int().cpu()
    table = torch.zeros((len(ctx), max(shared[g] + n for g, n in zip(group, need)) + 1), dtype=torch.int32)
    first = [sum(shared[:g]) for g in range(len(shared))]
    done = sum(shared)
    for i, (g, n) in enumerate(zip(group, need)):
        table[i, :shared[g]] = order[first[g]:first[g] + shared[g]]
        table[i, shared[g]:shared[g] + n] = order[done:done + n]
        done += n
    s["table"] = table.to("cuda")
    s["q"] = torch.randn((sum(new), Hq * D), generator=gen, device="cuda").half()
    s["ctx"], s["start"] = ints(ctx), ints([0] + list(np.cumsum(new)))
    counts = [group.count(g) for g in range(case["groups"])]
    s["grp_start"], s["grp_pages"] = ints([0] + list(np.cumsum(counts))), ints(shared)
    s["mask"], s["scale"] = None, D ** -0.5
    if not case["chain"]:
        rng = np.random.default_rng(seed)
        bits = []
        for t in new:  # each node's parent is a random earlier one; it sees its ancestors and itself
            tree = []
            for i in range(t):
                tree.append((tree[rng.integers(0, i)] if i else 0) | (1 << i))
            bits += tree
        s["mask"] = torch.tensor(bits, dtype=torch.int64, device="cuda")
    s["longest"], s["most"], s["most_pages"] = max(c + t for c, t in zip(ctx, new)), max(new), max(shared)
    # the plan of rows that a scheduler keeps beside its batch: sequence of each token, its place in the tree
    s["seq"] = ints([i for i, t in enumerate(new) for _ in range(t)])
    s["node"] = ints([j for t in new for j in range(t)])


def prepare_verify(s, gen):
    case = s["case"]
    V, tree = case["vocab"], trees(case)
    start = np.concatenate([[0], np.cumsum([len(t) for t in tree])])
    n = int(start[-1])
    s["start"], s["parent"] = ints(start), ints([p for t in tree for p in t])
    s["path_ld"] = max(depth(t) for t in tree)
    x = torch.randn((n, V), generator=gen, device="cuda") * 2.5
    x += 6.0 * (torch.rand(x.shape, generator=gen, device="cuda") > 0.9998)
    s["target"] = torch.exp(x.double() - x.double().logsumexp(-1, keepdim=True)).float()
    source = s["target"]
    s["draft"] = None
    if case["mode"] == "draft":
        x += case["near"] * torch.randn(x.shape, generator=gen, device="cuda")
        s["draft"] = source = torch.exp(x.double() - x.double().logsumexp(-1, keepdim=True)).float()
    # a node's token is drawn from its parent's distribution; a looked-up or greedy one is often the likeliest
    up = ints([int(start[i]) + p for i, t in enumerate(tree) for p in t]).long()
    u = torch.rand((n, 1), generator=gen, device="cuda", dtype=torch.float64)
    token = torch.empty(n, dtype=torch.int64, device="cuda")
    for a in range(0, n, 64):
        w = source[up[a:a + 64]]
        c = w.double().cumsum(-1)
        token[a:a + 64] = torch.searchsorted(c, u[a:a + 64] * c[:, -1:]).squeeze(-1).clamp(max=V - 1)
        if case["mode"] != "draft":
            often = torch.rand(w.shape[0], generator=gen, device="cuda") < 0.6
            token[a:a + 64] = torch.where(often, w.argmax(-1), token[a:a + 64])
    s["token"] = token.int()
    s["u"] = torch.rand(n, generator=gen, device="cuda")  # of a root: the number that the last token is drawn with
    # the plan of the plain form: children of every node in order, [sequences, nodes, most children]
    most = max(t[1:].count(p) for t in tree for p in range(len(t))) if any(len(t) > 1 for t in tree) else 1
    kids = np.full((len(tree), max(len(t) for t in tree), max(1, most)), -1)
    for i, t in enumerate(tree):
        for j in range(1, len(t)):
            row = kids[i, t[j]]
            row[np.argmax(row < 0)] = j
    s["kids"] = torch.from_numpy(kids).to("cuda")


def prepare_pool(s, gen):
    """Sequences whose pages are scattered over a pool, and what a program keeps of it: the page table, the pages of
    every sequence, the reference counts, the free pages as a stack with its size; all in one buffer of int32."""
    case = s["case"]
    n = lengths(case)
    more = len(forks(case)) if case["op"] == "fork" else 0
    rows, need = case["seqs"] + more, [-(-t // PAGE) for t in n]
    used, total = sum(need), sum(need) + more + 5 + sum(need) // 8
    ld = max(need) + 1
    s["pages"] = new_pool(case, gen, total)
    order = torch.randperm(total, generator=gen, device="cuda").int().cpu()
    table, counts, refs = (torch.full(n, v, dtype=torch.int32) for n, v in (((rows, ld), -1), ((rows,), 0), ((total,), 0)))
    done = 0
    for i, k in enumerate(need):
        table[i, :k] = order[done:done + k]
        counts[i] = k
        refs[table[i, :k].long()] = 1
        done += k
    free = torch.full((total,), -1, dtype=torch.int32)
    free[:total - used] = order[used:]
    s["saved"] = torch.cat([table.flatten(), counts, refs, free, torch.tensor([total - used], dtype=torch.int32)]).to("cuda")
    s["live"] = s["saved"].clone()
    at = np.cumsum([0, rows * ld, rows, total, total, 1])
    part = [s["live"][a:b] for a, b in zip(at[:-1], at[1:])]
    s["table"], s["seq_pages"], s["refs"], s["free"], s["n_free"] = part[0].view(rows, ld), *part[1:]
    if case["op"] == "fork":
        f = forks(case)
        s["src"], s["len"] = ints([a for a, _ in f]), ints([b for _, b in f])
        s["dst"], s["plan"] = ints([case["seqs"] + i for i in range(len(f))]), f
    else:
        s["gone"] = ints(list(range(0, case["seqs"], case["every"])))


# ---- the passes --------------------------------------------------------------------------------------
def run(state):
    if state["case"]["op"] in ("fork", "compact"):
        state["live"].copy_(state["saved"])  # a pass starts from the same pool; page contents stay where they were
    return run_own(state) if own else PLAIN[state["case"]["op"]](state)


def run_own(s):
    from quantized_decode_matvec_gb300 import mq
    case = s["case"]
    if "ready" not in s:
        mq.init()
        s["ready"] = True
    if case["op"] == "softmax":
        return mq.softmax(s["x"], scale=case["scale"])
    if case["op"] == "verify":
        return mq.verify_tree(s["target"], s["start"], s["token"], s["parent"], u=s["u"], draft=s["draft"],
                              greedy=case["mode"] == "greedy", path_ld=s["path_ld"])
    if "cache" not in s:  # the handles that a program keeps
        s["cache"] = mq.KVCache(s["pages"], s["table"], case["type"], case["kv"], case["dim"])
        if case["op"] == "attn":
            s["work"] = mq.attn_shared_workspace(s["cache"], case["heads"], s["q"].shape[0], case["groups"], s["most"])
        else:
            s["pool"] = mq.KVPool(s["cache"], s["seq_pages"], s["refs"], s["free"], s["n_free"])
    if case["op"] == "fork":
        mq.kv_fork(s["cache"], s["pool"], s["src"], s["dst"], s["len"])
        return s["live"], s["pages"]
    if case["op"] == "compact":
        mq.kv_free(s["cache"], s["pool"], s["gone"])
        mq.kv_compact(s["cache"], s["pool"])
        return s["live"], s["pages"]
    out = mq.attn_shared(s["cache"], s["q"], s["start"], s["ctx"], s["grp_start"], s["grp_pages"], mask=s["mask"],
                         scale=s["scale"], max_len=s["longest"], max_tokens=s["most"], max_pages=s["most_pages"],
                         out_type=case["out"], workspace=s["work"])
    if case["out"] == "q8_0":  # 34-byte blocks: f16 scale, 32 codes; the values they stand for
        n = out.shape[0]
        return out.view(torch.int8).view(n, -1, 34)[..., 2:] * out.view(torch.float16).view(n, -1, 17)[..., :1]
    return out


def softmax_plain(s):
    x = s["x"] * s["case"]["scale"]
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def verify_plain(s):
    """All sequences at once: a step down the trees per round, a child per inner round.  Probabilities, their sums and
    the random numbers meet in 64 bits: which token comes out hangs on it."""
    V, start = s["case"]["vocab"], s["start"].long()
    B, K = s["kids"].shape[0], s["kids"].shape[2]
    dev = s["target"].device
    one = torch.arange(B, device=dev)
    path = torch.zeros((B, s["path_ld"]), dtype=torch.int32, device=dev)
    count, at = torch.ones(B, dtype=torch.int64, device=dev), torch.zeros(B, dtype=torch.int64, device=dev)
    live, next_ = torch.ones(B, dtype=torch.bool, device=dev), torch.full((B,), -1, dtype=torch.int64, device=dev)
    ids = torch.arange(V, device=dev)
    for step in range(s["path_ld"]):
        p = s["target"][start[:-1] + at].double()
        taken = torch.full((B,), -1, dtype=torch.int64, device=dev)
        if s["case"]["mode"] == "greedy":
            best = p.argmax(-1)
            for k in range(K):
                c = s["kids"][one, at, k]
                hit = (c >= 0) & (taken < 0) & (s["token"][start[:-1] + c.clamp(min=0)].long() == best)
                taken = torch.where(hit, c, taken)
            last = best
        else:
            q = s["draft"][start[:-1] + at].double() if s["draft"] is not None else None
            mass = torch.ones(B, dtype=torch.float64, device=dev)
            rest, a = p, torch.zeros_like(mass)
            for k in range(K):
                c = s["kids"][one, at, k]
                x = s["token"][start[:-1] + c.clamp(min=0)].long()
                u = s["u"][start[:-1] + c.clamp(min=0)].double()
                try_ = (c >= 0) & (taken < 0)
                ok = try_ & (u * mass * (q[one, x] if q is not None else 1.0) < rest[one, x])
                taken = torch.where(ok, c, taken)
                no = try_ & ~ok
                if q is not None:
                    a = torch.where(no, a + mass, a)
                    rest = torch.where(no[:, None], (p - a[:, None] * q).clamp(min=0), rest)
                    mass = torch.where(no, rest.sum(-1), mass)
                else:
                    mass = torch.where(no, mass - rest[one, x], mass)
                    rest = torch.where(no[:, None] & (ids == x[:, None]), torch.zeros_like(rest), rest)
            empty = rest.sum(-1) <= 0
            rest = torch.where(empty[:, None], p, rest)
            c = rest.cumsum(-1)
            last = ((c <= (s["u"][start[:-1]].double() * c[:, -1])[:, None]).sum(-1)).clamp(max=V - 1)
        ends = live & (taken < 0)
        next_ = torch.where(ends, last, next_)
        live = live & (taken >= 0)
        if step + 1 < s["path_ld"]:
            path[:, step + 1] = torch.where(live, taken, path[:, step + 1].long()).int()
            count = torch.where(live, count + 1, count)
            at = torch.where(live, taken, at)
    return path, count.int(), next_.int()


def fork_plain(s):
    case = s["case"]
    # the sizes are the plan's, as a scheduler has them on the host
    free = s["pages"].shape[0] - sum(-(-t // PAGE) for t in lengths(case))
    for i, (src, length) in enumerate(s["plan"]):
        dst, full, rest = case["seqs"] + i, length // PAGE, length % PAGE
        s["table"][dst, :full] = s["table"][src, :full]
        s["refs"].index_add_(0, s["table"][src, :full], torch.ones(full, dtype=torch.int32, device="cuda"))
        if rest:
            free -= 1
            s["table"][dst, full] = s["free"][free]
            at = s["free"][free].long().view(1)
            s["refs"].index_fill_(0, at, 1)
            b = row_bytes(case, rest)
            moved = s["pages"].index_select(0, s["table"][src, full].view(1))[:, :, b]
            target = s["pages"].index_select(0, at)
            target[:, :, b] = moved
            s["pages"].index_copy_(0, at, target)
        s["seq_pages"][dst] = full + (1 if rest else 0)
    s["n_free"].fill_(free)
    return s["live"], s["pages"]


def compact_plain(s):
    case, n = s["case"], lengths(s["case"])
    total, need = s["pages"].shape[0], [-(-t // PAGE) for t in n]
    free = total - sum(need)
    for i in range(0, case["seqs"], case["every"]):  # pages of a sequence that nobody else has, in their order
        got = s["table"][i, :need[i]].clone()
        s["refs"].index_fill_(0, got.long(), 0)
        s["free"][free:free + need[i]] = got
        free += need[i]
        s["table"][i, :need[i]] = -1
        s["seq_pages"][i] = 0
    used = total - free
    taken = s["refs"] > 0
    # the k-th used page (in ascending order) behind the front takes the place of the k-th free one in it
    page = torch.arange(total, device="cuda")
    hole, far = torch.cumsum(~taken[:used], 0) - 1, torch.cumsum(taken[used:], 0) - 1
    nowhere = torch.full((1,), total, device="cuda")

    def by_rank(which, rank, at):
        out = torch.zeros(total + 1, dtype=torch.int64, device="cuda")
        return out.scatter_(0, torch.where(which, rank, nowhere), at)

    hole_at, far_at = by_rank(~taken[:used], hole, page[:used]), by_rank(taken[used:], far, page[used:])
    to = torch.cat([page[:used], torch.where(taken[used:], hole_at[far.clamp(min=0)], page[used:])])
    src = torch.cat([torch.where(taken[:used], page[:used], far_at[hole.clamp(min=0)]), page[used:]])
    s["pages"].copy_(s["pages"][src])
    s["refs"].copy_(s["refs"][src] * (page < used))
    t = s["table"]
    t.copy_(torch.where(t >= 0, to[t.clamp(min=0).long()].int(), t))
    s["free"][:free] = torch.arange(total - 1, used - 1, -1, dtype=torch.int32, device="cuda")
    s["n_free"].fill_(free)
    return s["live"], s["pages"]


def attn_plain(s):
    """Group by group: the scores of the prefix in one product, those of each sequence's own keys padded to the longest."""
    case = s["case"]
    group, prefix, ctx, new = batch(case)
    Hq, Hkv, D = case["heads"], case["kv"], case["dim"]
    G, outs = Hq // Hkv, []
    first_seq = first_tok = 0
    for g, tokens in enumerate(prefix):
        n, P = group.count(g), tokens // PAGE
        T = max(new[first_seq:first_seq + n])
        tok = sum(new[first_seq:first_seq + n])
        own_len = [c + t - P * PAGE for c, t in zip(ctx[first_seq:first_seq + n], new[first_seq:first_seq + n])]
        L = max(own_len)
        seq, node = s["seq"][first_tok:first_tok + tok].long() - first_seq, s["node"][first_tok:first_tok + tok].long()
        q = torch.zeros((n, T, Hq, D), device="cuda")
        q[seq, node] = s["q"][first_tok:first_tok + tok].view(-1, Hq, D).float()
        q = q.view(n, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(n, Hkv, T * G, D)
        used = s["table"][first_seq:first_seq + n, P:P - (-L // PAGE)].long()
        k, v = (get(s["pages"][used], case, w).permute(0, 2, 1, 3, 4).reshape(n, Hkv, -1, D)[:, :, :L].float()
                for w in (False, True))
        mine = torch.matmul(q, k.transpose(-1, -2)).view(n, Hkv, T, G, L) * s["scale"]
        j = torch.arange(L, device="cuda") + P * PAGE - s["ctx"][first_seq:first_seq + n].long()[:, None]
        seen = torch.zeros((n, T), dtype=torch.int64, device="cuda")
        seen[seq, node] = s["mask"][first_tok:first_tok + tok] if s["mask"] is not None else ((2 << node) - 1)
        bit = (seen[:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
        ok = (j < 0)[:, None, :] | ((j >= 0) & (j < 64))[:, None, :] & (bit == 1)
        mine = mine.masked_fill(~ok[:, None, :, None, :], -math.inf).view(n, Hkv, T * G, L)
        if P:
            blocks = s["pages"][s["table"][first_seq, :P].long()]  # [P, kv, block]
            pk, pv = (get(blocks, case, w).permute(1, 0, 2, 3).reshape(Hkv, P * PAGE, D).float() for w in (False, True))
            theirs = torch.matmul(q.transpose(0, 1).reshape(Hkv, n * T * G, D), pk.transpose(-1, -2)) * s["scale"]
            theirs = theirs.view(Hkv, n, T * G, P * PAGE).transpose(0, 1)
            m = torch.maximum(mine.amax(-1, keepdim=True), theirs.amax(-1, keepdim=True))
            a, b = torch.exp(theirs - m), torch.exp(mine - m)
            total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
            o = torch.matmul(a.transpose(0, 1).reshape(Hkv, n * T * G, -1), pv).view(Hkv, n, T * G, D).transpose(0, 1)
            o = (o + torch.matmul(b, v)) / total
        else:
            m = mine.amax(-1, keepdim=True)
            b = torch.exp(mine - torch.where(m == -math.inf, torch.zeros_like(m), m))
            total = b.sum(-1, keepdim=True)
            o = torch.matmul(b, v) / torch.where(total == 0, torch.ones_like(total), total)
        o = o.view(n, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(n, T, Hq * D)
        outs.append(o[seq, node])
        first_seq, first_tok = first_seq + n, first_tok + tok
    o = torch.cat(outs)
    if case["out"] == "q8_0":
        c, d = quantise(o)
        return (c.view(o.shape[0], -1, 32) * d.float()[..., None]).half()
    return o.half()


PLAIN = dict(attn=attn_plain, softmax=softmax_plain, verify=verify_plain, fork=fork_plain, compact=compact_plain)


# ---- what a pass cannot do without -------------------------------------------------------------------
def work(case):
    if case["op"] == "softmax":
        n = case["rows"] * case["vocab"]
        return dict(bytes=8 * n, flops=4 * n)
    if case["op"] == "verify":
        # the rows of the node that a path ends at: the target's, and the draft's where one was refused
        n = case["seqs"] * case["vocab"]
        rows = 2 if case["mode"] == "draft" else 1
        return dict(bytes=4 * n * rows, flops=2 * n * rows)
    if case["op"] == "fork":
        rest = sum(length % PAGE for _, length in forks(case))
        table = sum(-(-length // PAGE) for _, length in forks(case))
        return dict(bytes=2 * rest * token_bytes(case) + 16 * table, flops=table)
    if case["op"] == "compact":
        need = [-(-t // PAGE) for t in lengths(case)]
        total = sum(need) + 5 + sum(need) // 8
        used = sum(k for i, k in enumerate(need) if i % case["every"])
        moved = used * (total - used) / total  # on average over the orders of the pages
        return dict(bytes=int(2 * moved * PAGE * token_bytes(case) + 16 * total), flops=total)
    _, prefix, ctx, new = batch(case)
    group = batch(case)[0]
    D, Hq, n = case["dim"], case["heads"], sum(new)
    out = Hq * D * (2 if case["out"] == "f16" else 34 / 32)
    shared = [p // PAGE * PAGE for p in prefix]
    keys = sum(shared) + sum(c + t - shared[g] for g, c, t in zip(group, ctx, new))
    return dict(bytes=int(keys * token_bytes(case) + n * (Hq * D * 2 + out)),
                flops=sum(4 * (c + t) * t * Hq * D for c, t in zip(ctx, new)))


# ---- the definition in 64 bits -----------------------------------------------------------------------
def cached64(s, seq, n, head):
    """Keys and values (float64, [n, D]) of one head of a sequence's first n slots, byte by byte from the layout."""
    case = s["case"]
    D, size = case["dim"], s["pages"].shape[-1]
    slots = torch.arange(n, device="cuda")
    blocks = s["pages"][s["table"][seq].long()[slots // PAGE], head].reshape(-1, size)
    r = (slots % PAGE)[:, None]
    got = []
    for is_v in (0, 1):
        e = torch.arange(D, device="cuda")[None, :]
        if case["type"] == "f16":
            byte = is_v * PAGE * D * 2 + (e >> 6) * 8192 + r * 128 + ((((e & 63) >> 3) ^ (r & 7)) << 4) + 2 * (e & 7)
            got.append(torch.gather(blocks.view(torch.float16), 1, byte >> 1).double())
        else:
            turn = (r & 7) if D == 128 else (r >> 1) & 3
            code = torch.gather(blocks, 1, is_v * PAGE * D + r * D + (((e >> 4) ^ turn) << 4) + (e & 15)).double() - 128
            place = 2 * PAGE * D + is_v * PAGE * (D >> 4) + 2 * (r * (D >> 5) + (e >> 5))
            got.append((torch.gather(blocks.view(torch.float16), 1, place >> 1).double() * code).half().double())
    return got


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # copies and whole numbers
    s = prepare(case, seed)
    if case["op"] == "softmax":
        return torch.softmax(s["x"].double() * case["scale"], -1)
    if case["op"] == "verify":
        return exact_verify(s)
    _, _, ctx, new = batch(case)
    D, Hq, Hkv = case["dim"], case["heads"], case["kv"]
    if case["out"] == "q8_0" or sum(ctx) * Hkv > 1.2e8:
        return None  # codes of 8 bits have no value in 64; and what would take too long
    outs, first, G = [], 0, Hq // Hkv
    for i, (c, t) in enumerate(zip(ctx, new)):
        q = s["q"][first:first + t].double().view(t, Hkv, G, D)
        o = torch.zeros((t, Hkv, G, D), dtype=torch.float64, device="cuda")
        see = torch.ones((t, c + t), dtype=torch.bool)
        for a in range(t):
            bits = int(s["mask"][first + a]) if s["mask"] is not None else (2 << a) - 1
            see[a, c:] = torch.tensor([(bits >> b) & 1 == 1 for b in range(t)])
        see = see.to("cuda")[:, None, :]
        for h in range(Hkv):
            k, v = cached64(s, i, c + t, h)
            w = (q[:, h] @ k.T * s["scale"]).masked_fill(~see, -math.inf)
            o[:, h] = torch.softmax(w, -1) @ v
        outs.append(o.view(t, Hq * D))
        first += t
    return torch.cat(outs)


def exact_verify(s):
    """Sequence by sequence, with the residual distribution itself: R = p; a refused x: R = (R - q)+ / its sum."""
    case, start = s["case"], s["start"].tolist()
    token, parent, u = s["token"].tolist(), s["parent"].tolist(), s["u"].tolist()
    B = len(start) - 1
    path, count, last = torch.zeros((B, s["path_ld"]), dtype=torch.int32), [], []
    for b in range(B):
        i, n, nodes = 0, 1, range(1, start[b + 1] - start[b])
        while True:
            p = s["target"][start[b] + i].double()
            q = s["draft"][start[b] + i].double() if s["draft"] is not None else None
            R, go = p.clone(), None
            best = int(p.argmax()) if case["mode"] == "greedy" else None
            for c in (c for c in nodes if parent[start[b] + c] == i):
                x = token[start[b] + c]
                if best is not None:
                    if x == best and go is None:
                        go = c
                    continue
                if u[start[b] + c] * (float(q[x]) if q is not None else 1.0) < float(R[x]):
                    go = c
                    break
                if q is not None:
                    R = torch.relu(R - q)
                else:
                    R[x] = 0.0
                R = R / R.sum() if float(R.sum()) > 0 else R
            if go is None:
                break
            path[b, n], i, n = go, go, n + 1
        if best is None:
            R = p if float(R.sum()) <= 0 else R
            c = torch.cumsum(R, 0)
            best = min(case["vocab"] - 1, int(torch.searchsorted(c, u[start[b]] * c[-1], right=True)))
        count.append(n)
        last.append(best)
    return path.to("cuda"), ints(count), ints(last)
