"""Workloads of the serving operators over a paged K/V cache.

Three groups of operators, each with its plain form and the framework's call:

* tree:    attention of a tree of drafted tokens over a cache whose sequences
           differ in length (one drafted token is ordinary decoding);
* select:  per-block bounds of the cached keys, a cheap score that picks blocks
           for each query, and attention over the picked blocks only;
* evict:   the attention weight that each cached key has gathered, the keys to
           keep under a budget, and the cache compacted to them.

``own`` says which side ``run`` takes: False, the plain form in elementary
torch operations; True, the framework's kernels.
"""

import math

import torch

own = False

DEV = "cuda"
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# ------------------------------------------------------------------ cases --

def listed():
    """The cases that are always measured."""
    tree = dict(op="tree", D=128, kv="bf16", page=64)
    sel = dict(op="select", D=128, kv="bf16", page=64, block=64, sinks=1, recent=2)
    return [
        # one request: a draft of 8 nodes over a short context, where latency counts
        dict(tree, name="tree b1 t8 s1000", B=1, T=8, Hq=32, Hkv=8, lo=1000, hi=1000),
        # a busy server: 16-node drafts over contexts of mixed length, small pages
        dict(tree, name="tree b16 t16 s4000", B=16, T=16, Hq=32, Hkv=8, lo=517, hi=4001, page=16),
        # wide drafts over long contexts: the largest
        dict(tree, name="tree b16 t64 s16384", B=16, T=64, Hq=64, Hkv=8, lo=8192, hi=16384),
        # plain decoding (one token) of a large ragged batch over an E4M3 cache without pages
        dict(tree, name="tree b48 t1 s8192 e4m3", B=48, T=1, Hq=32, Hkv=8, lo=999, hi=8190, kv="e4m3", page=0),
        # one request decodes: blocks picked out of 8191 keys
        dict(sel, name="select b1 s8191", B=1, T=1, Hq=32, Hkv=8, lo=8191, hi=8191, top=16),
        # a batch of long contexts decodes two tokens each
        dict(sel, name="select b16 t2 s32768", B=16, T=2, Hq=64, Hkv=8, lo=20011, hi=32768, top=32),
        # a prompt: 128-token query tiles pick 128-key blocks, and attend to them
        dict(sel, name="select prompt s8192", op="prompt", B=1, T=8192, Hq=32, Hkv=8, lo=8192, hi=8192, page=0,
             block=128, top=16),
        # bounds of a batch of prompts just written to the cache
        dict(op="bounds", name="bounds b4 s16384", B=4, Hkv=8, D=128, kv="bf16", page=64, block=64, lo=12001, hi=16384),
        # the weight that a prompt's keys gathered over its own queries
        dict(op="weights", name="weights prompt s6144", B=1, T=6144, Hq=32, Hkv=8, D=128, kv="bf16", page=0, lo=6144, hi=6144),
        # one decoding step of a batch adds to the weights
        dict(op="weights", name="weights b32 t1 s8192", B=32, T=1, Hq=32, Hkv=8, D=128, kv="bf16", page=64, lo=3001, hi=8192),
        # one short sequence shrinks to its budget
        dict(op="evict", name="evict b1 s2049", B=1, Hkv=8, D=128, kv="bf16", page=16, lo=2049, hi=2049, budget=512),
        # a batch of long prompts shrinks to a quarter
        dict(op="evict", name="evict b8 s32768", B=8, Hkv=8, D=128, kv="bf16", page=64, lo=25001, hi=32768, budget=8192),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["tree", "tree", "select", "select", "prompt", "bounds", "weights", "weights", "evict", "evict"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    c = dict(op=op, Hkv=Hkv, D=rng.choice([64, 128, 128]), kv=rng.choice(["bf16", "bf16", "e4m3"]),
             page=rng.choice([0, 16, 32, 64, 128]))
    if op == "tree":
        c.update(B=_log_int(rng, 1, 32), T=_log_int(rng, 1, 64), Hq=Hkv * G)
        hi = _log_int(rng, 64, min(16384, 262144 // c["B"]))
        c.update(lo=rng.randint(1, hi), hi=hi)
    elif op == "select":
        c.update(B=_log_int(rng, 1, 16), T=rng.choice([1, 1, 2, 4]), Hq=Hkv * G, block=rng.choice([16, 32, 64, 128]),
                 top=_log_int(rng, 4, 48), sinks=rng.choice([0, 1]), recent=rng.choice([1, 2]))
        hi = _log_int(rng, 500, min(32768, 400000 // c["B"]))
        c.update(lo=rng.randint(hi // 4, hi), hi=hi)
    elif op == "prompt":
        S = _log_int(rng, 300, 6000)
        c.update(B=1, T=S, Hq=Hkv * min(G, 32 // Hkv), D=128, kv="bf16", page=0, lo=S, hi=S, block=128,
                 top=rng.randint(3, 16), sinks=1, recent=2)
    elif op == "bounds":
        c.update(B=_log_int(rng, 1, 8), block=rng.choice([16, 32, 64, 128]))
        hi = _log_int(rng, 100, 65536 // c["B"])
        c.update(lo=rng.randint(1, hi), hi=hi)
    elif op == "weights":
        if rng.random() < 0.4:
            S = _log_int(rng, 200, 5000)
            c.update(B=1, T=S, Hq=Hkv * min(G, 32 // Hkv), lo=S, hi=S)
        else:
            hi = _log_int(rng, 100, 16384)
            c.update(B=_log_int(rng, 1, 16), T=rng.choice([1, 1, 2, 5]), Hq=Hkv * G, lo=rng.randint(hi // 3 + 5, hi + 5), hi=hi + 5)
    else:
        hi = _log_int(rng, 300, 32768)
        c.update(B=_log_int(rng, 1, 8), lo=rng.randint(hi // 2, hi), hi=hi, budget=rng.randint(hi // 8 + 64, hi // 2 + 64))
    return c


def _lens(c):
    """Sequence lengths, spread evenly over [lo, hi]."""
    B = c["B"]
    return [c["hi"] if B == 1 else c["lo"] + (c["hi"] - c["lo"]) * b // (B - 1) for b in range(B)]


def _nodes(c):
    """Drafted nodes of each sequence: T at most, at least half of it."""
    return [c["T"] - 7 * b % (c["T"] // 2 + 1) for b in range(c["B"])]


def work(c):
    """Bytes and operations that one pass cannot do without."""
    lens, D, Hkv = _lens(c), c["D"], c["Hkv"]
    e = 2 if c["kv"] == "bf16" else 1
    row = Hkv * D * e  # one token's K (or V)
    n = sum(lens)
    if c["op"] == "bounds":
        blocks = sum(-(-s // c["block"]) for s in lens)
        return {"bytes": n * row + blocks * Hkv * 2 * D * 2, "flops": 2 * n * Hkv * D}
    if c["op"] == "evict":
        kept = sum(min(s, c["budget"]) for s in lens)
        return {"bytes": 4 * n * Hkv + kept * (4 * row + 4 * Hkv) + 4 * kept * Hkv, "flops": n * Hkv}
    T, Hq, B = c["T"], c["Hq"], c["B"]
    io = 2 * B * T * Hq * D * 2 + 4 * B * T * Hq  # q, o and lse
    if c["op"] == "tree":
        nodes = _nodes(c)
        pairs = sum(m * (s + m) for s, m in zip(lens, nodes))
        return {"bytes": 2 * (n + sum(nodes)) * row + io, "flops": 4 * Hq * D * pairs}
    if c["op"] == "select":
        blocks = sum(-(-s // c["block"]) for s in lens)
        keys = T * sum(min(s, c["top"] * c["block"]) for s in lens)
        return {"bytes": blocks * Hkv * 2 * D * 2 + 2 * keys * row + io + 4 * B * T * Hkv * c["top"],
                "flops": 4 * T * blocks * Hkv * D + 4 * keys * Hq * D}
    if c["op"] == "prompt":
        nb, pairs = -(-T // 128), 0
        for i in range(nb):
            pairs += min(i + 1, c["top"]) * 128 * 128 - 128 * 127 // 2  # causal in the last block
        return {"bytes": 2 * n * row + io + nb * nb * Hkv + nb * Hkv * 2 * D * 2, "flops": 4 * pairs * Hq * D}
    pairs = sum(T * s - T * (T - 1) // 2 for s in lens)  # causal
    acc = 4 * n * Hkv * (1 if T > 64 else 2)
    return {"bytes": n * row + B * T * Hq * (2 * D + 4) + acc, "flops": 2 * pairs * Hq * D + pairs * Hq}


# ----------------------------------------------------------------- inputs --

def _keys(c, gen, slots):
    """Keys (or values) of `slots` tokens: noise, a bias of each channel and an offset shared by 64 neighbours."""
    Hkv, D = c["Hkv"], c["D"]
    near = torch.randn(-(-slots // 64), 1, Hkv, D, generator=gen, device=DEV, dtype=BF16)
    x = torch.randn(near.shape[0], 64, Hkv, D, generator=gen, device=DEV, dtype=BF16)
    x = x.mul_(0.8).add_(near, alpha=0.5).add_(torch.randn(Hkv, D, generator=gen, device=DEV, dtype=BF16), alpha=0.4)
    x = x.view(-1, Hkv, D)[:slots]
    return x if c["kv"] == "bf16" else (x * 64).to(E4M3)


def _cache(c, gen, rows, out_rows=0):
    """K and V of B sequences with room for `rows` tokens: [B, rows, Hkv, D], or pools of pages and a page table."""
    B, page, s = c["B"], c["page"], {}
    if page == 0:
        s["k"] = _keys(c, gen, B * rows).view(B, rows, c["Hkv"], c["D"])
        s["v"] = _keys(c, gen, B * rows).view(B, rows, c["Hkv"], c["D"])
        s["table"] = None
    else:
        per = -(-rows // page)
        s["k"] = _keys(c, gen, B * per * page).view(B * per, page, c["Hkv"], c["D"])
        s["v"] = _keys(c, gen, B * per * page).view(B * per, page, c["Hkv"], c["D"])
        s["table"] = torch.randperm(B * per, generator=gen, device=DEV).to(torch.int32).view(B, per)
    if out_rows:
        per = -(-out_rows // page) if page else 0
        shape = (B, out_rows) if page == 0 else (B * per, page)
        for name in ("k_out", "v_out"):
            s[name] = torch.zeros(shape + s["k"].shape[2:], dtype=BF16, device=DEV).to(s["k"].dtype)
        s["out_table"] = None if page == 0 else torch.randperm(B * per, generator=gen, device=DEV).to(torch.int32).view(B, per)
    s["scale"] = None if c["kv"] == "bf16" else torch.full((1,), 1 / 64, device=DEV)
    return s


def _tree(c, gen):
    """Who sees whom among the drafted nodes: each node's parent is an earlier node, and a node sees itself and its ancestors."""
    B, T = c["B"], c["T"]
    parent = (torch.rand(B, T, generator=gen, device=DEV) * torch.arange(T, device=DEV)).long()  # node 0: the root
    sees = torch.eye(T, device=DEV).expand(B, T, T).clone()
    step = torch.zeros(B, T, T, device=DEV).scatter_(2, parent[:, :, None], 1.0)
    hops = max(1, (T - 1).bit_length())
    sees = ((sees + step) > 0).float()
    for _ in range(hops):
        sees = ((sees @ sees) > 0).float()
    return sees.to(torch.uint8)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)
    op, T = c["op"], c.get("T", 0)
    top = int(lens.max())
    s = {"case": c}
    if op == "tree":
        s.update(_cache(c, gen, top + T), lens=lens)
        s["tree_lens"] = torch.tensor(_nodes(c), dtype=torch.int32, device=DEV)
        s["mask"] = _tree(c, gen)
    elif op == "evict":
        s.update(_cache(c, gen, top, out_rows=min(top, c["budget"])), lens=lens)
        w = torch.rand(c["B"], c["Hkv"], top, generator=gen, device=DEV).clamp_(min=1e-7)
        s["weights"] = (-w.log()) ** 3  # heavy-tailed, as gathered weights are
        s["weights_out"] = torch.empty(c["B"], c["Hkv"], min(top, c["budget"]), device=DEV)
    else:
        s.update(_cache(c, gen, top), lens=lens)
    if T:
        s["q"] = torch.randn(c["B"], T, c["Hq"], c["D"], generator=gen, device=DEV, dtype=BF16)
    if op in ("select", "prompt", "bounds"):
        s["bounds"] = torch.zeros(c["B"], c["Hkv"], -(-top // c["block"]), 2, c["D"], dtype=BF16, device=DEV)
        if op != "bounds":
            s["bounds"].copy_(_plain_bounds(s))
    if op == "weights":
        s["lse"] = _plain_lse(s)
        s["weights"] = torch.rand(c["B"], c["Hkv"], top, generator=gen, device=DEV)
    return s


# ------------------------------------------------------------ plain forms --

def _values(x):
    """What 8-bit codes stand for."""
    return x.float() if x.element_size() == 1 else x


def _tokens(x, table):
    """Cached rows in order, in 32 bits: [B, Hkv, slots, D]."""
    x = x if table is None else x[table.long()].flatten(1, 2)
    return x.float().transpose(1, 2)


def _kv(s):
    scale = 1.0 if s["scale"] is None else s["scale"]
    return _tokens(s["k"], s["table"]) * scale, _tokens(s["v"], s["table"]) * scale


def _grouped(q, Hkv):
    """[B, T, Hq, D] -> [B, Hkv, T * G, D] in 32 bits, token-major."""
    B, T, Hq, D = q.shape
    return q.float().view(B, T, Hkv, Hq // Hkv, D).transpose(1, 2).reshape(B, Hkv, -1, D)


def _softmax_v(scores, v):
    """softmax(scores) v and the log-sum-exp; a row without a key gives 0 and -inf."""
    top = scores.amax(-1, keepdim=True)
    p = (scores - top.masked_fill(top == -math.inf, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total.masked_fill(total == 0, 1)
    return o, (total.log() + top).squeeze(-1)


def _answer(s, o, lse, Hkv):
    """[B, Hkv, T * G, D] and its sums back to [B, T, Hq, D] and [B, Hq, T]."""
    B, T, Hq, D = s["q"].shape
    o = o.view(B, Hkv, T, Hq // Hkv, D).transpose(1, 2).reshape(B, T, Hq, D).to(BF16)
    return o, lse.view(B, Hkv, T, Hq // Hkv).transpose(2, 3).reshape(B, Hq, T)


def _positions(s):
    """Key positions, and the position of each query token: the last T of its sequence."""
    T = s["q"].shape[1]
    at = s["lens"].long()[:, None] - T + torch.arange(T, device=DEV)
    slots = s["k"].shape[1] if s["table"] is None else s["table"].shape[1] * s["k"].shape[1]
    return torch.arange(slots, device=DEV), at


def _plain_tree(s):
    q, Hkv = s["q"], s["k"].shape[2]
    B, T, Hq, D = q.shape
    k, v = _kv(s)
    scores = (_grouped(q, Hkv) @ k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, T, Hq // Hkv, -1)
    node = torch.arange(k.shape[2], device=DEV) - s["lens"].long()[:, None]
    valid = (node < s["tree_lens"][:, None]) & (node >= 0)
    sees = s["mask"].bool().gather(2, node.clamp(0, T - 1)[:, None].expand(B, T, -1)) & valid[:, None]
    sees = (sees | (node < 0)[:, None]) & (torch.arange(T, device=DEV) < s["tree_lens"][:, None])[:, :, None]
    scores.masked_fill_(~sees[:, None, :, None], -math.inf)
    o, lse = _softmax_v(scores.flatten(2, 3), v)
    o, lse = _answer(s, o, lse, Hkv)
    return {"o": o, "lse": lse}


def _plain_bounds(s):
    """Smallest and largest key of each block and channel."""
    block = s["case"]["block"]
    k = _tokens(s["k"], s["table"])
    slots = s["bounds"].shape[2] * block
    k = torch.nn.functional.pad(k, (0, 0, 0, max(0, slots - k.shape[2])))[:, :, :slots]
    out = (torch.arange(slots, device=DEV) >= s["lens"][:, None])[:, None, :, None]
    lo = k.masked_fill(out, math.inf).unflatten(2, (-1, block)).amin(3)
    hi = k.masked_fill(out, -math.inf).unflatten(2, (-1, block)).amax(3)
    past = torch.isinf(lo)  # blocks past the sequence's end keep what the buffer held
    both = torch.stack([lo, hi], 3)
    return torch.where(past[:, :, :, None], s["bounds"].float(), both).to(BF16)


def _picked(c, score, seen):
    """Which `top` blocks are picked: the first `sinks` and last `recent` of the `seen` ones, then the best scores; ties go to the lowest."""
    j = torch.arange(score.shape[-1], device=DEV)
    forced = (j < c["sinks"]) | (j >= seen[..., None] - c["recent"])
    score = score.masked_fill(forced, math.inf).masked_fill(j >= seen[..., None], -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order).contiguous())
    return (rank < c["top"]) & (j < seen[..., None])


def _halves(s, tile):
    """Sums of the positive and of the negative parts of the queries of each (tile of tokens, KV head), in 64 bits: whole numbers depend on them."""
    q, Hkv = s["q"], s["k"].shape[2]
    B, T, Hq, D = q.shape
    x = torch.nn.functional.pad(q.double(), (0, 0, 0, 0, 0, -T % tile)).view(B, -1, tile, Hkv, Hq // Hkv, D)
    return x.clamp(min=0).sum((2, 4)), x.clamp(max=0).sum((2, 4))


def _scores(s, tile):
    up, down = _halves(s, tile)  # [B, tiles, Hkv, D]
    b = s["bounds"].double()
    return (up.transpose(1, 2) @ b[:, :, :, 1].transpose(2, 3) + down.transpose(1, 2) @ b[:, :, :, 0].transpose(2, 3)).transpose(1, 2)


def _plain_select(s):
    c, q, Hkv = s["case"], s["q"], s["k"].shape[2]
    B, T, Hq, D = q.shape
    pos, at = _positions(s)
    score = _scores(s, 1)  # [B, T, Hkv, blocks]
    seen = ((at + c["block"]) // c["block"])[:, :, None].expand(B, T, Hkv)
    picked = _picked(c, score, seen)
    n = score.shape[-1]
    j = torch.where(picked, torch.arange(n, device=DEV), n).sort(-1)[0]
    j = torch.nn.functional.pad(j, (0, max(0, c["top"] - n)), value=n)[..., : c["top"]]
    blocks = torch.where(j < n, j, -1).to(torch.int32)
    key = (j[..., None] * c["block"] + torch.arange(c["block"], device=DEV)).flatten(3)  # [B, T, Hkv, keys]
    hidden = (j >= n).repeat_interleave(c["block"], -1) | (key > at[:, :, None, None])
    key = key.clamp(max=pos.numel() - 1)
    b = torch.arange(B, device=DEV)[:, None, None, None]
    h = torch.arange(Hkv, device=DEV)[None, None, :, None]
    row = key if s["table"] is None else key % s["k"].shape[1]
    first = b if s["table"] is None else s["table"].long()[b, key // s["k"].shape[1]]
    scale = 1.0 if s["scale"] is None else s["scale"]
    k = s["k"][first, row, h].float() * scale  # [B, T, Hkv, keys, D]
    v = s["v"][first, row, h].float() * scale
    x = q.float().view(B, T, Hkv, Hq // Hkv, D)
    scores = (x @ k.transpose(3, 4)).mul_(1 / math.sqrt(D)).masked_fill_(hidden[:, :, :, None], -math.inf)
    o, lse = _softmax_v(scores, v)
    return {"blocks": blocks, "o": o.reshape(B, T, Hq, D).to(BF16), "lse": lse.reshape(B, T, Hq).transpose(1, 2)}


def _plain_prompt(s):
    c, q, Hkv = s["case"], s["q"], s["k"].shape[2]
    B, T, Hq, D = q.shape
    score = _scores(s, 128)
    last = torch.arange(128, T + 128, 128, device=DEV).clamp(max=T) - 1
    seen = (last // 128 + 1)[None, :, None].expand(score.shape[:3])
    mask = _picked(c, score, seen).transpose(1, 2)  # [B, Hkv, tiles, blocks]
    k, v = _kv(s)
    scores = (_grouped(q, Hkv) @ k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, T, Hq // Hkv, T)
    pos = torch.arange(T, device=DEV)
    sees = mask.repeat_interleave(128, 2)[:, :, :T].repeat_interleave(128, 3)[..., :T] & (pos[:, None] >= pos)
    scores.masked_fill_(~sees[:, :, :, None], -math.inf)
    o, lse = _softmax_v(scores.flatten(2, 3), v)
    o, lse = _answer(s, o, lse, Hkv)
    return {"mask": mask.to(torch.uint8), "o": o, "lse": lse}


def _causal_scores(s):
    """Scaled scores [B, Hkv, T, G, slots], -inf where a query does not see a key."""
    q, Hkv = s["q"], s["k"].shape[2]
    B, T, Hq, D = q.shape
    k, _ = _kv(s)
    pos, at = _positions(s)
    scores = (_grouped(q, Hkv) @ k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, T, Hq // Hkv, -1)
    return scores.masked_fill_((pos > at[:, :, None])[:, None, :, None], -math.inf)


def _plain_lse(s):
    B, T, Hq, _ = s["q"].shape
    return _causal_scores(s).logsumexp(-1).transpose(2, 3).reshape(B, Hq, T)


def _plain_weights(s):
    B, T, Hq, _ = s["q"].shape
    scores = _causal_scores(s)
    lse = s["lse"].view(B, scores.shape[1], -1, T).transpose(2, 3)
    w = (scores - lse[..., None]).exp_().sum((2, 3))[..., : s["weights"].shape[2]]
    if T > 64:  # a prompt's weights are new, a step's are added
        s["weights"].copy_(w)
    else:
        s["weights"].add_(w)
    return {"weights": s["weights"]}


def _plain_evict(s):
    c, w, lens = s["case"], s["weights"], s["lens"].long()
    budget = s["weights_out"].shape[2]
    n = w.shape[2]
    pos = torch.arange(n, device=DEV)
    counts = lens.clamp(max=budget)
    forced = (pos < SINKS) | (pos >= lens[:, None] - RECENT)
    score = w.masked_fill(forced[:, None], math.inf).masked_fill((pos >= lens[:, None])[:, None], -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True)[1][..., :budget]
    order = torch.where(torch.arange(budget, device=DEV) < counts[:, None, None], order, n).sort(-1)[0]
    live = order < n
    keep = torch.where(live, order, -1).to(torch.int32)
    at = order.clamp(max=n - 1)
    s["weights_out"].copy_(torch.where(live, w.gather(2, at), 0.0))
    B, Hkv = w.shape[:2]
    b, h = torch.arange(B, device=DEV)[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None]
    to = torch.arange(budget, device=DEV).expand(B, Hkv, budget)
    for x, y in ((s["k"], s["k_out"]), (s["v"], s["v_out"])):
        x, z = x.view(torch.int16 if x.element_size() == 2 else torch.uint8), y.view(torch.int16 if y.element_size() == 2 else torch.uint8)
        page = x.shape[1]
        src = (b, at, h) if s["table"] is None else (s["table"].long()[b, at // page], at % page, h)
        dst = (b, to, h) if s["table"] is None else (s["out_table"].long()[b, to // page], to % page, h)
        z[dst] = torch.where(live[..., None], x[src], z[dst])
    return {"keep": keep, "counts": counts.to(torch.int32), "k": _values(s["k_out"]), "v": _values(s["v_out"]), "weights": s["weights_out"]}


SINKS, RECENT = 4, 32  # kept by every eviction here: the first tokens and the newest


# -------------------------------------------------------------------- run --

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "bounds":
        return {"bounds": _plain_bounds(s)}
    return {"tree": _plain_tree, "select": _plain_select, "prompt": _plain_prompt, "weights": _plain_weights, "evict": _plain_evict}[op](s)


def _own(s):
    from precision_attention_fmha_b200 import fmha

    c = s["case"]
    op = c["op"]
    sf = None if s["scale"] is None else fmha.Scale(s["scale"], "per_tensor")
    if op == "bounds":
        return {"bounds": fmha.key_bounds(s["k"], s["lens"], c["block"], page_table=s["table"], bounds=s["bounds"])}
    if op == "evict":
        keep, counts = fmha.evict_select(s["weights"], s["lens"], s["weights_out"].shape[2], sinks=SINKS, recent=RECENT)
        fmha.cache_compact(s["k"], s["v"], keep, counts, page_table=s["table"], k_out=s["k_out"], v_out=s["v_out"],
                           out_page_table=s["out_table"], weights=s["weights"], weights_out=s["weights_out"])
        return {"keep": keep, "counts": counts, "k": _values(s["k_out"]), "v": _values(s["v_out"]), "weights": s["weights_out"]}
    q = s["q"]
    B, T, Hq, _ = q.shape
    if op == "weights":
        fmha.key_weights(q, s["k"], s["lse"], s["weights"], s["lens"], page_table=s["table"], accumulate=T <= 64, sf_k=sf)
        return {"weights": s["weights"]}
    lse = torch.empty(B, Hq, T, device=q.device)
    if op == "tree":
        o = fmha.fmha_fwd_tree(q, s["k"], s["v"], s["lens"], tree_mask=s["mask"], tree_lens=s["tree_lens"],
                               page_table=s["table"], sf_k=sf, sf_v=sf, lse=lse)
        return {"o": o, "lse": lse}
    if op == "prompt":
        mask = fmha.select_blocks(q, s["bounds"], s["lens"], c["block"], c["top"], sink_blocks=c["sinks"],
                                  recent_blocks=c["recent"], q_tile=128)
        o = fmha.fmha_fwd_block_sparse(q, s["k"], s["v"], mask, causal=True, lse=lse)
        return {"mask": mask, "o": o, "lse": lse}
    blocks = fmha.select_blocks(q, s["bounds"], s["lens"], c["block"], c["top"], sink_blocks=c["sinks"], recent_blocks=c["recent"])
    o = fmha.fmha_fwd_selected(q, s["k"], s["v"], blocks, s["lens"], c["block"], page_table=s["table"], sf_k=sf, sf_v=sf, lse=lse)
    return {"blocks": blocks, "o": o, "lse": lse}


# ------------------------------------------------------------------ exact --

def _row64(s, name, b, h, keys):
    """The cached rows of one sequence and KV head at `keys`, in 64 bits."""
    x = s[name]
    scale = 1.0 if s["scale"] is None else float(s["scale"])
    if s["table"] is None:
        return x[b, keys, h].double() * scale
    page = x.shape[1]
    return x[s["table"][b].long()[keys // page], keys % page, h].double() * scale


def _attend64(q, k, v, sees):
    """One group of query rows [R, D] over keys [N, D]; sees [R, N]."""
    z = (q.double() @ k.t()) / math.sqrt(q.shape[1])
    z = torch.where(sees, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, 1)
    w = torch.where(sees, torch.exp(z - lse[:, None]), torch.zeros_like(z))
    return w @ v, lse


def _exact_pick(c, score, seen):
    """Ids of the picked blocks of one query, ascending."""
    ids = sorted(range(seen), key=lambda j: (0 if j < c["sinks"] or j >= seen - c["recent"] else 1, -score[j], j))
    # forced blocks first, in order of their ids; then by score
    forced = [j for j in range(seen) if j < c["sinks"] or j >= seen - c["recent"]]
    rest = [j for j in ids if j not in set(forced)]
    return sorted((forced + rest)[: c["top"]])


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    lens, Hkv, op = _lens(c), c["Hkv"], c["op"]
    B = c["B"]
    if op == "bounds":
        out = s["bounds"].double()
        for b in range(B):
            for h in range(Hkv):
                k = _row64(dict(s, scale=None), "k", b, h, torch.arange(lens[b], device=DEV))
                for j, part in enumerate(k.split(c["block"])):
                    out[b, h, j, 0], out[b, h, j, 1] = part.min(0)[0], part.max(0)[0]
        return {"bounds": out}
    if op == "evict":
        budget = s["weights_out"].shape[2]
        w = torch.zeros(B, Hkv, budget, dtype=torch.float64, device=DEV)
        ko, vo = s["k_out"].double(), s["v_out"].double()
        for b in range(B):
            n = lens[b]
            m = min(n, budget)
            for h in range(Hkv):
                x = s["weights"][b, h, :n].double().clone()
                x[:SINKS] = math.inf
                x[max(0, n - RECENT):] = math.inf
                keys = torch.argsort(x, descending=True, stable=True)[:m].sort()[0]
                w[b, h, :m] = s["weights"][b, h, keys].double()
                to = torch.arange(m, device=DEV)
                one = dict(s, scale=None)
                if s["table"] is None:
                    ko[b, to, h], vo[b, to, h] = _row64(one, "k", b, h, keys), _row64(one, "v", b, h, keys)
                else:
                    page = s["k"].shape[1]
                    at = (s["out_table"][b].long()[to // page], to % page, torch.full_like(to, h))
                    ko[at], vo[at] = _row64(one, "k", b, h, keys), _row64(one, "v", b, h, keys)
        return {"keep": None, "counts": None, "k": ko, "v": vo, "weights": w}
    q, T, Hq = s["q"], c["T"], c["Hq"]
    G = Hq // Hkv
    if op == "weights":
        w = s["weights"].double() * (1 if T <= 64 else 0)
        for b in range(B):
            n = lens[b]
            keys = torch.arange(n, device=DEV)
            at = n - T + torch.arange(T, device=DEV)
            for h in range(Hkv):
                k = _row64(s, "k", b, h, keys)
                for g in range(h * G, h * G + G):
                    z = (q[b, :, g].double() @ k.t()) / math.sqrt(c["D"]) - s["lse"][b, g].double()[:, None]
                    w[b, h, :n] += torch.where(keys <= at[:, None], z.exp(), torch.zeros_like(z)).sum(0)
        return {"weights": w}
    o = torch.zeros(B, T, Hq, c["D"], dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, h * G + G)
            if op == "tree":
                m = int(s["tree_lens"][b])
                keys = torch.arange(lens[b] + m, device=DEV)
                k, v = _row64(s, "k", b, h, keys), _row64(s, "v", b, h, keys)
                sees = torch.cat([torch.ones(m, lens[b], dtype=torch.bool, device=DEV), s["mask"][b, :m, :m] != 0], 1)
                for g in range(h * G, h * G + G):
                    o[b, :m, g], lse[b, g, :m] = _attend64(q[b, :m, g], k, v, sees)
                continue
            bd = s["bounds"][b, h].double()
            if op == "select":
                for t in range(T):
                    x = q[b, t, heads].double()
                    score = (torch.relu(x).sum(0) * bd[:, 1] - torch.relu(-x).sum(0) * bd[:, 0]).sum(1).tolist()
                    at = lens[b] - T + t
                    ids = _exact_pick(c, score, at // c["block"] + 1)
                    keys = torch.cat([torch.arange(j * c["block"], min((j + 1) * c["block"], at + 1), device=DEV) for j in ids])
                    k, v = _row64(s, "k", b, h, keys), _row64(s, "v", b, h, keys)
                    o[b, t, heads], lse[b, heads, t] = _attend64(x, k, v, torch.ones(G, keys.numel(), dtype=torch.bool, device=DEV))
                continue
            for t in range(0, T, 128):
                end = min(T, t + 128)
                x = q[b, t:end, heads].double().reshape(-1, c["D"])
                score = (torch.relu(x).sum(0) * bd[:, 1] - torch.relu(-x).sum(0) * bd[:, 0]).sum(1).tolist()
                ids = _exact_pick(c, score, (end - 1) // 128 + 1)
                keys = torch.cat([torch.arange(j * 128, min((j + 1) * 128, T), device=DEV) for j in ids])
                k, v = _row64(s, "k", b, h, keys), _row64(s, "v", b, h, keys)
                for g in range(h * G, h * G + G):
                    sees = keys <= torch.arange(t, end, device=DEV)[:, None]
                    o[b, t:end, g], lse[b, g, t:end] = _attend64(q[b, t:end, g], k, v, sees)
    whole = {"tree": {}, "select": {"blocks": None}, "prompt": {"mask": None}}[op]
    return {**whole, "o": o, "lse": lse}
