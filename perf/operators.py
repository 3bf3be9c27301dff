"""Cases of the serving operators around a paged key / value cache: the
rotating append, attention of drafted tokens over the cache, sampling from
the logits, and the acceptance of a drafted tree.

``run`` computes a case in elementary torch operations, or, where ``own`` is
true, by the library's calls on the same state; ``exact`` gives the same
outputs from the definitions in 64 bits."""
import math
import random

import torch

own = False

F16, F32 = torch.float16, torch.float32


def listed():
    return [
        # One user's next token: the call whose launch and latency are all there is.
        dict(name="append-token", op="append", seqs=1, n=1, ctx=700, hq=16, hkv=8, d=128, page=64, rot=128,
             interleaved=False, factor=1.0, orig=0, tree=False),
        # A verification step: drafted trees of a batch, part of each head rotated in pairs of neighbours,
        # frequencies scaled by parts for a context past the trained one, small pages.
        dict(name="append-trees", op="append", seqs=24, n=27, ctx=900, hq=32, hkv=8, d=64, page=16, rot=48,
             interleaved=True, factor=8.0, orig=4096, tree=True),
        # Chunks of four prompts entering the cache together.
        dict(name="append-chunks", op="append", seqs=4, n=2048, ctx=300, hq=32, hkv=8, d=128, page=64, rot=128,
             interleaved=False, factor=4.0, orig=8192, tree=False),
        # One user's next token over a short context.
        dict(name="attend-token", op="attend", seqs=1, n=1, ctx=1000, hq=16, hkv=8, d=128, page=64, tree=False),
        # Plain decoding of a batch whose contexts differ a lot: the cache's bytes are the work.
        dict(name="attend-batch", op="attend", seqs=40, n=1, ctx=12000, hq=32, hkv=4, d=128, page=16, tree=False),
        # Drafted trees of a batch over long contexts.
        dict(name="attend-trees", op="attend", seqs=8, n=61, ctx=20000, hq=32, hkv=8, d=128, page=64, tree=True),
        # A prompt's chunk after a cached prefix, two users: products, not bytes.
        dict(name="attend-chunk", op="attend", seqs=2, n=1024, ctx=6000, hq=32, hkv=8, d=128, page=128, tree=False),
        # One row of logits, all the usual limits on.
        dict(name="sample-one", op="sample", rows=1, vocab=151936, half=False, top_k=50, top_p=0.95, min_p=0.02,
             masked=0.0),
        # A batch of users with settings of their own, some of them with none, a grammar's mask on some rows.
        dict(name="sample-batch", op="sample", rows=61, vocab=151936, half=False, top_k=-1, top_p=-1.0, min_p=-1.0,
             masked=0.5),
        # Every node of drafted trees, half-precision logits, an odd vocabulary, only the nucleus.
        dict(name="sample-nodes", op="sample", rows=256, vocab=50257, half=True, top_k=0, top_p=0.9, min_p=0.0,
             masked=0.0),
        # One user's drafted tokens, every layer's cache.
        dict(name="accept-one", op="accept", seqs=1, n=16, ctx=40, hkv=8, d=128, page=16, layers=28),
        # A batch's drafted trees.
        dict(name="accept-batch", op="accept", seqs=32, n=64, ctx=60, hkv=8, d=128, page=16, layers=28),
    ]


def _spread(rng, lo, hi):
    """An integer of lo .. hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sample", "sample", "accept"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    page = rng.choice([1, 8, 16, 24, 64, 128, 256])
    if op == "append":
        seqs = _spread(rng, 1, 64)
        rot = d if rng.random() < 0.5 else 2 * rng.randint(1, d // 2)
        return dict(op=op, seqs=seqs, n=_spread(rng, 1, max(1, 8192 // seqs)), ctx=_spread(rng, 1, 1000),
                    hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, d=d, page=page, rot=rot,
                    interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 1.0, 2.5, 8.0]),
                    orig=rng.choice([0, 4096, 8192]), tree=rng.random() < 0.5)
    if op == "attend":
        tree = rng.random() < 0.5
        n = _spread(rng, 1, 64 if tree else 1024)
        seqs = _spread(rng, 1, max(1, min(40, 2048 // n)))
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        # no more products and no more cached bytes than the largest listed ones
        most = min(250000 // seqs, int(1.3e11 / (4 * hq * d * n * seqs)) - n)
        return dict(op=op, seqs=seqs, n=n, ctx=_spread(rng, 1, max(2, min(60000, most))), hq=hq, hkv=hkv, d=d,
                    page=page, tree=tree)
    if op == "sample":
        vocab = _spread(rng, 1000, 200000)
        return dict(op=op, rows=_spread(rng, 1, max(1, min(256, 9000000 // vocab))), vocab=vocab,
                    half=rng.random() < 0.4, top_k=rng.choice([-1, 0, 1, 20, 50, 400]),
                    top_p=rng.choice([-1.0, 1.0, 0.5, 0.9, 0.99]), min_p=rng.choice([-1.0, 0.0, 0.05, 0.3]),
                    masked=rng.choice([0.0, 0.0, 0.5]))
    return dict(op=op, seqs=_spread(rng, 1, 32), n=_spread(rng, 1, 64), ctx=_spread(rng, 1, 60), hkv=hkv, d=d,
                page=page, layers=_spread(rng, 1, 28))


# ------------------------------------------------------------------ inputs ---

THETA, ALPHA, BETA, AMPLITUDE = 1.0e6, 1.0, 32.0, 1.05


def _sizes(case):
    """Cached positions and new rows of each sequence: ragged, the same for every seed."""
    r = random.Random("%s %s %s" % (case["seqs"], case["n"], case["ctx"]))
    s = case["seqs"]
    ctx = [case["ctx"]] + [max(0, int(case["ctx"] * r.uniform(0.05, 1.0))) for _ in range(s - 1)]
    if case["n"] == 1:
        n = [1] * s
    else:
        n = [case["n"]] + [r.randint(max(1, case["n"] // 3), case["n"]) for _ in range(s - 1)]
    return ctx, n


def _parents(n, r):
    """A tree in breadth-first order: the root, up to eight children of it, then children of a moving window."""
    fan = min(8, max(1, n // 2))
    p = [-1]
    for i in range(1, n):
        p.append(0 if i <= fan else min(i - 1, max(1, p[-1]) + r.choice([0, 0, 1, 1, 2])))
    return p


def _trees(case):
    r = random.Random("tree %s %s %s" % (case["seqs"], case["n"], case["ctx"]))
    return [_parents(n, r) for n in _sizes(case)[1]]


def _path(parents, i):
    p = []
    while i >= 0:
        p.append(i)
        i = parents[i]
    return p[::-1]


def _accepted_path(parents):
    """The longest path whose moves do not read a place that another of them writes, so that a case can run twice."""
    best = [0]
    for i in range(len(parents)):
        p = _path(parents, i)
        if len(p) > len(best) and all(src == dst or src >= len(p) for dst, src in enumerate(p)):
            best = p
    return best


def _frequencies(case):
    """Turns of each pair for one position: theta^(-2i/rot) / 2 pi, scaled for a longer context."""
    out = []
    for i in range(case["rot"] // 2):
        f = THETA ** (-2.0 * i / case["rot"]) / (2.0 * math.pi)
        if case["factor"] != 1.0:
            keep = min(1.0, max(0.0, (case["orig"] * f - ALPHA) / (BETA - ALPHA))) if case["orig"] else 0.0
            f = f * keep + f / case["factor"] * (1.0 - keep)
        out.append(f)
    return out


def _signed64(u):
    return u - (1 << 64) if u >= 1 << 63 else u


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    normal = lambda *shape, dtype=F16: torch.randn(*shape, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    s = dict(case=case)
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        # a body of unlikely tokens and a few that the model means, as a trained head gives them
        x = normal(rows, vocab, dtype=F32) * 2.0
        for _ in range(3):
            at = torch.randint(0, vocab, (rows, 12), generator=g, device="cuda")
            x.scatter_add_(1, at, normal(rows, 12, dtype=F32) * 3.0 + 7.0)
        if case["masked"]:
            some = torch.rand(rows, 1, generator=g, device="cuda") < case["masked"]
            x.masked_fill_(some & (torch.rand(rows, vocab, generator=g, device="cuda") < 0.97), float("-inf"))
        s["logits"] = x.half() if case["half"] else x
        mixed = lambda v, choices: [v if v >= 0 else r.choice(choices) for _ in range(rows)]  # noqa: E731
        s["temperature"] = torch.tensor([r.choice([0.0, 0.6, 0.8, 1.0, 1.3]) if rows > 1 else 0.8
                                         for _ in range(rows)], device="cuda")
        s["top_k"] = ints(mixed(case["top_k"], [0, 20, 40, 200]))
        s["top_p"] = torch.tensor(mixed(case["top_p"], [1.0, 0.8, 0.95]), device="cuda")
        s["min_p"] = torch.tensor(mixed(case["min_p"], [0.0, 0.0, 0.05]), device="cuda")
        s["u"] = torch.rand(rows, generator=g, device="cuda")
        s["tokens"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty(rows, dtype=F32, device="cuda")
        return s
    ctx, n = _sizes(case)
    hkv, d, page = case["hkv"], case["d"], case["page"]
    seqs, rows = len(ctx), sum(n)
    pages = [-(-(c + k) // page) for c, k in zip(ctx, n)]
    n_pages, width = sum(pages), max(pages)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
    at = 0
    for i, p in enumerate(pages):
        table[i, :p] = order[at:at + p]
        at += p
    start = [0]
    for k in n:
        start.append(start[-1] + k)
    layers = case.get("layers", 1)
    s.update(ctx=ints(ctx), start=ints(start), table=table, rows=rows, width=width, n_pages=n_pages,
             longest=max(c + k for c, k in zip(ctx, n)), most=max(n),
             k_pool=normal(layers, n_pages, hkv, page, d), v_pool=normal(layers, n_pages, hkv, page, d))
    if case["op"] != "accept":
        hq = case["hq"]
        s["q"] = normal(rows, hq * d)
    if case["op"] == "append":
        s["k"], s["v"] = normal(rows, hkv * d), normal(rows, hkv * d)
        s["q_out"] = torch.empty_like(s["q"])
        trees = _trees(case) if case["tree"] else None
        s["positions"] = ints([c + (len(_path(trees[i], j)) - 1 if trees else j)
                               for i, c in enumerate(ctx) for j in range(n[i])])
        turns = _frequencies(case)
        s["turns"] = torch.tensor(turns, dtype=torch.float64, device="cuda")
        # the library's table: the same frequencies in units of 2^-64 turns
        s["freqs"] = torch.tensor([_signed64(int(round(f * 2.0 ** 64))) for f in turns], dtype=torch.int64,
                                  device="cuda")
    if case["op"] == "attend":
        s["out"] = torch.empty_like(s["q"])
        s["mask"], s["words"] = None, 0
        if case["tree"]:
            words = (max(n) + 31) // 32
            bits = []
            for p in _trees(case):
                seen = []
                for j in range(len(p)):
                    seen.append((seen[p[j]] if j else 0) | 1 << j)
                bits += [[(m >> 32 * w & 0xFFFFFFFF) for w in range(words)] for m in seen]
            s["mask"] = torch.tensor(bits, dtype=torch.int64).to(torch.int32).cuda()
            s["words"] = words
        s["workspace"] = torch.empty(_workspace_bytes(case, rows), dtype=torch.uint8, device="cuda")
    if case["op"] == "accept":
        trees = _trees(case)
        draft, parents, sampled = [], [], []
        for p in trees:
            tok = [r.randrange(0, 50000) * 64 + j % 64 for j in range(len(p))]  # siblings differ
            smp = [r.randrange(0, 50000) * 64 + 63 - j % 64 if r.random() < 0.7 else 7 for j in range(len(p))]
            path = _accepted_path(p)
            children = set(tok)
            smp = [x if x not in children else 5 for x in smp]
            for a, b in zip(path, path[1:]):
                smp[a] = tok[b]
            draft += tok
            parents += p
            sampled += smp
        s.update(draft=ints(draft), parents=ints(parents), sampled=ints(sampled),
                 accepted=torch.empty(seqs, dtype=torch.int32, device="cuda"),
                 path=torch.empty(rows, dtype=torch.int32, device="cuda"),
                 next_token=torch.empty(seqs, dtype=torch.int32, device="cuda"),
                 ctx_out=torch.empty(seqs, dtype=torch.int32, device="cuda"))
    return s


def _workspace_bytes(case, rows):
    # the workspace that a program allocates once; the same bound for every tree
    return 256 << 20


# --------------------------------------------------------------- the passes ---

def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "sample": _own_sample, "accept": _own_accept}[op](s)
    return {"append": _plain_append, "attend": _plain_attend, "sample": _plain_sample, "accept": _plain_accept}[op](s)


def _own_cache(s):
    import bit_quantized_gemv_q4_gb300 as q4
    c = s["case"]
    return q4, q4.PagedCache(s["k_pool"], s["v_pool"], s["n_pages"], c["page"], c["hkv"], c["d"], s["table"],
                             c["seqs"], s["width"])


def _own_append(s):
    c = s["case"]
    q4, cache = _own_cache(s)
    q4.q4_paged_append(cache, s["ctx"], s["start"], s["rows"], s["k"], s["v"], q=s["q"], q_out=s["q_out"],
                       n_q_heads=c["hq"], positions=s["positions"], freqs=s["freqs"], rot_dim=c["rot"],
                       layout=q4.Q4_ROPE_INTERLEAVED if c["interleaved"] else q4.Q4_ROPE_HALF, amplitude=AMPLITUDE)
    return dict(q=s["q_out"], k=s["k_pool"], v=s["v_pool"])


def _own_attend(s):
    q4, cache = _own_cache(s)
    q4.q4_tree_attention(cache, s["ctx"], s["start"], s["rows"], s["q"], s["case"]["hq"], s["out"], s["workspace"],
                         s["workspace"].numel(), mask=s["mask"], mask_words=s["words"])
    return s["out"]


def _own_sample(s):
    import bit_quantized_gemv_q4_gb300 as q4
    q4.q4_sample(s["logits"], q4.Q4_F16 if s["case"]["half"] else q4.Q4_F32, s["case"]["rows"], s["case"]["vocab"],
                 s["tokens"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                 u=s["u"], probs=s["probs"])
    return dict(tokens=s["tokens"], probs=s["probs"])


def _own_accept(s):
    c = s["case"]
    q4, cache = _own_cache(s)
    q4.q4_tree_accept(cache, s["ctx"], s["start"], s["rows"], s["draft"], s["parents"], s["sampled"], s["accepted"],
                      s["path"], s["next_token"], s["ctx_out"], n_layers=c["layers"],
                      layer_stride=s["k_pool"][0].numel())
    return dict(accepted=s["accepted"], path=s["path"], next_token=s["next_token"], ctx=s["ctx_out"], k=s["k_pool"],
                v=s["v_pool"])


def _rows(s):
    """Sequence of each row and the row's place in it."""
    t = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["start"][1:].long(), t, right=True)
    return seq, t - s["start"][seq]


def _rotate(x, cos, sin, heads, rot, interleaved):
    x = x.float().reshape(x.shape[0], heads, -1)
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    c, n = cos[:, None], sin[:, None]
    p, m = a * c - b * n, b * c + a * n
    turned = torch.stack([p, m], -1).flatten(-2) if interleaved else torch.cat([p, m], -1)
    return torch.cat([turned, x[..., rot:]], -1).half()


def _plain_append(s):
    c = s["case"]
    turns = s["positions"].double()[:, None] * s["turns"]
    angle = (turns - turns.floor()) * (2.0 * math.pi)
    cos, sin = (angle.cos() * AMPLITUDE).float(), (angle.sin() * AMPLITUDE).float()
    q = _rotate(s["q"], cos, sin, c["hq"], c["rot"], c["interleaved"]).reshape(s["rows"], -1)
    k = _rotate(s["k"], cos, sin, c["hkv"], c["rot"], c["interleaved"])
    seq, i = _rows(s)
    slot = s["ctx"][seq] + i
    at = s["table"][seq, slot // c["page"]].long()
    s["k_pool"][0, at, :, slot % c["page"]] = k
    s["v_pool"][0, at, :, slot % c["page"]] = s["v"].reshape(s["rows"], c["hkv"], c["d"])
    return dict(q=q, k=s["k_pool"], v=s["v_pool"])


def _padded(s, x):
    """Rows [rows, ...] as [seqs, most, ...], zeros behind each sequence's own."""
    seq, i = _rows(s)
    out = torch.zeros(s["case"]["seqs"], s["most"], *x.shape[1:], dtype=x.dtype, device="cuda")
    out[seq, i] = x
    return out, seq, i


def _plain_attend(s):
    c = s["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    q, seq, i = _padded(s, s["q"].float().reshape(s["rows"], hkv, hq // hkv, d))
    keys = lambda pool: pool[0][s["table"].long()].float().permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :s["longest"]]  # noqa: E731
    at = torch.arange(s["longest"], device="cuda") - s["ctx"][:, None]  # place among the new rows, negative: cached
    new = (s["start"][1:] - s["start"][:-1])[:, None]
    j = at.clamp(0, s["most"] - 1)[:, None, :]
    if s["mask"] is None:
        sees = torch.arange(s["most"], device="cuda")[None, :, None] >= j
    else:
        words = _padded(s, s["mask"])[0].long()
        sees = (words.gather(2, (j // 32).expand(-1, s["most"], -1)) >> (j % 32)) & 1 == 1
    sees = (sees | (at < 0)[:, None, :]) & (at < new)[:, None, :]
    scores = torch.einsum("snhgd,shld->shgnl", q, keys(s["k_pool"])) * (1.0 / math.sqrt(d))
    scores.masked_fill_(~sees[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(top.isinf(), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    values = keys(s["v_pool"]).masked_fill_((at >= new)[:, None, :, None], 0.0)
    out = torch.einsum("shgnl,shld->snhgd", p / torch.where(total == 0, torch.ones_like(total), total), values)
    return out[seq, i].reshape(s["rows"], hq * d).half()


def _plain_sample(s):
    vocab = s["case"]["vocab"]
    value, token = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
    greedy = ~(s["temperature"] > 0)
    t = torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"]).double()
    w = ((value.double() - value[:, :1].double()) / t[:, None]).exp()
    place = torch.arange(vocab, device="cuda")
    k = torch.where(s["top_k"] > 0, s["top_k"], torch.full_like(s["top_k"], vocab))
    w = torch.where(place < k[:, None], w, torch.zeros_like(w))
    total = w.cumsum(-1)
    # the nucleus ends with the first token that brings the sum to top_p
    p = s["top_p"].double()[:, None]
    nucleus = (p >= 1) | (place == 0) | (total - w < p * total[:, -1:])
    w = torch.where(nucleus & (w >= s["min_p"].double()[:, None]) & (~greedy[:, None] | (place == 0)), w,
                    torch.zeros_like(w))
    total = w.cumsum(-1)
    at = (total <= s["u"].double()[:, None] * total[:, -1:]).sum(-1, keepdim=True).clamp(max=vocab - 1)
    return dict(tokens=token.gather(1, at)[:, 0].int(), probs=(w.gather(1, at) / total[:, -1:])[:, 0].float())


def _plain_accept(s):
    c = s["case"]
    seqs, most, page = c["seqs"], s["most"], c["page"]
    draft, seq, i = _padded(s, s["draft"].long())
    parent, smp = _padded(s, s["parents"].long())[0], _padded(s, s["sampled"].long())[0]
    place = torch.arange(most, device="cuda")
    new = (s["start"][1:] - s["start"][:-1]).long()[:, None]
    live = (place < new) & (place > 0)
    up = parent.clamp(min=0)
    hit = live & (draft == smp.gather(1, up)) & (smp.gather(1, up) >= 0)
    # of two children with the sampled token the first one counts
    same = hit[:, :, None] & hit[:, None, :] & (up[:, :, None] == up[:, None, :])
    hit = hit & ~(same & (place[None, :, None] > place[None, None, :])).any(-1)
    hit = hit | (place == 0)
    # reached: every edge up to the root is hit; the ancestors by doubling
    jump = torch.where(place == 0, place, up)
    for _ in range(max(1, most.bit_length())):
        hit = hit & hit.gather(1, jump)
        jump = jump.gather(1, jump)
    hit = hit & (place < new)
    accepted = hit.sum(-1)
    path = torch.sort(torch.where(hit, place, place + most), -1).values
    last = path.gather(1, (accepted - 1).clamp(min=0)[:, None])[:, 0]
    next_token = torch.where(accepted > 0, smp.gather(1, (last % most)[:, None])[:, 0], torch.full_like(last, -1))
    path = torch.where(place < accepted[:, None], path, torch.full_like(path, -1))
    src = s["ctx"][:, None] + torch.where(path >= 0, path, torch.zeros_like(path))
    dst = s["ctx"][:, None] + place
    who, which = torch.nonzero((path != place) & (path >= 0), as_tuple=True)
    src, dst = src[who, which], dst[who, which]
    a, b = s["table"][who, src // page].long(), s["table"][who, dst // page].long()
    for pool in (s["k_pool"], s["v_pool"]):
        pool[:, b, :, dst % page] = pool[:, a, :, src % page]
    return dict(accepted=accepted.int(), path=path[seq, i].int(), next_token=next_token.int(),
                ctx=(s["ctx"] + accepted).int(), k=s["k_pool"], v=s["v_pool"])


# -------------------------------------------------------------------- work ---

def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return dict(bytes=n * (2 if case["half"] else 4) + case["rows"] * 28, flops=4 * n)
    ctx, n = _sizes(case)
    rows, row = sum(n), case["hkv"] * case["d"] * 2
    if case["op"] == "append":
        return dict(bytes=2 * rows * (case["hq"] * case["d"] * 2 + 2 * row) + 4 * rows,
                    flops=3 * rows * (case["hq"] + case["hkv"]) * case["rot"])
    if case["op"] == "attend":
        seen = sum(c * k + (0 if case["tree"] else k * (k + 1) // 2) for c, k in zip(ctx, n))
        return dict(bytes=2 * row * sum(c + k for c, k in zip(ctx, n)) + 4 * rows * case["hq"] * case["d"],
                    flops=4 * case["hq"] * case["d"] * seen)
    moved = sum(sum(a != b for b, a in enumerate(_accepted_path(p))) for p in _trees(case))
    return dict(bytes=4 * moved * row * case["layers"] + 16 * rows + 20 * len(n), flops=0)


# -------------------------------------------------- the definitions, 64 bits ---

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample, "accept": _exact_accept}[
        case["op"]](s)


def _slots(s, seq, count):
    """(page, place in it) of a sequence's first `count` positions."""
    page = s["case"]["page"]
    j = torch.arange(count, device="cuda")
    return s["table"][seq].long()[j // page], j % page


def _exact_append(s):
    c = s["case"]
    rot, d = c["rot"], c["d"]
    pairs = [(2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2) for i in range(rot // 2)]
    first = torch.tensor([a for a, _ in pairs], device="cuda")
    second = torch.tensor([b for _, b in pairs], device="cuda")

    def turned(x, heads):
        x = x.double().reshape(s["rows"], heads, d)
        out = x.clone()
        angle = 2.0 * math.pi * torch.remainder(s["positions"].double()[:, None] * s["turns"], 1.0)
        co, si = AMPLITUDE * torch.cos(angle)[:, None, :], AMPLITUDE * torch.sin(angle)[:, None, :]
        out[..., first] = co * x[..., first] - si * x[..., second]
        out[..., second] = si * x[..., first] + co * x[..., second]
        return out

    q, k = turned(s["q"], c["hq"]).reshape(s["rows"], -1), turned(s["k"], c["hkv"])
    v = s["v"].double().reshape(s["rows"], c["hkv"], d)
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    ctx, start = s["ctx"].tolist(), s["start"].tolist()
    for i in range(c["seqs"]):
        a, b = start[i], start[i + 1]
        page, place = _slots(s, i, ctx[i] + b - a)
        page, place = page[ctx[i]:], place[ctx[i]:]
        kp[0, page, :, place] = k[a:b]
        vp[0, page, :, place] = v[a:b]
    return dict(q=q, k=kp, v=vp)


def _exact_attend(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device="cuda")
    ctx, start = s["ctx"].tolist(), s["start"].tolist()
    for i in range(c["seqs"]):
        a, b = start[i], start[i + 1]
        n = b - a
        page, place = _slots(s, i, ctx[i] + n)
        sees = torch.ones(n, ctx[i] + n, dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            sees[:, ctx[i]:] = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        else:
            bit = torch.arange(n, device="cuda")
            sees[:, ctx[i]:] = (s["mask"][a:b].long()[:, bit // 32] >> (bit % 32)) % 2 == 1
        for h in range(hkv):
            k, v = s["k_pool"][0, page, h, place].double(), s["v_pool"][0, page, h, place].double()
            for e in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = s["q"][a:b, e * d:(e + 1) * d].double() @ k.T / math.sqrt(d)
                x[~sees] = -math.inf
                out[a:b, e] = torch.nan_to_num(torch.softmax(x, -1), nan=0.0) @ v
    return out.reshape(s["rows"], hq * d)


def _exact_sample(s):
    tokens, probs = [], []
    for i in range(s["case"]["rows"]):
        x = s["logits"][i].double()
        temperature, u = float(s["temperature"][i]), float(s["u"][i])
        order = torch.argsort(-x, stable=True)
        if temperature <= 0:
            tokens.append(int(order[0]))
            probs.append(1.0)
            continue
        k = int(s["top_k"][i])
        order = order[:k] if k > 0 else order
        w = torch.exp((x[order] - x[order[0]]) / temperature)
        p = float(s["top_p"][i])
        if p < 1:
            total = torch.cumsum(w, 0)
            enough = int(torch.searchsorted(total, p * total[-1:])[0]) + 1
            w = w[:enough]
        w = w[w >= float(s["min_p"][i])]
        total = torch.cumsum(w, 0)
        at = min(int(torch.searchsorted(total, u * total[-1:], right=True)[0]), len(w) - 1)
        tokens.append(int(order[at]))
        probs.append(float(w[at] / total[-1]))
    return dict(tokens=torch.tensor(tokens, device="cuda"),
                probs=torch.tensor(probs, dtype=torch.float64, device="cuda"))


def _exact_accept(s):
    c = s["case"]
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    ctx, start = s["ctx"].tolist(), s["start"].tolist()
    draft, parents, sampled = s["draft"].tolist(), s["parents"].tolist(), s["sampled"].tolist()
    accepted, paths, after = [], [], []
    for i in range(c["seqs"]):
        a, n = start[i], start[i + 1] - start[i]
        path, at = [0], 0
        while True:
            found = [j for j in range(at + 1, n) if parents[a + j] == at and draft[a + j] == sampled[a + at]]
            if not found:
                break
            at = found[0]
            path.append(at)
        accepted.append(len(path))
        after.append(sampled[a + at])
        paths += path + [-1] * (n - len(path))
        page, place = _slots(s, i, ctx[i] + n)
        for dst, src in enumerate(path):
            x, y = ctx[i] + src, ctx[i] + dst
            kp[:, page[y], :, place[y]] = kp[:, page[x], :, place[x]]
            vp[:, page[y], :, place[y]] = vp[:, page[x], :, place[x]]
    t = lambda v: torch.tensor(v, device="cuda")  # noqa: E731
    return dict(accepted=t(accepted), path=t(paths), next_token=t(after),
                ctx=t([x + y for x, y in zip(ctx, accepted)]), k=kp, v=vp)
