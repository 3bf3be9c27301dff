"""Cases of the serving operators around a paged key / value cache in 8 bits
(the append that quantises, attention over it, reading it back, accepting a
drafted tree in it), and of the append that normalises queries and keys.

The cache holds e4m3 codes and an fp32 scale for each 16 positions of a page
and kv head.  ``run`` computes a case in elementary torch operations, or, where
``own`` is true, by the library's calls on the same state; ``exact`` gives the
same outputs from the definitions in 64 bits."""
import math
import random

import torch

own = False

F16, F32, F64, F8 = torch.float16, torch.float32, torch.float64, torch.float8_e4m3fn
BLOCK = 16          # positions of a page that share a scale
GREATEST = 61440.0  # 240 * 2^8: the greatest value that the cache holds


def listed():
    return [
        # One user's next token into an fp16 cache, queries and keys normalised: a launch's latency.
        dict(name="norm-token", op="norm", seqs=1, n=1, ctx=700, hq=16, hkv=8, d=128, page=64, rot=128,
             interleaved=False, norm=True),
        # Chunks of four prompts entering an fp16 cache together, queries and keys normalised.
        dict(name="norm-chunks", op="norm", seqs=4, n=2048, ctx=300, hq=32, hkv=8, d=128, page=64, rot=128,
             interleaved=False, norm=True),
        # A batch's next tokens into the 8-bit cache: blocks at every stage of filling, some of whose scales grow.
        dict(name="append8-tokens", op="append8", seqs=40, n=1, ctx=900, hq=16, hkv=8, d=128, page=64, rot=128,
             interleaved=False, norm=True),
        # Chunks of four prompts entering the 8-bit cache together, part of each head rotated in neighbouring pairs.
        dict(name="append8-chunks", op="append8", seqs=4, n=2048, ctx=300, hq=32, hkv=8, d=128, page=64, rot=64,
             interleaved=True, norm=False),
        # One user's next token over a short context.
        dict(name="attend8-token", op="attend8", seqs=1, n=1, ctx=1000, hq=16, hkv=8, d=128, page=64, tree=False),
        # Plain decoding of a batch whose contexts differ a lot: the cache's bytes are the work.
        dict(name="attend8-batch", op="attend8", seqs=48, n=1, ctx=14000, hq=32, hkv=8, d=128, page=16, tree=False),
        # Drafted trees of a batch over long contexts.
        dict(name="attend8-trees", op="attend8", seqs=8, n=61, ctx=20000, hq=32, hkv=8, d=128, page=64, tree=True),
        # A prompt's chunk after a cached prefix, two users: products, not bytes.
        dict(name="attend8-chunk", op="attend8", seqs=2, n=1024, ctx=6000, hq=32, hkv=8, d=128, page=128, tree=False),
        # The end of one user's cached prefix, read back.
        dict(name="read8-tail", op="read8", seqs=1, n=61, ctx=700, hkv=8, d=128, page=64),
        # Several users' whole prefixes, read back for another cache.
        dict(name="read8-prefixes", op="read8", seqs=12, n=4000, ctx=40, hkv=8, d=128, page=24),
        # One user's drafted tokens, every layer's cache.
        dict(name="accept8-one", op="accept8", seqs=1, n=16, ctx=40, hkv=8, d=128, page=16, layers=28),
        # A batch's drafted trees.
        dict(name="accept8-batch", op="accept8", seqs=32, n=64, ctx=60, hkv=8, d=128, page=16, layers=28),
    ]


def _spread(rng, lo, hi):
    """An integer of lo .. hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "append8", "append8", "attend8", "attend8", "attend8", "read8", "accept8"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    page = rng.choice([1, 8, 16, 24, 64, 128, 256])
    if op in ("norm", "append8"):
        seqs = _spread(rng, 1, 64)
        rot = d if rng.random() < 0.5 else 2 * rng.randint(1, d // 2)
        return dict(op=op, seqs=seqs, n=_spread(rng, 1, max(1, 8192 // seqs)), ctx=_spread(rng, 1, 1000),
                    hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, d=d, page=page, rot=rot,
                    interleaved=rng.random() < 0.5, norm=op == "norm" or rng.random() < 0.5)
    if op == "attend8":
        tree = rng.random() < 0.5
        n = _spread(rng, 1, 64 if tree else 1024)
        seqs = _spread(rng, 1, max(1, min(48, 2048 // n)))
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        # no more products and no more cached bytes than the largest listed ones
        most = min(250000 // seqs, int(1.3e11 / (4 * hq * d * n * seqs)) - n)
        return dict(op=op, seqs=seqs, n=n, ctx=_spread(rng, 1, max(2, min(60000, most))), hq=hq, hkv=hkv, d=d,
                    page=page, tree=tree)
    if op == "read8":
        seqs = _spread(rng, 1, 32)
        return dict(op=op, seqs=seqs, n=_spread(rng, 1, max(1, 40000 // seqs)), ctx=_spread(rng, 1, 1000), hkv=hkv, d=d,
                    page=page)
    return dict(op=op, seqs=_spread(rng, 1, 32), n=_spread(rng, 1, 64), ctx=_spread(rng, 1, 60), hkv=hkv, d=d,
                page=page, layers=_spread(rng, 1, 28))


# ------------------------------------------------------------------ inputs ---

THETA, AMPLITUDE, EPS = 1.0e6, 1.05, 1.0e-6


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


def _blocks(page):
    return -(-page // BLOCK)


def _cached(normal, *shape):
    """Codes and scales of a cache that a model has filled: a magnitude of its own for each head and element, and a
    token now and then that is larger than the others."""
    layers, pages, heads, page, d = shape
    x = normal(*shape, dtype=F32)
    x *= (normal(layers, 1, heads, 1, d, dtype=F32) * 0.7).exp_()
    x *= (normal(layers, pages, heads, page, 1, dtype=F32) * 0.5).exp_()
    nb = _blocks(page)
    top = torch.zeros(layers, pages, heads, nb * BLOCK, device="cuda")
    top[..., :page] = x.abs().amax(-1)
    scale = _scale_for(top.unflatten(-1, (nb, BLOCK)).amax(-1))
    x /= scale.repeat_interleave(BLOCK, -1)[..., :page, None]
    return x.to(F8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    normal = lambda *shape, dtype=F16: torch.randn(*shape, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    s = dict(case=case)
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
             longest=max(c + k for c, k in zip(ctx, n)), most=max(n))
    if case["op"] == "norm":
        s["k_pool"], s["v_pool"] = (normal(layers, n_pages, hkv, page, d) for _ in range(2))
    else:
        s["k_pool"], s["k_scales"] = _cached(normal, layers, n_pages, hkv, page, d)
        s["v_pool"], s["v_scales"] = _cached(normal, layers, n_pages, hkv, page, d)
    if case["op"] in ("norm", "append8"):
        hq = case["hq"]
        s["q"], s["k"], s["v"] = normal(rows, hq * d), normal(rows, hkv * d), normal(rows, hkv * d)
        s["k"] *= (normal(hkv * d, dtype=F32) * 0.7).exp_().half()  # elements of unlike magnitudes
        s["q_out"] = torch.empty_like(s["q"])
        s["q_weight"], s["k_weight"] = (1.0 + 0.3 * normal(d, dtype=F32)).half(), (1.0 + 0.3 * normal(d, dtype=F32)).half()
        turns = [THETA ** (-2.0 * i / case["rot"]) / (2.0 * math.pi) for i in range(case["rot"] // 2)]
        s["turns"] = torch.tensor(turns, dtype=F64, device="cuda")
        # the library's table: the same frequencies in units of 2^-64 turns (all below a half turn)
        s["freqs"] = torch.tensor([int(round(f * 2.0 ** 64)) for f in turns], dtype=torch.int64, device="cuda")
    if case["op"] == "attend8":
        s["q"] = normal(rows, case["hq"] * d)
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
        # the workspace that a program allocates once; enough for any call
        s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    if case["op"] == "read8":
        s["k_out"], s["v_out"] = (torch.empty(rows, hkv * d, dtype=F16, device="cuda") for _ in range(2))
    if case["op"] == "accept8":
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


# --------------------------------------------------------------- the passes ---

def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _own_append, "append8": _own_append, "attend8": _own_attend, "read8": _own_read,
                "accept8": _own_accept}[op](s)
    return {"norm": _plain_norm, "append8": _plain_append8, "attend8": _plain_attend, "read8": _plain_read,
            "accept8": _plain_accept}[op](s)


def _own_cache(s):
    import bit_quantized_gemv_q4_gb300 as q4
    c = s["case"]
    sizes = (s["n_pages"], c["page"], c["hkv"], c["d"], s["table"], c["seqs"], s["width"])
    if c["op"] == "norm":
        return q4, q4.PagedCache(s["k_pool"], s["v_pool"], *sizes)
    return q4, q4.PagedCache8(s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"], *sizes)


def _own_append(s):
    c = s["case"]
    q4, cache = _own_cache(s)
    call = q4.q4_paged_append_norm if c["op"] == "norm" else q4.q4_paged_append8
    call(cache, s["ctx"], s["start"], s["rows"], s["k"], s["v"],
         norm=q4.HeadNorm(s["q_weight"], s["k_weight"], EPS) if c["norm"] else None, q=s["q"], q_out=s["q_out"],
         n_q_heads=c["hq"], freqs=s["freqs"], rot_dim=c["rot"],
         layout=q4.Q4_ROPE_INTERLEAVED if c["interleaved"] else q4.Q4_ROPE_HALF, amplitude=AMPLITUDE)
    return _appended(s, s["q_out"])


def _appended(s, q):
    out = dict(q=q, k=s["k_pool"], v=s["v_pool"])
    return out if s["case"]["op"] == "norm" else dict(out, k_scales=s["k_scales"], v_scales=s["v_scales"])


def _own_attend(s):
    q4, cache = _own_cache(s)
    q4.q4_tree_attention8(cache, s["ctx"], s["start"], s["rows"], s["q"], s["case"]["hq"], s["out"], s["workspace"],
                          s["workspace"].numel(), mask=s["mask"], mask_words=s["words"])
    return s["out"]


def _own_read(s):
    q4, cache = _own_cache(s)
    q4.q4_paged_read8(cache, s["ctx"], s["start"], s["rows"], s["k_out"], s["v_out"])
    return dict(k=s["k_out"], v=s["v_out"])


def _own_accept(s):
    c = s["case"]
    q4, cache = _own_cache(s)
    q4.q4_tree_accept8(cache, s["ctx"], s["start"], s["rows"], s["draft"], s["parents"], s["sampled"], s["accepted"],
                       s["path"], s["next_token"], s["ctx_out"], n_layers=c["layers"],
                       layer_stride=s["k_pool"][0].numel(), scale_stride=s["k_scales"][0].numel())
    return dict(accepted=s["accepted"], path=s["path"], next_token=s["next_token"], ctx=s["ctx_out"], k=s["k_pool"],
                v=s["v_pool"], k_scales=s["k_scales"], v_scales=s["v_scales"])


def _rows(s):
    """Sequence of each row and the row's place in it."""
    t = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["start"][1:].long(), t, right=True)
    return seq, t - s["start"][seq]


def _place(s, seq, slot):
    """Page and place in it of a position of a sequence."""
    page = s["case"]["page"]
    return s["table"][seq, slot // page].long(), slot % page


def _scale_for(top):
    """2^e, e of -15 .. 8 the least with top <= 448 * 2^e."""
    m, e = torch.frexp(top)  # top = m * 2^e, m of [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-15, 8)
    return torch.ldexp(torch.ones_like(top), e)


def _turned(s, x, heads, weight, cos, sin):
    c = s["case"]
    rot = c["rot"]
    x = x.float().reshape(x.shape[0], heads, -1)
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    co, si = cos[:, None], sin[:, None]
    p, m = a * co - b * si, b * co + a * si
    t = torch.stack([p, m], -1).flatten(-2) if c["interleaved"] else torch.cat([p, m], -1)
    return torch.cat([t, x[..., rot:]], -1)


def _plain_rows(s):
    """Queries (rounded), keys and values (fp32) of the new rows, their sequences and positions."""
    c = s["case"]
    seq, i = _rows(s)
    slot = s["ctx"][seq] + i
    turns = slot.double()[:, None] * s["turns"]
    angle = (turns - turns.floor()) * (2.0 * math.pi)
    cos, sin = (angle.cos() * AMPLITUDE).float(), (angle.sin() * AMPLITUDE).float()
    q = _turned(s, s["q"], c["hq"], s["q_weight"], cos, sin).reshape(s["rows"], -1).half()
    k = _turned(s, s["k"], c["hkv"], s["k_weight"], cos, sin)
    return q, k, s["v"].float().reshape(s["rows"], c["hkv"], c["d"]), seq, slot


def _plain_norm(s):
    q, k, v, seq, slot = _plain_rows(s)
    at, place = _place(s, seq, slot)
    s["k_pool"][0, at, :, place] = k.half()
    s["v_pool"][0, at, :, place] = v.half()
    return _appended(s, q)


def _plain_append8(s):
    c = s["case"]
    q, k, v, seq, slot = _plain_rows(s)
    at, place = _place(s, seq, slot)
    nb = _blocks(c["page"])
    block = at * nb + place // BLOCK
    cached = slot - place % BLOCK < s["ctx"][seq]  # the block holds cached positions
    # the cached positions of the blocks that the sequences go on with
    back = torch.arange(1, BLOCK, device="cuda")
    old = s["ctx"].long()[:, None] - back
    has = (s["start"][1:] > s["start"][:-1])[:, None] & (back <= (s["ctx"].long() % c["page"] % BLOCK)[:, None])
    who, which = torch.nonzero(has, as_tuple=True)
    old_at, old_place = _place(s, who, old[who, which])
    old_block = old_at * nb + old_place // BLOCK
    for x, pool, scales in ((k, s["k_pool"], s["k_scales"]), (v, s["v_pool"], s["v_scales"])):
        x = x.clamp(-GREATEST, GREATEST)
        flat = scales[0].transpose(1, 2).reshape(-1, c["hkv"]).clone()  # [pages * blocks, heads]
        top = torch.zeros_like(flat).index_reduce_(0, block, x.abs().amax(-1), "amax")
        now = _scale_for(top[block])
        now = torch.where(cached[:, None], torch.maximum(now, flat[block]), now)
        ratio = torch.ones_like(flat)
        ratio[block] = flat[block] / now
        flat[block] = now
        scales[0] = flat.reshape(s["n_pages"], nb, -1).transpose(1, 2)
        pool[0, old_at, :, old_place] = (pool[0, old_at, :, old_place].float() * ratio[old_block][..., None]).to(F8)
        pool[0, at, :, place] = (x / now[..., None]).to(F8)
    return _appended(s, q)


def _values(s, pool, scales):
    """What layer 0 of a pool stands for, fp32."""
    return pool[0].float() * scales[0].repeat_interleave(BLOCK, -1)[..., :s["case"]["page"], None]


def _padded(s, x):
    """Rows [rows, ...] as [seqs, most, ...], zeros behind each sequence's own."""
    seq, i = _rows(s)
    out = torch.zeros(s["case"]["seqs"], s["most"], *x.shape[1:], dtype=x.dtype, device="cuda")
    out[seq, i] = x
    return out, seq, i


def _plain_attend(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    q, seq, i = _padded(s, s["q"].float().reshape(s["rows"], hkv, hq // hkv, d))
    keys = lambda pool, scales: _values(s, pool, scales)[s["table"].long()].permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :s["longest"]]  # noqa: E731
    at = torch.arange(s["longest"], device="cuda") - s["ctx"][:, None]  # place among the new rows, negative: cached
    new = (s["start"][1:] - s["start"][:-1])[:, None]
    j = at.clamp(0, s["most"] - 1)[:, None, :]
    if s["mask"] is None:
        sees = torch.arange(s["most"], device="cuda")[None, :, None] >= j
    else:
        words = _padded(s, s["mask"])[0].long()
        sees = (words.gather(2, (j // 32).expand(-1, s["most"], -1)) >> (j % 32)) & 1 == 1
    sees = (sees | (at < 0)[:, None, :]) & (at < new)[:, None, :]
    scores = torch.einsum("snhgd,shld->shgnl", q, keys(s["k_pool"], s["k_scales"])) * (1.0 / math.sqrt(d))
    scores.masked_fill_(~sees[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(top.isinf(), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    values = keys(s["v_pool"], s["v_scales"]).masked_fill_((at >= new)[:, None, :, None], 0.0)
    out = torch.einsum("shgnl,shld->snhgd", p / torch.where(total == 0, torch.ones_like(total), total), values)
    return out[seq, i].reshape(s["rows"], hq * d).half()


def _plain_read(s):
    seq, i = _rows(s)
    at, place = _place(s, seq, s["ctx"][seq] + i)
    block = place // BLOCK
    out = [(pool[0, at, :, place].float() * scales[0, at, :, block][..., None]).reshape(s["rows"], -1).half()
           for pool, scales in ((s["k_pool"], s["k_scales"]), (s["v_pool"], s["v_scales"]))]
    return dict(k=out[0], v=out[1])


def _plain_accept(s):
    c = s["case"]
    most, page = s["most"], c["page"]
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
    ctx = s["ctx"].long()[:, None]
    nb = _blocks(page)
    # every position up to the last new one, and where its row comes from
    at = torch.arange(s["longest"], device="cuda")
    there = at < ctx + new
    src = at.expand(c["seqs"], -1).clone()
    who, which = torch.nonzero((path != place) & (path >= 0), as_tuple=True)
    src[who, ctx[who, 0] + which] = ctx[who, 0] + path[who, which]
    who, dst = torch.nonzero(there, as_tuple=True)
    src = src[who, dst]
    a, a_place = _place(s, who, src)
    b, b_place = _place(s, who, dst)
    moved = (src != dst)[:, None]
    block = b * nb + b_place // BLOCK
    for pool, scales in ((s["k_pool"], s["k_scales"]), (s["v_pool"], s["v_scales"])):
        flat = scales.permute(1, 3, 0, 2).reshape(s["n_pages"] * nb, -1).clone()  # [pages * blocks, layers * heads]
        was = flat[a * nb + a_place // BLOCK]
        now = flat.clone().index_reduce_(0, block, torch.where(moved, was, torch.zeros_like(was)), "amax")
        ratio = (was / now[block]).reshape(len(a), c["layers"], -1, 1)
        scales.copy_(now.reshape(s["n_pages"], nb, c["layers"], -1).permute(2, 0, 3, 1))
        pool.permute(1, 3, 0, 2, 4)[b, b_place] = (pool.permute(1, 3, 0, 2, 4)[a, a_place].float() * ratio).to(F8)
    return dict(accepted=accepted.int(), path=path[seq, i].int(), next_token=next_token.int(),
                ctx=(s["ctx"] + accepted).int(), k=s["k_pool"], v=s["v_pool"], k_scales=s["k_scales"],
                v_scales=s["v_scales"])


# -------------------------------------------------------------------- work ---

def work(case):
    ctx, n = _sizes(case)
    rows, row = sum(n), case["hkv"] * case["d"]  # elements of a row's keys
    if case["op"] in ("norm", "append8"):
        held = 2 * row if case["op"] == "norm" else row + 4 * case["hkv"] / BLOCK
        heads = case["hq"] + case["hkv"]
        return dict(bytes=rows * (4 * case["hq"] * case["d"] + 2 * (2 * row + held)),
                    flops=rows * heads * (3 * case["rot"] + (4 * case["d"] if case["norm"] else 0)))
    held = 2 * (row + 4 * case["hkv"] / BLOCK)  # keys and values of a position
    if case["op"] == "attend8":
        seen = sum(c * k + (0 if case["tree"] else k * (k + 1) // 2) for c, k in zip(ctx, n))
        return dict(bytes=held * sum(c + k for c, k in zip(ctx, n)) + 4 * rows * case["hq"] * case["d"],
                    flops=4 * case["hq"] * case["d"] * seen)
    if case["op"] == "read8":
        return dict(bytes=rows * (held + 4 * row), flops=2 * rows * row)
    moved = sum(sum(a != b for b, a in enumerate(_accepted_path(p))) for p in _trees(case))
    return dict(bytes=2 * moved * held * case["layers"] + 16 * rows + 20 * len(n), flops=0)


# -------------------------------------------------- the definitions, 64 bits ---

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_append, "append8": _exact_append, "attend8": _exact_attend, "read8": _exact_read,
            "accept8": _exact_accept}[case["op"]](s)


def _slots(s, seq, first, count):
    """(page, place in it) of `count` positions of a sequence."""
    page = s["case"]["page"]
    j = torch.arange(first, first + count, device="cuda")
    return s["table"][seq].long()[j // page], j % page


def _code(x):
    """The e4m3 number nearest to each x of at most 448 (ties to the even one): steps of 2^-3 of its power of two."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _least_scale(top):
    e = -15
    while e < 8 and top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _exact_append(s):
    c = s["case"]
    rot, d, hkv = c["rot"], c["d"], c["hkv"]
    pairs = [(2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2) for i in range(rot // 2)]
    first = torch.tensor([a for a, _ in pairs], device="cuda")
    second = torch.tensor([b for _, b in pairs], device="cuda")
    ctx, start = s["ctx"].tolist(), s["start"].tolist()
    positions = torch.cat([torch.arange(ctx[i], ctx[i] + start[i + 1] - start[i], device="cuda") for i in range(c["seqs"])])

    def turned(x, heads, weight):
        x = x.double().reshape(s["rows"], heads, d)
        if c["norm"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * weight.double()
        out = x.clone()
        angle = 2.0 * math.pi * torch.remainder(positions.double()[:, None] * s["turns"], 1.0)
        co, si = AMPLITUDE * torch.cos(angle)[:, None, :], AMPLITUDE * torch.sin(angle)[:, None, :]
        out[..., first] = co * x[..., first] - si * x[..., second]
        out[..., second] = si * x[..., first] + co * x[..., second]
        return out

    q = turned(s["q"], c["hq"], s["q_weight"]).reshape(s["rows"], -1)
    k, v = turned(s["k"], hkv, s["k_weight"]), s["v"].double().reshape(s["rows"], hkv, d)
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    if c["op"] == "norm":
        for i in range(c["seqs"]):
            a, b = start[i], start[i + 1]
            page, place = _slots(s, i, ctx[i], b - a)
            kp[0, page, :, place] = k[a:b]
            vp[0, page, :, place] = v[a:b]
        return dict(q=q, k=kp, v=vp)
    table = s["table"].tolist()
    out = []
    for x, pool, scales in ((k, kp, s["k_scales"]), (v, vp, s["v_scales"])):
        scales = scales.double()
        old = scales[0].cpu()
        now = old.clone()
        x = x.clamp(-GREATEST, GREATEST)
        tops = x.abs().amax(-1).cpu()
        for i in range(c["seqs"]):
            n = start[i + 1] - start[i]
            p = ctx[i]
            while p < ctx[i] + n:
                place = p % c["page"]
                b = place // BLOCK
                end = min(p - place + min((b + 1) * BLOCK, c["page"]), ctx[i] + n)  # of the block's new rows
                before = p - (place - b * BLOCK)  # the block's first position
                page = table[i][p // c["page"]]
                at = start[i] + p - ctx[i]
                scale = torch.tensor([_least_scale(float(t)) for t in tops[at:at + end - p].amax(0)], dtype=F64)
                if before < p:
                    scale = torch.maximum(scale, old[page, :, b])
                    if (scale > old[page, :, b]).any():
                        lo, hi = b * BLOCK, place
                        pool[0, page, :, lo:hi] = _code(pool[0, page, :, lo:hi] * (old[page, :, b] / scale).cuda()[:, None, None])
                now[page, :, b] = scale
                pool[0, page, :, place:place + end - p] = _code(x[at:at + end - p].transpose(0, 1) / scale.cuda()[:, None, None])
                p = end
        scales[0] = now.cuda()
        out.append((pool, scales))
    return dict(q=q, k=out[0][0], v=out[1][0], k_scales=out[0][1], v_scales=out[1][1])


def _exact_values(s, pool, scales, page, h, place):
    return pool[0, page, h, place].double() * scales[0, page, h, place // BLOCK].double()[:, None]


def _exact_attend(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    out = torch.zeros(s["rows"], hq, d, dtype=F64, device="cuda")
    ctx, start = s["ctx"].tolist(), s["start"].tolist()
    for i in range(c["seqs"]):
        a, b = start[i], start[i + 1]
        n = b - a
        page, place = _slots(s, i, 0, ctx[i] + n)
        sees = torch.ones(n, ctx[i] + n, dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            sees[:, ctx[i]:] = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        else:
            bit = torch.arange(n, device="cuda")
            sees[:, ctx[i]:] = (s["mask"][a:b].long()[:, bit // 32] >> (bit % 32)) % 2 == 1
        for h in range(hkv):
            k = _exact_values(s, s["k_pool"], s["k_scales"], page, h, place)
            v = _exact_values(s, s["v_pool"], s["v_scales"], page, h, place)
            for e in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = s["q"][a:b, e * d:(e + 1) * d].double() @ k.T / math.sqrt(d)
                x[~sees] = -math.inf
                out[a:b, e] = torch.nan_to_num(torch.softmax(x, -1), nan=0.0) @ v
    return out.reshape(s["rows"], hq * d)


def _exact_read(s):
    c = s["case"]
    ctx, start = s["ctx"].tolist(), s["start"].tolist()
    out = [torch.zeros(s["rows"], c["hkv"], c["d"], dtype=F64, device="cuda") for _ in range(2)]
    for i in range(c["seqs"]):
        page, place = _slots(s, i, ctx[i], start[i + 1] - start[i])
        for h in range(c["hkv"]):
            out[0][start[i]:start[i + 1], h] = _exact_values(s, s["k_pool"], s["k_scales"], page, h, place)
            out[1][start[i]:start[i + 1], h] = _exact_values(s, s["v_pool"], s["v_scales"], page, h, place)
    return dict(k=out[0].reshape(s["rows"], -1), v=out[1].reshape(s["rows"], -1))


def _exact_accept(s):
    c = s["case"]
    kp, vp, ks, vs = (s[x].double() for x in ("k_pool", "v_pool", "k_scales", "v_scales"))
    ctx, start, table = s["ctx"].tolist(), s["start"].tolist(), s["table"].tolist()
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
        moves = {}  # (page, block) of the rows that move in: (place, source page, source place)
        where = lambda j: (table[i][j // c["page"]], j % c["page"])  # noqa: E731
        for dst, src in enumerate(path):
            if src != dst:
                page, place = where(ctx[i] + dst)
                moves.setdefault((page, place // BLOCK), []).append((place, *where(ctx[i] + src), ctx[i] + dst))
        for (page, b), rows in moves.items():
            first = rows[0][3] - (rows[0][0] - b * BLOCK)  # the block's first position
            count = min(BLOCK, c["page"] - b * BLOCK, ctx[i] + n - first)
            for pool, scales in ((kp, ks), (vp, vs)):
                come = [(place, pool[:, p, :, r].clone(), scales[:, p, :, r // BLOCK].clone()) for place, p, r, _ in rows]
                was = scales[:, page, :, b].clone()
                now = was.clone()
                for _, _, scale in come:
                    now = torch.maximum(now, scale)
                lo = b * BLOCK
                pool[:, page, :, lo:lo + count] = _code(pool[:, page, :, lo:lo + count] * (was / now)[..., None, None])
                for place, x, scale in come:
                    pool[:, page, :, place] = _code(x * (scale / now)[..., None])
                scales[:, page, :, b] = now
    t = lambda v: torch.tensor(v, device="cuda")  # noqa: E731
    return dict(accepted=t(accepted), path=t(paths), next_token=t(after),
                ctx=t([x + y for x, y in zip(ctx, accepted)]), k=kp, v=vp, k_scales=ks, v_scales=vs)
