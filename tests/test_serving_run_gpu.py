"""The paged-cache calls, the sampling and the GEMVs together, as a server
runs them: two sequences decoded token by token against the fp64 oracle of the
whole stack; again with drafted trees (append, tree attention, sampling and
acceptance as one step, captured or not), against the same steps one token at
a time; and a prompt cached by q4_prefill continued by the paged calls.

Two runs that reach a position in batches of different shape differ in their
logits by the fp16 roundings of the activations on the way (2^-11 each, some
20 of them in two layers, at random: about 20^0.5 2^-11 = 2e-3 of the logits'
norm), so the logits are compared to 3e-3, and a run's tokens with what the
oracle samples from that run's own logits: the cumulated probabilities move by
as much as a flat distribution's tokens are wide, so tokens of two such runs
may differ rightly."""
import numpy as np
import pytest

import oracle
import q4synth
from helpers import dev_q4, torch_dev

torch = pytest.importorskip("torch")
import bit_quantized_gemv_q4_gb300 as q4  # noqa: E402

pytestmark = pytest.mark.gpu

D, VOCAB, PAGE, THETA = 64, 1000, 16, 1.0e6


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from bit_quantized_gemv_q4_gb300 import build
    build.build()


class Model:
    def __init__(self, seed=77):
        self.shape = q4synth.tiny_decode_shape(n_layers=2, hidden=256, q=256, kv=128, ffn=512, vocab=VOCAB)
        self.host, self.host_lm = q4synth.decode_weights(self.shape, base_seed=seed)
        self.layers = [{k: (*dev_q4(m), m.N) for k, m in d.items()} for d in self.host]
        self.lm = (*dev_q4(self.host_lm), VOCAB)
        g = np.random.default_rng(seed)
        self.emb = (g.standard_normal((VOCAB, 256)) * 0.5).astype(np.float16)
        self.demb = torch_dev(self.emb)
        self.freqs = torch.empty(D // 2, dtype=torch.int64, device="cuda")
        q4.q4_rope_frequencies(self.freqs, D, theta=THETA)
        n = q4.q4_tree_attention_workspace_bytes(D)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")


class Server:
    """Caches of two layers for S sequences, and a step over M <= 8 rows."""

    def __init__(self, model, S, max_pages=4):
        self.m, self.S = model, S
        self.n_pages = S * max_pages
        self.kp = torch.zeros(2, self.n_pages, 2, PAGE, D, dtype=torch.float16, device="cuda")
        self.vp = torch.zeros_like(self.kp)
        order = np.random.default_rng(5).permutation(self.n_pages).astype(np.int32).reshape(S, max_pages)
        self.table = torch_dev(order)
        self.ctx = torch.zeros(S, dtype=torch.int32, device="cuda")
        self.caches = [q4.PagedCache(self.kp[i], self.vp[i], self.n_pages, PAGE, 2, D, self.table, S, max_pages)
                       for i in range(2)]
        f16 = lambda *s: torch.empty(*s, dtype=torch.float16, device="cuda")  # noqa: E731
        self.qkv, self.a, self.act = f16(8, 512), f16(8, 256), f16(8, 512)
        self.logits = torch.empty(8, VOCAB, device="cuda")
        self.tokens = torch.empty(8, dtype=torch.int32, device="cuda")

    def step(self, tok, start, positions, M, mask=None, u=None):
        """Rows' tokens in, the rows' sampled tokens out (and the logits kept)."""
        m = self.m
        h = m.demb[tok[:M].long()]
        for lay, cache in zip(m.layers, self.caches):
            seg = lambda n, y, res=None, ld=0: q4.Segment(*lay[n], y=y, residual=res, ldy=ld)  # noqa: E731
            q, k, v = self.qkv[:M, :256], self.qkv[:M, 256:384], self.qkv[:M, 384:]
            q4.q4_gemv_ex([seg("q", q, ld=512), seg("k", k, ld=512), seg("v", v, ld=512)], h, M, 256, out_dtype=q4.Q4_F16,
                          rmsnorm=True)
            q4.q4_paged_append(cache, self.ctx, start, M, k, v, q=q, q_out=q, n_q_heads=4, positions=positions,
                               freqs=m.freqs, rot_dim=D)
            q4.q4_tree_attention(cache, self.ctx, start, M, q, 4, self.a, m.ws, m.ws.numel(), mask=mask,
                                 mask_words=1 if mask is not None else 0)
            h2 = torch.empty_like(h)
            q4.q4_gemv_ex([seg("o", h2, res=h)], self.a, M, 256, out_dtype=q4.Q4_F16)
            q4.q4_gemv_ex([seg("gate", self.act), seg("up", None)], h2, M, 256, out_dtype=q4.Q4_F16, mode=q4.Q4_GEMV_GLU,
                          rmsnorm=True)
            h = torch.empty_like(h2)
            q4.q4_gemv_ex([seg("down", h, res=h2)], self.act, M, 512, out_dtype=q4.Q4_F16)
        q4.q4_gemv_ex([q4.Segment(*m.lm, y=self.logits)], h, M, 256, rmsnorm=True)
        q4.q4_sample(self.logits, q4.Q4_F32, M, VOCAB, self.tokens, temperature=self.temperature, top_k=self.top_k,
                     top_p=self.top_p, u=u)

    temperature = top_k = top_p = None

    def settings(self, t, k, p):
        full = lambda v, d: torch.full((8,), v, dtype=d, device="cuda")  # noqa: E731
        self.temperature, self.top_k, self.top_p = full(t, torch.float32), full(k, torch.int32), full(p, torch.float32)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


PROMPTS = [[3, 141, 59, 26, 535], [897, 93, 238]]


def uniform(s, pos):
    return float(np.float32((s * 7919 + pos * 104729) % 9973 / 9973.0))


def plain_decode(model, n, settings):
    """Prompts as one causal step, then a token per sequence and step."""
    sv = Server(model, 2)
    sv.settings(*settings)
    flat, start = sum(PROMPTS, []), ints(0, 5, 8)
    u = torch.tensor([uniform(s, i) for s, p in enumerate(PROMPTS) for i in range(len(p))], device="cuda")
    sv.step(ints(*flat), start, None, 8, u=u)
    sv.ctx += ints(5, 3)
    last = sv.tokens[[4, 7]].clone()
    out, logits = [last.tolist()], [sv.logits[[4, 7]].cpu().numpy()]
    for _ in range(n - 1):
        pos = sv.ctx.tolist()
        sv.step(last, ints(0, 1, 2), None, 2, u=torch.tensor([uniform(s, pos[s]) for s in range(2)], device="cuda"))
        sv.ctx += 1
        last = sv.tokens[:2].clone()
        out.append(last.tolist())
        logits.append(sv.logits[:2].cpu().numpy())
    assert q4.q4_device_status() == 0
    return sv, np.array(out).T, np.stack(logits, 1)  # [2][n], [2][n][vocab]


SETTINGS = [(0.0, 0, 1.0), (0.9, 40, 0.95), (1.3, 0, 1.0)]


@pytest.mark.parametrize("settings", SETTINGS)
def test_logits_of_the_stack_against_the_oracle(settings):
    m = Model()
    _, toks, logits = plain_decode(m, 6, settings)
    for s, prompt in enumerate(PROMPTS):
        caches = [(np.zeros((2, 64, D), np.float16), np.zeros((2, 64, D), np.float16)) for _ in range(2)]
        seq = prompt + toks[s].tolist()
        for i, t in enumerate(seq[:-1]):
            ref, _, _ = oracle.decode_step_attn(m.host, m.host_lm, m.emb[t:t + 1], caches, i, D, THETA)
            j = i - len(prompt) + 1
            if j >= 0:
                got = logits[s, j].astype(np.float64)
                assert np.linalg.norm(got - ref[0]) <= 3e-3 * np.linalg.norm(ref[0]), (s, i)
                t_, k_, p_ = settings
                assert toks[s, j] == oracle.sample(logits[s, j], t_, k_, p_, 0.0, uniform(s, i))[0]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("settings", SETTINGS)
def test_drafted_trees_against_one_token_at_a_time(settings, graph):
    m = Model()
    n = 14
    _, guess, _ = plain_decode(m, n + 4, settings)  # what the drafts are made from
    sv = Server(m, 2)
    sv.settings(*settings)
    u8 = torch.tensor([uniform(s, i) for s, p in enumerate(PROMPTS) for i in range(len(p))], device="cuda")
    sv.step(ints(*sum(PROMPTS, [])), ints(0, 5, 8), None, 8, u=u8)
    sv.ctx += ints(5, 3)
    done = [[int(sv.tokens[4])], [int(sv.tokens[7])]]   # sampled tokens
    seen = [[], []]                                       # the logits behind the later ones
    # trees of 4 rows: rows 1 and 2 continue the root, row 3 continues one of them
    draft, parents, pos = ints(*[0] * 8), ints(*[0] * 8), ints(*[0] * 8)
    mask, u, start = ints(*[0] * 8), torch.zeros(8, device="cuda"), ints(0, 4, 8)
    acc, path, nxt = ints(0, 0), ints(*[0] * 8), ints(0, 0)

    def step():
        sv.step(draft, start, pos, 8, mask=mask, u=u)
        c = q4.PagedCache(sv.kp, sv.vp, sv.n_pages, PAGE, 2, D, sv.table, 2, 4)
        q4.q4_tree_accept(c, sv.ctx, start, 8, draft, parents, sv.tokens, acc, path, nxt, sv.ctx, n_layers=2,
                          layer_stride=sv.kp[0].numel())

    captured = None
    rng = np.random.default_rng(3)
    taken = 0
    t_, k_, p_ = settings
    while min(len(d) for d in done) < n:
        ctx = sv.ctx.tolist()
        toks, pars = [], []
        for s in range(2):
            ahead = guess[s, len(done[s]):len(done[s]) + 2].tolist()
            ahead += [0] * (2 - len(ahead))
            right = int(rng.integers(0, 3))  # drafted tokens that follow the guess
            par = [-1, 0, 0, int(rng.integers(1, 3))]
            tok = [done[s][-1], (ahead[0] + 1) % VOCAB, (ahead[0] + 2) % VOCAB, (ahead[1] + 1) % VOCAB]
            if right >= 1:
                tok[par[3]] = ahead[0]
            if right == 2:
                tok[3] = ahead[1]
            depth = [0, 1, 1, 2]
            sees = oracle.tree_sees(par)
            toks.append(tok)
            pars.append(par)
            draft[4 * s:4 * s + 4] = ints(*tok)
            parents[4 * s:4 * s + 4] = ints(*par)
            pos[4 * s:4 * s + 4] = ints(*[ctx[s] + x for x in depth])
            mask[4 * s:4 * s + 4] = ints(*[int(sum(1 << j for j in range(4) if r[j])) for r in sees])
            u[4 * s:4 * s + 4] = torch.tensor([uniform(s, ctx[s] + x) for x in depth], device="cuda")
        if not graph:
            step()
        else:
            if captured is None:
                keep = sv.ctx.clone()
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    step()  # warms up; what it commits is taken back (the rows are appended again)
                torch.cuda.current_stream().wait_stream(side)
                sv.ctx.copy_(keep)
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    step()
            captured.replay()
        assert q4.q4_device_status() == 0
        sampled, logits = sv.tokens.tolist(), sv.logits.cpu().numpy()
        for s in range(2):
            depth = [0, 1, 1, 2]
            for i in range(4):
                assert sampled[4 * s + i] == oracle.sample(logits[4 * s + i], t_, k_, p_, 0.0, uniform(s, ctx[s] + depth[i]))[0]
            want = oracle.tree_path(toks[s], pars[s], sampled[4 * s:4 * s + 4])
            assert acc[s] == len(want) and path[4 * s:4 * s + 4].tolist() == want + [-1] * (4 - len(want))
            assert int(nxt[s]) == sampled[4 * s + want[-1]] and int(sv.ctx[s]) == ctx[s] + len(want)
            done[s] += [toks[s][j] for j in want[1:]] + [int(nxt[s])]
            seen[s] += [logits[4 * s + j] for j in want]
            taken += len(want) - 1
    assert taken > 0  # (some drafts were right)
    # the same tokens one at a time: the logits, and the cache that is left
    plain = Server(m, 2)
    plain.settings(0.0, 0, 1.0)
    plain.step(ints(*sum(PROMPTS, [])), ints(0, 5, 8), None, 8)
    plain.ctx += ints(5, 3)
    for i in range(min(len(d) for d in done) - 1):
        plain.step(ints(done[0][i], done[1][i]), ints(0, 1, 2), None, 2)
        plain.ctx += 1
        ref = plain.logits[:2].cpu().numpy().astype(np.float64)
        for s in range(2):
            assert np.linalg.norm(seen[s][i] - ref[s]) <= 3e-3 * np.linalg.norm(ref[s]), (s, i)
    assert q4.q4_device_status() == 0
    for s in range(2):
        j = np.arange(min(int(sv.ctx[s]), int(plain.ctx[s])))
        t1, t2 = sv.table[s].cpu().numpy(), plain.table[s].cpu().numpy()
        for a, b in ((sv.kp, plain.kp), (sv.vp, plain.vp)):
            x = a.cpu().numpy()[:, t1[j // PAGE], :, j % PAGE].astype(np.float64)
            y = b.cpu().numpy()[:, t2[j // PAGE], :, j % PAGE].astype(np.float64)
            assert np.linalg.norm(x - y) <= 3e-3 * np.linalg.norm(y)


def test_prefilled_cache_continues_in_the_paged_calls():
    # q4_prefill fills contiguous caches; one page per sequence, they are a pool
    m = Model()
    max_seq = 48
    g = np.random.default_rng(9)
    prompt = [int(x) for x in g.integers(0, VOCAB, 20)]
    kc = torch.zeros(2, 1, 2, max_seq, D, dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    pos = ints(0)
    dl = [{**{k: (*dev_q4(x), x.N, x.K) for k, x in d.items()}, "k_cache": kc[i], "v_cache": vc[i]}
          for i, d in enumerate(m.host)]
    table = q4.LayerTable(dl, (*dev_q4(m.host_lm), VOCAB, 256), hidden=256, M=1, flags=q4.Q4_DECODE_ATTENTION, head_dim=D,
                          max_seq=max_seq, rope_theta=THETA, pos=pos)
    n = q4.q4_prefill_workspace_bytes(table, 16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    logits = torch.empty(1, VOCAB, device="cuda")
    h = m.demb[torch.tensor(prompt, device="cuda")]
    q4.q4_prefill(table, h, len(prompt), 16, logits, ws, n)
    sv = Server(m, 1, max_pages=1)
    sv.settings(0.0, 0, 1.0)
    sv.n_pages = 1
    sv.caches = [q4.PagedCache(kc[i], vc[i], 1, max_seq, 2, D, ints(0), 1, 1) for i in range(2)]
    sv.ctx = ints(len(prompt))
    last = torch.empty(1, dtype=torch.int32, device="cuda")
    q4.q4_sample(logits, q4.Q4_F32, 1, VOCAB, last)
    seq = prompt + [int(last)]
    sv.step(last, ints(0, 1), None, 1)
    assert q4.q4_device_status() == 0
    caches = [(np.zeros((2, 64, D), np.float16), np.zeros((2, 64, D), np.float16)) for _ in range(2)]
    for i, t in enumerate(seq):
        ref, _, _ = oracle.decode_step_attn(m.host, m.host_lm, m.emb[t:t + 1], caches, i, D, THETA)
    got = sv.logits[0].cpu().numpy().astype(np.float64)
    assert np.linalg.norm(got - ref[0]) <= 3e-3 * np.linalg.norm(ref[0])
