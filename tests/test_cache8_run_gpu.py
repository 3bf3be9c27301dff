"""The 8-bit cache's calls together, as a server runs them over two layers'
pools: drafted trees appended with norms and rotation, attended, sampled,
accepted; then attended again as single tokens.  Every step is checked against
the fp64 oracle over the cache as the GPU left it, the acceptance code by code,
and the captured step against the same calls made one by one."""
import numpy as np
import pytest

import oracle
from helpers import torch_dev, ulp16
from serving_helpers import mask_words, rand16, random_tree

torch = pytest.importorskip("torch")
import bit_quantized_gemv_q4_gb300 as q4  # noqa: E402
from test_tree_attention8_gpu import close  # noqa: E402

pytestmark = pytest.mark.gpu

S, HQ, HKV, D, PAGE, LAYERS, VOCAB, MAX_PAGES = 3, 4, 2, 64, 24, 2, 500, 6
EPS = 1e-3


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from bit_quantized_gemv_q4_gb300 import build
    build.build()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, rows):
        g = np.random.default_rng(3)
        n_pages = S * MAX_PAGES
        self.nb, self.n_pages, self.rows = -(-PAGE // 16), n_pages, rows
        self.codes = [torch.full((LAYERS, n_pages, HKV, PAGE, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.full((LAYERS, n_pages, HKV, self.nb), float("nan"), device="cuda") for _ in range(2)]
        self.table_h = g.permutation(n_pages).astype(np.int32).reshape(S, MAX_PAGES)
        self.table = torch_dev(self.table_h)
        self.weights = [(1 + 0.3 * g.standard_normal(D)).astype(np.float16) for _ in range(2)]
        self.norm = q4.HeadNorm(*[torch_dev(w) for w in self.weights], eps=EPS)
        self.freqs = torch.empty(D // 2, dtype=torch.int64, device="cuda")
        q4.q4_rope_frequencies(self.freqs, D, theta=1e4)
        self.caches = [q4.PagedCache8(self.codes[0][i], self.codes[1][i], self.scales[0][i], self.scales[1][i], n_pages, PAGE,
                                      HKV, D, self.table, S, MAX_PAGES) for i in range(LAYERS)]
        self.ctx = ints(*[0] * S)
        self.start = ints(*[0] * (S + 1))
        f16 = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
        self.q = [f16(rows, HQ * D) for _ in range(LAYERS)]
        self.k, self.v = ([f16(rows, HKV * D) for _ in range(LAYERS)] for _ in range(2))
        self.turned, self.out = ([f16(rows, HQ * D) for _ in range(LAYERS)] for _ in range(2))
        self.positions, self.mask = ints(*[0] * rows), ints(*[0] * rows)
        self.logits, self.u = torch.zeros(rows, VOCAB, device="cuda"), torch.zeros(rows, device="cuda")
        self.top_k = ints(*[20] * rows)
        self.draft, self.parents, self.sampled, self.path = (ints(*[0] * rows) for _ in range(4))
        self.accepted, self.next, self.ctx_out = (ints(*[0] * S) for _ in range(3))
        self.ws = torch.empty(q4.q4_tree_attention_workspace_bytes(D), dtype=torch.uint8, device="cuda")

    def step(self):
        for i, c in enumerate(self.caches):
            q4.q4_paged_append8(c, self.ctx, self.start, self.rows, self.k[i], self.v[i], norm=self.norm, q=self.q[i],
                                q_out=self.turned[i], n_q_heads=HQ, positions=self.positions, freqs=self.freqs, rot_dim=D)
            q4.q4_tree_attention8(c, self.ctx, self.start, self.rows, self.turned[i], HQ, self.out[i], self.ws,
                                  self.ws.numel(), mask=self.mask, mask_words=1)
        q4.q4_sample(self.logits, q4.Q4_F32, self.rows, VOCAB, self.sampled, top_k=self.top_k, u=self.u)

    def accept(self):
        whole = q4.PagedCache8(*self.codes, *self.scales, self.n_pages, PAGE, HKV, D, self.table, S, MAX_PAGES)
        q4.q4_tree_accept8(whole, self.ctx, self.start, self.rows, self.draft, self.parents, self.sampled, self.accepted,
                           self.path, self.next, self.ctx_out, n_layers=LAYERS, layer_stride=self.codes[0][0].numel(),
                           scale_stride=self.scales[0][0].numel())

    def state(self):
        return [x.cpu().numpy() for x in self.codes + self.scales]


def fill(sv, g, n):
    """Inputs of a step with trees of n rows per sequence; returns the trees."""
    rows, ctx = sum(n), sv.ctx.cpu().numpy()
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    trees = [random_tree(g, m, fan=2) for m in n]
    depth = []
    for t in trees:
        d = []
        for i, p in enumerate(t):
            d.append(0 if p < 0 else d[p] + 1)
        depth.append(d)
    put = lambda dst, x: dst[:len(x)].copy_(torch_dev(np.asarray(x)))  # noqa: E731
    put(sv.start, start)
    put(sv.positions, np.concatenate([c + np.array(d) for c, d in zip(ctx, depth)]).astype(np.int32))
    sees = [oracle.tree_sees(t) for t in trees]
    put(sv.mask, mask_words([r for m in sees for r in m], 1).view(np.int32).ravel())
    size = np.exp(g.standard_normal((rows, 1)))
    for i in range(LAYERS):
        put(sv.q[i], rand16(g, rows, HQ * D))
        put(sv.k[i], rand16(g, rows, HKV * D))
        put(sv.v[i], (rand16(g, rows, HKV * D) * size).astype(np.float16))
    put(sv.logits, (g.standard_normal((rows, VOCAB)) * 3).astype(np.float32))
    put(sv.u, g.random(rows).astype(np.float32))
    put(sv.parents, np.concatenate(trees).astype(np.int32))
    return start, trees, sees


def check_attention(sv, ctx, start, sees):
    codes_k, codes_v, ks, vs = sv.state()
    values = lambda c, s: oracle.e4m3_values(c) * np.repeat(s.astype(np.float64), 16, -1)[..., :PAGE, None]  # noqa: E731
    k, v = values(codes_k, ks), values(codes_v, vs)
    for i in range(LAYERS):
        q, out = sv.turned[i].cpu().numpy(), sv.out[i].cpu().numpy()
        for s in range(S):
            a, b = start[s], start[s + 1]
            L = ctx[s] + b - a
            full = np.concatenate([np.ones((b - a, ctx[s]), bool), sees[s]], 1)
            kk = oracle.paged_rows(k[i], sv.table_h[s], np.arange(L))
            qq = q[a:b].reshape(-1, HQ, D)
            ref, A = oracle.tree_attention(qq, kk, oracle.paged_rows(v[i], sv.table_h[s], np.arange(L)), full)
            B = np.stack([np.abs(qq[:, h].astype(np.float64)) @ np.abs(kk[:, h // (HQ // HKV)]).T for h in range(HQ)], 1)
            assert close(out[a:b].reshape(ref.shape), ref, A, B.max(-1, keepdims=True) / np.sqrt(D)).all()


def run(graph):
    """Five steps of trees; with a graph, the calls of a step captured once and replayed."""
    g = np.random.default_rng(11)
    sv = Server(24)
    log = []
    captured = None
    for turn in range(5):
        n = [int(x) for x in g.integers(1, 9, S)]
        start, trees, sees = fill(sv, g, n)
        ctx = sv.ctx.cpu().numpy().copy()
        if not graph or turn == 0:
            sv.step()  # (and once before the capture)
        else:
            if captured is None:
                torch.cuda.synchronize()
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    sv.step()
            captured.replay()
        assert q4.q4_device_status() == 0
        check_attention(sv, ctx, start, sees)
        # rows' queries: normalised and rotated
        rows = start[-1]
        turned = oracle.rope_pairs(oracle.head_norm(sv.q[0].cpu().numpy()[:rows].reshape(rows, HQ, D), sv.weights[0], EPS),
                                   sv.positions.cpu().numpy()[:rows], oracle.rope_turns(D, 1e4))
        got = sv.turned[0].cpu().numpy()[:rows].reshape(turned.shape)
        assert np.all(np.abs(got - turned) <= ulp16(turned) / 2 + 5e-6 * np.abs(turned).max())
        tokens = sv.sampled.cpu().numpy()[:rows]
        logits, u = sv.logits.cpu().numpy(), sv.u.cpu().numpy()
        assert tokens.tolist() == [oracle.sample(logits[r], top_k=20, u=float(u[r]))[0] for r in range(rows)]
        # some drafted tokens are the sampled ones
        draft = np.array([-5 - r for r in range(rows)], np.int32)
        for s in range(S):
            for j in range(1, n[s]):
                if g.random() < 0.6:
                    draft[start[s] + j] = tokens[start[s] + trees[s][j]]
        sv.draft[:rows].copy_(torch_dev(draft))
        want = sv.state()
        sv.accept()
        assert q4.q4_device_status() == 0
        paths = [oracle.tree_path(draft[start[s]:start[s + 1]], trees[s], tokens[start[s]:start[s + 1]]) for s in range(S)]
        for s in range(S):
            for i in range(2):
                oracle.cache8_accept(want[i], want[2 + i], sv.table_h[s], int(ctx[s]), n[s], paths[s])
        for x, y in zip(want, sv.state()):
            assert np.array_equal(x.view(np.uint8), y.view(np.uint8))
        assert sv.accepted.tolist() == [len(p) for p in paths]
        assert sv.ctx_out.tolist() == [int(c) + len(p) for c, p in zip(ctx, paths)]
        log += [x.tobytes() for x in sv.state()] + [sv.out[1].cpu().numpy()[:rows].tobytes()]
        sv.ctx.copy_(sv.ctx_out)
    assert min(sv.ctx.tolist()) >= 5
    return log


def test_trees_step_by_step_and_captured():
    assert run(False) == run(True)


def test_committed_tokens_read_back_and_go_on_in_an_fp16_cache():
    # the accepted rows move to an fp16 cache, where the next token sees the same values
    g = np.random.default_rng(12)
    sv = Server(24)
    start, trees, sees = fill(sv, g, [8, 5, 7])
    sv.step()
    sv.ctx += ints(8, 5, 7)  # all rows as a prompt that is kept
    n16 = [torch.zeros(sv.n_pages, HKV, PAGE, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    c16 = q4.PagedCache(*n16, sv.n_pages, PAGE, HKV, D, sv.table, S, MAX_PAGES)
    k, v = (torch.empty(20, HKV * D, dtype=torch.float16, device="cuda") for _ in range(2))
    q4.q4_paged_read8(sv.caches[0], ints(0, 0, 0), sv.start, 20, k, v)
    q4.q4_paged_append(c16, ints(0, 0, 0), sv.start, 20, k, v)
    one = ints(0, 1, 2, 3)
    q, kn, vn = (torch_dev(rand16(g, 3, h * D)) for h in (HQ, HKV, HKV))
    q4.q4_paged_append8(sv.caches[0], sv.ctx, one, 3, kn, vn)
    q4.q4_paged_read8(sv.caches[0], sv.ctx, one, 3, kn, vn)  # what the cache made of them
    q4.q4_paged_append(c16, sv.ctx, one, 3, kn, vn)
    a, b = torch.empty_like(q), torch.empty_like(q)
    q4.q4_tree_attention8(sv.caches[0], sv.ctx, one, 3, q, HQ, a, sv.ws, sv.ws.numel())
    # (a block whose scale the new token made grow has been rounded again: read it all once more)
    total = (sv.ctx + 1).tolist()
    ends = ints(0, *np.cumsum(total).tolist())
    k, v = (torch.empty(sum(total), HKV * D, dtype=torch.float16, device="cuda") for _ in range(2))
    q4.q4_paged_read8(sv.caches[0], ints(0, 0, 0), ends, sum(total), k, v)
    q4.q4_paged_append(c16, ints(0, 0, 0), ends, sum(total), k, v)
    q4.q4_tree_attention(c16, sv.ctx, one, 3, q, HQ, b, sv.ws, sv.ws.numel())
    assert q4.q4_device_status() == 0
    a, b = a.cpu().numpy().astype(np.float64), b.cpu().numpy().astype(np.float64)
    # each is within 2^-11 + 4e-5 of sum |p v| (at most the greatest value here) and a rounding of the truth
    top = v.abs().max().item()
    assert np.abs(a - b).max() <= 2 * (2.0 ** -11 + 1e-4) * top + 2.0 ** -10 * np.abs(b).max()


def test_calls_on_another_stream_and_without_rows():
    a, b = Server(24), Server(24)
    for sv in (a, b):
        fill(sv, np.random.default_rng(14), [4, 9, 2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a.step()
    with torch.cuda.stream(side):
        b.step()
    torch.cuda.synchronize()
    for x, y in zip(a.state(), b.state()):
        assert np.array_equal(x.view(np.uint8), y.view(np.uint8))
    before = a.state()
    a.start.zero_()  # nobody has a row
    a.step()
    a.accept()
    assert q4.q4_device_status() == 0
    assert a.accepted.tolist() == [0] * S and a.ctx_out.tolist() == a.ctx.tolist() and a.next.tolist() == [-1] * S
    for x, y in zip(before, a.state()):
        assert np.array_equal(x.view(np.uint8), y.view(np.uint8))
