"""GPU parity of the attention over a paged cache against the fp64 oracle:
trees, random masks, rows that see nothing, prompt chunks, batched decoding;
groups of query heads, page sizes that end inside a tile, empty sequences and
contexts, splits over many CTAs, strides; NaN and infinities where a row does
not look; graphs, streams and the cache that q4_prefill's layout makes."""
import numpy as np
import pytest

import oracle
from helpers import torch_dev, ulp16
from serving_helpers import Batch, mask_words, rand16, random_tree

torch = pytest.importorskip("torch")
import bit_quantized_gemv_q4_gb300 as q4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from bit_quantized_gemv_q4_gb300 import build
    build.build()


def workspace(d):
    n = q4.q4_tree_attention_workspace_bytes(d)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n  # NaN where nobody wrote


def seen_by(b, kind, g):
    """Per sequence, bool [n][n] over its own rows."""
    out = []
    for n in b.n:
        if kind == "causal":
            out.append(np.tril(np.ones((n, n), bool)))
        elif kind == "tree":
            out.append(oracle.tree_sees(random_tree(g, n)) if n else np.zeros((0, 0), bool))
        elif kind == "random":
            m = g.random((n, n)) < 0.3
            m[::3] = False
            out.append(m)
        else:  # nothing
            out.append(np.zeros((n, n), bool))
    return out


def expected(b, q, sees, scale=None):
    a, A = [], []
    for s in range(b.S):
        L = b.ctx[s] + b.n[s]
        full = np.concatenate([np.ones((b.n[s], b.ctx[s]), bool), sees[s]], 1)
        x, y = oracle.tree_attention(q[b.start[s]:b.start[s + 1]], b.rows_of(b.k[0], s, np.arange(L)),
                                     b.rows_of(b.v[0], s, np.arange(L)), full, scale)
        a.append(x)
        A.append(y)
    return np.concatenate(a), np.concatenate(A)


# A probability enters the product as fp16: 2^-11 of it; the scores (fp32, up
# to 128 terms of |q k| / sqrt(d) about 7 in sum) and exp2 add under 2e-5 of
# it; the sums' fp32 roundings 1e-6.  Then one fp16 rounding of the output.
def close(got, a, A):
    return np.abs(np.asarray(got, np.float64) - a) <= (2.0 ** -11 + 4e-5) * A + ulp16(a) / 2 + 1e-12


def attend(b, c, q, kind, sees, words=None, scale=0.0, ld=0, stream=None, tail=2):
    T, Hq, d = q.shape
    mask, w = None, 0
    if kind != "causal":
        w = words or max(1, -(-max(b.n) // 32))
        mask = mask_words([r for m in sees for r in m] + [np.zeros(1, bool)] * tail, w)
        mask = torch_dev(mask.view(np.int32))
    width = ld or Hq * d
    dq = torch.full((T + tail, width), float("nan"), dtype=torch.float16, device="cuda")
    dq[:T, :Hq * d] = torch_dev(q.reshape(T, -1))
    out = torch.full((T + tail, width), -5.0, dtype=torch.float16, device="cuda")
    ws, n = workspace(d)
    q4.q4_tree_attention(c, b.dctx, b.dstart, T + tail, dq, Hq, out, ws, n, mask=mask, mask_words=w, scale=scale,
                         ldq=width, ldo=width, stream=stream)
    return out


def check(out, b, q, a, A):
    T, Hq, d = q.shape
    got = out.cpu().numpy()
    ok = close(got[:T, :Hq * d].reshape(a.shape), a, A)
    assert ok.all(), (np.argwhere(~ok)[:5], np.abs(got[:T, :Hq * d].reshape(a.shape) - a)[~ok][:5])
    assert np.all(got[T:] == -5.0) and np.all(got[:, Hq * d:] == -5.0)


CASES = [
    # d, Hkv, G, page, ctx, n
    (128, 2, 2, 16, [5, 0, 130], [1, 1, 1]),
    (128, 1, 8, 64, [63, 64, 65, 1], [1, 1, 1, 1]),
    (128, 2, 1, 7, [0, 700], [5, 12]),
    (128, 2, 4, 24, [200, 31, 0], [9, 33, 64]),
    (128, 1, 5, 1, [90], [40]),
    (64, 2, 4, 16, [0, 1, 300], [8, 0, 17]),
    (64, 1, 16, 100, [129, 77], [3, 70]),
    (64, 4, 1, 64, [2000], [1]),
    (64, 3, 2, 33, [10, 20, 30, 0, 0], [0, 1, 2, 3, 0]),
    (128, 8, 2, 128, [9000], [2]),
    (128, 1, 7, 256, [513], [100]),
]


# rows per kv head around the job sizes of both kernels, pages around its boxes
CASES += [
    (128, 2, 4, 64, [260, 127, 128], [32, 32, 32]),
    (128, 1, 3, 128, [129], [43]),
    (128, 1, 1, 8, [40, 0, 900], [128, 129, 64]),
    (64, 1, 1, 32, [300, 1], [256, 257]),
    (64, 2, 8, 16, [5000], [16]),
    (128, 8, 2, 256, [3000, 20], [33, 70]),
    (128, 2, 2, 40, [1000, 255], [65, 64]),
    (64, 1, 5, 384, [11], [300]),
]


@pytest.mark.parametrize("kind", ["causal", "tree", "random", "nothing"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, kind):
    d, Hkv, G, page, ctx, n = CASES[case]
    g = np.random.default_rng(100 + case)
    b = Batch(g, ctx, n, Hkv, d, page)
    q = rand16(g, b.rows, Hkv * G, d)
    sees = seen_by(b, kind, g)
    a, A = expected(b, q, sees)
    out = attend(b, b.to_device(q4), q, kind, sees)
    assert q4.q4_device_status() == 0
    check(out, b, q, a, A)


def test_attention_scale_stride_and_more_mask_words_than_rows():
    g = np.random.default_rng(3)
    b = Batch(g, [100, 3], [20, 7], 2, 64, 16)
    q = rand16(g, b.rows, 6, 64)
    sees = seen_by(b, "tree", g)
    a, A = expected(b, q, sees, scale=0.37)
    out = attend(b, b.to_device(q4), q, "tree", sees, words=3, scale=0.37, ld=6 * 64 + 40)
    assert q4.q4_device_status() == 0
    assert np.all(np.abs(out.cpu().numpy()[:27, :384].reshape(a.shape) - a) <= (2.0 ** -11 + 2e-4) * A + ulp16(a) / 2)


def test_rows_past_the_mask_are_seen_by_nobody():
    g = np.random.default_rng(4)
    b = Batch(g, [10], [40], 1, 64, 16)
    q = rand16(g, 40, 2, 64)
    sees = [np.tril(np.ones((40, 40), bool))]
    sees[0][:, 32:] = False
    a, A = expected(b, q, sees)
    out = attend(b, b.to_device(q4), q, "tree", [s[:, :32] for s in sees], words=1)
    assert q4.q4_device_status() == 0
    check(out, b, q, a, A)


@pytest.mark.parametrize("d,G", [(128, 1), (128, 2), (64, 8), (128, 16), (64, 1)])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan, 65504.0])
def test_values_that_a_row_does_not_see_do_not_reach_it(d, G, value):
    # one branch of a tree holds infinities or NaN in its keys and values
    g = np.random.default_rng(5)
    b = Batch(g, [70, 0], [24, 11], 1, d, 16)
    for s, j in ((0, 7), (1, 4), (0, 23)):
        p = b.ctx[s] + j
        b.v[0, b.table[s, p // 16], 0, p % 16, ::5] = value
        b.k[0, b.table[s, p // 16], 0, p % 16, 3] = value
    q = rand16(g, b.rows, G, d)
    sees = seen_by(b, "tree", g)
    with np.errstate(all="ignore"):
        a, A = expected(b, q, sees)
    got = attend(b, b.to_device(q4), q, "tree", sees).cpu().numpy()[:b.rows].reshape(a.shape)
    assert q4.q4_device_status() == 0
    clean = np.concatenate([~sees[0][:, [7, 23]].any(1), ~sees[1][:, 4]])
    assert clean.any() and not clean.all()
    assert close(got[clean], a[clean], A[clean]).all()
    if value != 65504.0:  # what sees them is not finite, as in the formula
        odd = ~np.isfinite(a[~clean])
        assert (~np.isfinite(got[~clean]))[odd].all()


def test_uniform_and_dominant_scores():
    # equal keys average the values; a dominant one takes all, and probabilities
    # 2^-30 of it still count where 4000 of them stand against it
    g = np.random.default_rng(6)
    d = 128
    b = Batch(g, [4000], [1], 1, d, 64)
    b.k[np.isfinite(b.k)] = 0
    q = np.ones((1, 1, d), np.float16)
    sees = [np.ones((1, 1), bool)]
    a, A = expected(b, q, sees)
    check(attend(b, b.to_device(q4), q, "causal", sees), b, q, a, A)
    b.k[0, b.table[0, 0], 0, 0] = 1.625  # score 18.4: e^-18.4 = 2^-26.5
    a, A = expected(b, q, sees)
    check(attend(b, b.to_device(q4), q, "causal", sees), b, q, a, A)
    assert q4.q4_device_status() == 0


def test_prefill_cache_is_a_pool_of_one_page():
    g = np.random.default_rng(7)
    Hkv, d, max_seq = 4, 64, 300
    kc, vc = rand16(g, Hkv, max_seq, d), rand16(g, Hkv, max_seq, d)
    q = rand16(g, 3, 8, d)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    c = q4.PagedCache(torch_dev(kc), torch_dev(vc), 1, max_seq, Hkv, d, ints(0), 1, 1)
    out = torch.empty(3, 8 * d, dtype=torch.float16, device="cuda")
    ws, n = workspace(d)
    q4.q4_tree_attention(c, ints(250), ints(0, 3), 3, torch_dev(q.reshape(3, -1)), 8, out, ws, n)
    assert q4.q4_device_status() == 0
    sees = np.tril(np.ones((3, 253), bool), 250)
    a, A = oracle.tree_attention(q, kc[:, :253].transpose(1, 0, 2), vc[:, :253].transpose(1, 0, 2), sees)
    assert close(out.cpu().numpy().reshape(a.shape), a, A).all()


def test_bits_do_not_depend_on_the_run_or_the_stream():
    g = np.random.default_rng(8)
    b = Batch(g, [3000, 10, 777], [5, 64, 1], 2, 128, 16)
    q = rand16(g, b.rows, 8, 128)
    sees = seen_by(b, "tree", g)
    c = b.to_device(q4)
    first = attend(b, c, q, "tree", sees)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            again = attend(b, c, q, "tree", sees, stream=s)
        s.synchronize()
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))


def test_graph_replays_as_the_sequences_grow():
    g = np.random.default_rng(9)
    b = Batch(g, [500, 40, 0], [4, 4, 4], 2, 64, 16)
    q = rand16(g, 12, 4, 64)
    c = b.to_device(q4)
    dq, out = torch_dev(q.reshape(12, -1)), torch.empty(12, 256, dtype=torch.float16, device="cuda")
    ws, n = workspace(64)
    run = lambda: q4.q4_tree_attention(c, b.dctx, b.dstart, 12, dq, 4, out, ws, n)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for ctx, start in (([500, 40, 0], [0, 4, 8, 12]), ([100, 3, 0], [0, 1, 9, 12]), ([30, 30, 0], [0, 12, 12, 12])):
        use = [min(c0 + n0, x + (start[i + 1] - start[i])) for i, (c0, n0, x) in enumerate(zip([500, 40, 0], [4, 4, 4], ctx))]
        rows = [start[i + 1] - start[i] for i in range(3)]
        ctx = [u - r for u, r in zip(use, rows)]
        if min(ctx) < 0:
            continue
        b.dctx.copy_(torch.tensor(ctx, dtype=torch.int32))
        b.dstart.copy_(torch.tensor(start, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        assert q4.q4_device_status() == 0
        b.ctx, b.n, b.start = ctx, rows, np.array(start)
        a, A = expected(b, q, seen_by(b, "causal", g))
        assert close(out.cpu().numpy().reshape(a.shape), a, A).all()


def test_bad_sizes_and_pages():
    g = np.random.default_rng(10)
    for what in ("page", "ctx", "room", "order"):
        b = Batch(g, [40, 20, 9], [2, 3, 2], 1, 64, 16)
        q = rand16(g, 7, 2, 64)
        sees = seen_by(b, "causal", g)
        a, A = expected(b, q, sees)
        c = b.to_device(q4)
        keep = [0, 1, 5, 6]  # rows of the other sequences
        if what == "page":
            b.dtable[1, 0] = b.n_pages
        elif what == "ctx":
            b.dctx[1] = -1
        elif what == "room":
            b.dctx[1] = 16 * b.max_pages
        else:
            b.dstart[2] = 1  # the second sequence ends before it starts; the third would start at 1
            keep = [0, 1]
        out = attend(b, c, q, "causal", sees)
        assert q4.q4_device_status() == -7, what
        got = out.cpu().numpy()[:7].reshape(a.shape)
        if what == "order":
            assert close(got[:1], a[:1], A[:1]).all()
        else:
            assert close(got[keep], a[keep], A[keep]).all(), what
        if what in ("ctx", "room"):
            assert np.all(got[2:5] == -5.0)
        assert q4.q4_device_status() == 0


def test_many_sequences():
    g = np.random.default_rng(11)
    S = 700
    n = [int(x) for x in g.integers(0, 3, S)]
    b = Batch(g, [int(x) for x in g.integers(0, 90, S)], n, 1, 64, 16)
    q = rand16(g, b.rows, 4, 64)
    sees = seen_by(b, "causal", g)
    a, A = expected(b, q, sees)
    out = attend(b, b.to_device(q4), q, "causal", sees)
    assert q4.q4_device_status() == 0
    check(out, b, q, a, A)


def test_no_rows():
    g = np.random.default_rng(12)
    b = Batch(g, [5, 6], [1, 1], 1, 64, 16)
    c = b.to_device(q4)
    b.dstart.zero_()
    out = torch.full((2, 64), -5.0, dtype=torch.float16, device="cuda")
    ws, n = workspace(64)
    for rows in (0, 2):
        q4.q4_tree_attention(c, b.dctx, b.dstart, rows, torch.zeros_like(out), 1, out, ws, n)
        assert q4.q4_device_status() == 0
    assert bool((out == -5.0).all())


# jobs (sequence, kv head, block of rows) around the limits of the launch's forms: 14, 36, 74, and many
@pytest.mark.parametrize("S,Hkv", [(1, 14), (7, 2), (5, 3), (12, 3), (37, 1), (37, 2), (25, 3), (70, 1), (120, 3)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("G,most", [(2, 1), (3, 9)])
def test_numbers_of_jobs(S, Hkv, wide, G, most):
    g = np.random.default_rng(S * 100 + Hkv * 10 + most)
    ctx = [int(x) for x in g.integers(0, 400, S)]
    n = [int(x) for x in g.integers(0, most + 1, S)]
    n[-1] = most
    b = Batch(g, ctx, n, Hkv, 64, 16)
    if wide:  # a table for long contexts: places without a page
        b.table = np.pad(b.table, ((0, 0), (0, 9000 // 16 - b.max_pages)), constant_values=-1)
        b.max_pages = b.table.shape[1]
    q = rand16(g, b.rows, Hkv * G, 64)
    sees = seen_by(b, "tree", g)
    a, A = expected(b, q, sees)
    out = attend(b, b.to_device(q4), q, "tree", sees)
    assert q4.q4_device_status() == 0
    check(out, b, q, a, A)


# a batch for each form of the launch: clusters, the line of mma.sync jobs, tcgen05
FORMS = {
    "clusters": dict(ctx=[120, 3, 250], n=[2, 1, 2], Hkv=2, G=2, d=128, page=16),
    "line": dict(ctx=[90, 0, 300, 17, 64] * 8, n=[1, 2, 1, 3, 1] * 8, Hkv=2, G=2, d=64, page=24),
    "tcgen05": dict(ctx=[300, 0, 129], n=[40, 17, 64], Hkv=2, G=4, d=128, page=16),
}


def form(name, seed):
    f = FORMS[name]
    g = np.random.default_rng(seed)
    b = Batch(g, f["ctx"], f["n"], f["Hkv"], f["d"], f["page"])
    return g, b, rand16(g, b.rows, f["Hkv"] * f["G"], f["d"])


@pytest.mark.parametrize("name", FORMS)
def test_forms_replay_with_other_sizes(name):
    g, b, q = form(name, 21)
    T, Hq, d = q.shape
    c = b.to_device(q4)
    dq, out = torch_dev(q.reshape(T, -1)), torch.empty(T, Hq * d, dtype=torch.float16, device="cuda")
    ws, n = workspace(d)
    run = lambda: q4.q4_tree_attention(c, b.dctx, b.dstart, T, dq, Hq, out, ws, n)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    end = [x + y for x, y in zip(b.ctx, b.n)]  # positions that exist
    rng = np.random.default_rng(22)
    for turn in range(4):
        if turn == 1:
            rows = [0] * b.S  # nobody has a row
        elif turn == 2:
            rows = [0] * (b.S - 1) + [min(end[-1], T)]  # the last sequence has all it can have
        else:
            rows = [int(rng.integers(0, min(e, T // b.S) + 1)) for e in end]
        ctx = [int(rng.integers(0, e - r + 1)) for e, r in zip(end, rows)]
        b.ctx, b.n = ctx, rows
        b.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        b.dctx.copy_(torch_dev(np.array(ctx, np.int32)))
        b.dstart.copy_(torch_dev(b.start))
        out.fill_(-5.0)
        graph.replay()
        assert q4.q4_device_status() == 0
        got, R = out.cpu().numpy(), sum(rows)
        assert np.all(got[R:] == -5.0)
        if R:
            a, A = expected(b, q, seen_by(b, "causal", g))
            assert close(got[:R].reshape(a.shape), a, A).all(), turn


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("what", ["page", "ctx", "room"])
def test_forms_leave_a_bad_sequence_out(name, what):
    g, b, q = form(name, 23)
    sees = seen_by(b, "tree", g)
    c = b.to_device(q4)
    bad = b.S - 1
    if what == "page":
        b.dtable[bad, 0] = b.n_pages
    elif what == "ctx":
        b.dctx[bad] = -1
    else:
        b.dctx[bad] = b.page * b.max_pages
    rows = slice(b.start[bad], b.start[bad + 1])
    if what == "page":  # its positions read as zeros: keys and values
        first = min(b.page, b.ctx[bad])
        page = b.table[bad, 0]
        b.k[0, page, :, :first] = 0
        b.v[0, page, :, :first] = 0
    a, A = expected(b, q, sees)
    out = attend(b, c, q, "tree", sees)
    assert q4.q4_device_status() == -7
    got = out.cpu().numpy()[:b.rows].reshape(a.shape)
    ok = close(got, a, A)
    if what != "page":
        assert np.all(got[rows] == -5.0)
        ok[rows] = True
    assert ok.all()
    assert q4.q4_device_status() == 0


def test_calls_side_by_side_and_graphs_that_share_a_workspace():
    made = {}
    for name in FORMS:
        g, b, q = form(name, 25)
        T, Hq, d = q.shape
        made[name] = (b, b.to_device(q4), torch_dev(q.reshape(T, -1)), Hq, d, T)
    ws128, n128 = workspace(128)

    def call(name, out, ws, n):
        b, c, dq, Hq, d, T = made[name]
        q4.q4_tree_attention(c, b.dctx, b.dstart, T, dq, Hq, out, ws, n)

    new = lambda name: torch.empty(made[name][5], made[name][3] * made[name][4], dtype=torch.float16, device="cuda")  # noqa: E731
    alone = {}
    for name in FORMS:
        alone[name] = new(name)
        call(name, alone[name], *workspace(made[name][4]))
        torch.cuda.synchronize()
    # a workspace and a stream each, many calls in flight
    streams = {name: torch.cuda.Stream() for name in FORMS}
    spaces = {name: workspace(made[name][4]) for name in FORMS}
    outs = {name: [new(name) for _ in range(20)] for name in FORMS}
    torch.cuda.synchronize()
    for i in range(20):
        for name in FORMS:
            with torch.cuda.stream(streams[name]):
                call(name, outs[name][i], *spaces[name])
    torch.cuda.synchronize()
    assert q4.q4_device_status() == 0
    for name in FORMS:
        for o in outs[name]:
            assert torch.equal(o.view(torch.int16), alone[name].view(torch.int16)), name
    # one workspace, graphs one after another
    graphs, res = [], []
    for name in ("tcgen05", "clusters", "tcgen05"):
        out, graph = new(name), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(name, out, ws128, n128)
        graphs.append(graph)
        res.append((name, out))
    for _ in range(5):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for name, out in res:
        assert torch.equal(out.view(torch.int16), alone[name].view(torch.int16)), name


# pools of more than 2^31 elements: the pages in use lie at the far end
@pytest.mark.parametrize("page,n,G", [(64, [1, 2], 2), (64, [40, 3], 4), (48, [20, 1], 1), (7, [9, 1], 2)])
def test_pages_past_32_bit_offsets(page, n, G):
    g = np.random.default_rng(31)
    ctx, Hkv, d = [200, 77], 2, 128
    b = Batch(g, ctx, n, Hkv, d, page, spare=0)
    far = (1 << 31) // (Hkv * page * d) + 5  # pages before them
    pools = []
    for pool in (b.k, b.v):
        t = torch.empty(far + b.n_pages, Hkv, page, d, dtype=torch.float16, device="cuda")
        t[far:] = torch_dev(pool[0])
        pools.append(t)
    table = np.where(b.table >= 0, b.table + far, -1).astype(np.int32)
    dtable = torch_dev(table)
    b.dctx, b.dstart = torch_dev(np.array(ctx, np.int32)), torch_dev(b.start)
    c = q4.PagedCache(pools[0], pools[1], far + b.n_pages, page, Hkv, d, dtable, b.S, b.max_pages)
    q = rand16(g, b.rows, Hkv * G, d)
    sees = seen_by(b, "tree", g)
    a, A = expected(b, q, sees)
    out = attend(b, c, q, "tree", sees)
    assert q4.q4_device_status() == 0
    check(out, b, q, a, A)


# Infinities and NaN among the new rows' values, in every form of the launch:
# mma.sync jobs of 16, 32 and 64 rows, several to a CTA (a tile each) or shared by
# several, in pages that come by TMA and, of 7 and 12 rows, row by row; clusters;
# tcgen05 with one and two row streams.  n, ctx: from, to; wide: a table that
# rules the clusters out.
ODD = {
    "64 rows, short, pages of 7": dict(S=700, Hkv=2, G=4, n=(9, 16), ctx=(0, 40), d=64, page=7),
    "64 rows, short, pages of 12": dict(S=120, Hkv=1, G=8, n=(24, 30), ctx=(0, 30), d=128, page=12),
    "64 rows, shared": dict(S=12, Hkv=2, G=4, n=(16, 20), ctx=(300, 1500), d=128, page=7, wide=True),
    "16 rows, short": dict(S=600, Hkv=1, G=2, n=(1, 6), ctx=(0, 60), d=64, page=16),
    "16 rows, short, pages of 7": dict(S=600, Hkv=1, G=2, n=(1, 6), ctx=(0, 60), d=128, page=7),
    "32 rows, short": dict(S=600, Hkv=1, G=4, n=(5, 7), ctx=(0, 60), d=128, page=8),
    "16 rows, shared": dict(S=20, Hkv=1, G=2, n=(2, 6), ctx=(500, 2000), d=64, page=16, wide=True),
    "64 rows, clusters": dict(S=5, Hkv=2, G=4, n=(12, 16), ctx=(0, 500), d=64, page=7),
    "tcgen05, short": dict(S=170, Hkv=1, G=4, n=(9, 30), ctx=(0, 90), d=128, page=16),
    "tcgen05, two streams": dict(S=30, Hkv=2, G=4, n=(33, 60), ctx=(0, 300), d=64, page=8),
    "tcgen05, shared": dict(S=5, Hkv=1, G=4, n=(20, 50), ctx=(500, 3000), d=128, page=64),
}


@pytest.mark.parametrize("kind", ["tree", "causal"])
@pytest.mark.parametrize("name", ODD)
def test_infinities_and_nan_reach_what_sees_them_in_every_form(name, kind):
    f = ODD[name]
    g = np.random.default_rng(40 + len(name))
    draw = lambda r: [int(x) for x in g.integers(r[0], r[1] + 1, f["S"])]  # noqa: E731
    b = Batch(g, draw(f["ctx"]), draw(f["n"]), f["Hkv"], f["d"], f["page"])
    if f.get("wide"):
        b.table = np.pad(b.table, ((0, 0), (0, 9000 // b.page)), constant_values=-1)
        b.max_pages = b.table.shape[1]
    for s in range(b.S):
        for j in np.flatnonzero(g.random(b.n[s]) < 0.15):
            p = b.ctx[s] + j
            for h in range(b.Hkv):
                b.v[0, b.table[s, p // b.page], h, p % b.page, g.integers(0, b.d, 3)] = g.choice([np.inf, -np.inf, np.nan], 3)
    q = rand16(g, b.rows, b.Hkv * f["G"], b.d)
    sees = seen_by(b, kind, g)
    with np.errstate(all="ignore"):
        a, A = expected(b, q, sees)
    got = attend(b, b.to_device(q4), q, kind, sees).cpu().numpy()[:b.rows].reshape(a.shape)
    assert q4.q4_device_status() == 0
    odd = ~np.isfinite(a)
    assert odd.any() and not odd.all(axis=(1, 2)).any()
    for what in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(what(got), what(a)), (what, np.argwhere(what(got) != what(a))[:5])
    assert close(got[~odd], a[~odd], A[~odd]).all()


# Few rows among many places go to clusters, which look no further than their own
# sequence: a bad one behind it, with and without rows, is latched and left out.
@pytest.mark.parametrize("S,n,bad", [(1, {0: 1}, 0), (2, {0: 1}, 1), (40, {s: 1 for s in range(40)}, 39),
                                     (40, {s: 1 for s in range(40)}, 0), (512, {0: 1, 1: 2}, 511),
                                     (512, {0: 1, 511: 1}, 511), (300, {7: 3}, 290)])
@pytest.mark.parametrize("what", ["ctx", "room", "end"])
def test_clusters_latch_a_bad_sequence_wherever_it_stands(S, n, bad, what):
    g = np.random.default_rng(S + bad)
    rows = [n.get(s, 0) for s in range(S)]
    b = Batch(g, [int(x) for x in g.integers(1, 60, S)], rows, 1, 64, 16)
    q = rand16(g, b.rows, 2, 64)
    sees = seen_by(b, "causal", g)
    a, A = expected(b, q, sees)
    c = b.to_device(q4)
    if what == "end" and bad == S - 1:
        b.dstart[S] = b.rows + 5  # more rows than the call has (two among them that belong to nobody)
    elif what == "room":
        b.dctx[bad] = 16 * b.max_pages + 1 - rows[bad]
    else:
        b.dctx[bad] = -1
    out = attend(b, c, q, "causal", sees)
    assert q4.q4_device_status() == -7
    got = out.cpu().numpy()[:b.rows].reshape(a.shape)
    mine = slice(b.start[bad], b.start[bad + 1])
    assert np.all(got[mine] == -5.0)
    ok = close(got, a, A)
    ok[mine] = True
    assert ok.all()
    assert q4.q4_device_status() == 0


@pytest.mark.parametrize("n,G,page", [(1, 1, 64), (3, 4, 16), (20, 1, 7), (40, 2, 7), (40, 1, 64), (200, 1, 16), (9, 8, 128)])
def test_small_probabilities_beside_dominant_ones_in_every_form(n, G, page):
    # every 64th position has a score 17.0 above the others' (e^-17 = 2^-24.5) and
    # no value: what comes out is the small probabilities' share alone
    g = np.random.default_rng(44)
    b = Batch(g, [3000], [n], 1, 128, page)
    at = np.arange(3000 + n)
    where = b.table[0][at // page], 0, at % page
    b.k[0][where] = np.where(at[:, None] % 64 == 0, 1.5, 0.0)
    b.v[0][where] = np.where(at[:, None] % 64 == 0, 0.0, 4096 * (1 + g.random((3000 + n, 128))))
    q = np.ones((n, G, 128), np.float16)
    sees = seen_by(b, "causal", g)
    a, A = expected(b, q, sees)
    assert np.all(a > 2.0 ** -8)
    check(attend(b, b.to_device(q4), q, "causal", sees), b, q, a, A)
    assert q4.q4_device_status() == 0


# Batches of unlike sequences, and tables of which few places are in use: one
# kernel takes them all.
MIXED = {
    "a chunk among single tokens": dict(d=128, Hkv=1, G=4, page=16, n=[1] * 60 + [300] + [1] * 60),
    "chunks among single tokens": dict(d=64, Hkv=2, G=2, page=64, n=[1, 1, 200, 1, 130, 1, 1, 0, 17]),
    "a chunk among single tokens, pages of 7": dict(d=64, Hkv=1, G=2, page=7, n=[1] * 30 + [150] + [1] * 5),
    "trees in a table mostly idle": dict(d=128, Hkv=2, G=4, page=16, n=([0] * 30 + [61]) * 4 + [0] * 90),
    "single tokens in a table mostly idle": dict(d=64, Hkv=2, G=4, page=16, n=([0] * 60 + [1]) * 9),
    "a single token behind a chunk": dict(d=128, Hkv=1, G=8, page=32, n=[130, 1]),
}


@pytest.mark.parametrize("kind", ["causal", "random"])
@pytest.mark.parametrize("name", MIXED)
def test_unlike_sequences_and_idle_places(name, kind):
    f = MIXED[name]
    g = np.random.default_rng(60 + len(name))
    b = Batch(g, [int(x) for x in g.integers(0, 400, len(f["n"]))], f["n"], f["Hkv"], f["d"], f["page"])
    q = rand16(g, b.rows, f["Hkv"] * f["G"], f["d"])
    sees = seen_by(b, kind, g)
    a, A = expected(b, q, sees)
    out = attend(b, b.to_device(q4), q, kind, sees)
    assert q4.q4_device_status() == 0
    check(out, b, q, a, A)
