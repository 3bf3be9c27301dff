"""GPU parity of the attention over the 8-bit paged cache against the fp64
oracle over what the codes stand for: the fp16 attention's cases (trees, random
masks, rows that see nothing, chunks, batched decoding, every form of the
launch), blocks of unlike scales, NaN codes where a row does not look, graphs
that replay with other sizes, sequences and pages that do not fit, pools past
2^31 elements."""
import numpy as np
import pytest

import oracle
from helpers import torch_dev, ulp16
from serving_helpers import Batch8, mask_words, rand16
from test_tree_attention_gpu import CASES, FORMS, MIXED, ODD, seen_by, workspace

torch = pytest.importorskip("torch")
import bit_quantized_gemv_q4_gb300 as q4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from bit_quantized_gemv_q4_gb300 import build
    build.build()


def batch(g, ctx, n, Hkv, d, page, **kw):
    return Batch8(g, ctx, n, Hkv, d, page, spread=0.5, **kw)


def expected(b, q, sees, scale=None):
    """(a, A, B): outputs, sums of |p v|, and each row's greatest sum of |q k| times the scale."""
    a, A, B = [], [], []
    f = 1 / np.sqrt(b.d) if scale is None else scale
    for s in range(b.S):
        L, rows = b.ctx[s] + b.n[s], slice(b.start[s], b.start[s + 1])
        full = np.concatenate([np.ones((b.n[s], b.ctx[s]), bool), sees[s]], 1)
        k = b.rows_of(b.k[0], s, np.arange(L))
        x, y = oracle.tree_attention(q[rows], k, b.rows_of(b.v[0], s, np.arange(L)), full, scale)
        a.append(x)
        A.append(y)
        m = np.zeros(y.shape[:2] + (1,))
        if L:
            G = q.shape[1] // b.Hkv
            for h in range(q.shape[1]):
                m[:, h, 0] = f * np.nan_to_num(np.abs(q[rows, h].astype(np.float64)) @ np.nan_to_num(np.abs(k[:, h // G])).T).max(-1)
        B.append(m)
    return np.concatenate(a), np.concatenate(A), np.concatenate(B)


# As for the fp16 cache: a probability enters the product as fp16 (2^-11 of it),
# exp2 and the sums add under 4e-5 of it.  The scores' sums over up to 128
# elements, 16 at a time, lose at most 8 x 2^-23 of their magnitude, which moves
# a probability and the sum it is divided by: 2^-19 of B together.  Then one
# fp16 rounding of the output.
def close(got, a, A, B):
    return np.abs(np.asarray(got, np.float64) - a) <= (2.0 ** -11 + 4e-5 + 2.0 ** -19 * B) * A + ulp16(a) / 2 + 1e-12


def attend(b, c, q, kind, sees, words=None, scale=0.0, ld=0, tail=2):
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
    q4.q4_tree_attention8(c, b.dctx, b.dstart, T + tail, dq, Hq, out, ws, n, mask=mask, mask_words=w, scale=scale,
                          ldq=width, ldo=width)
    return out


def check(out, b, q, a, A, B):
    T, Hq, d = q.shape
    got = out.cpu().numpy()
    ok = close(got[:T, :Hq * d].reshape(a.shape), a, A, B)
    assert ok.all(), (np.argwhere(~ok)[:5], np.abs(got[:T, :Hq * d].reshape(a.shape) - a)[~ok][:5])
    assert np.all(got[T:] == -5.0) and np.all(got[:, Hq * d:] == -5.0)


@pytest.mark.parametrize("kind", ["causal", "tree", "random", "nothing"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, kind):
    d, Hkv, G, page, ctx, n = CASES[case]
    g = np.random.default_rng(100 + case)
    b = batch(g, ctx, n, Hkv, d, page)
    q = rand16(g, b.rows, Hkv * G, d)
    sees = seen_by(b, kind, g)
    want = expected(b, q, sees)
    out = attend(b, b.to_device(q4), q, kind, sees)
    assert q4.q4_device_status() == 0
    check(out, b, q, *want)


@pytest.mark.parametrize("page,n", [(16, [3, 1]), (7, [3, 1]), (16, [50, 40]), (64, [40, 70])])
def test_blocks_of_unlike_scales(page, n):
    # neighbouring blocks whose scales are 2^-15, 2^-3, 1 and 2^7 (the greatest that any code may have): small values
    # beside great ones
    g = np.random.default_rng(page)
    b = batch(g, [200, 77], n, 2, 128, page)
    for name in ("k", "v"):
        scales = getattr(b, name + "_scales")
        scales[...] = np.where(np.isnan(scales), np.nan, g.choice([2.0 ** -15, 2.0 ** -3, 1.0, 2.0 ** 7], scales.shape))
    b.k_scales[b.k_scales > 1] = 2.0 ** -4  # (scores that one position does not win alone)
    b.set_values()
    q = (rand16(g, b.rows, 4, 128) * np.float16(0.02)).astype(np.float16)
    sees = seen_by(b, "tree", g)
    want = expected(b, q, sees)
    out = attend(b, b.to_device(q4), q, "tree", sees)
    assert q4.q4_device_status() == 0
    check(out, b, q, *want)


def test_scale_stride_and_more_mask_words_than_rows():
    g = np.random.default_rng(3)
    b = batch(g, [100, 3], [20, 7], 2, 64, 16)
    q = rand16(g, b.rows, 6, 64)
    sees = seen_by(b, "tree", g)
    want = expected(b, q, sees, scale=0.37)
    out = attend(b, b.to_device(q4), q, "tree", sees, words=3, scale=0.37, ld=6 * 64 + 40)
    assert q4.q4_device_status() == 0
    check(out, b, q, *want)


def test_rows_past_the_mask_are_seen_by_nobody():
    g = np.random.default_rng(4)
    b = batch(g, [10], [40], 1, 64, 16)
    q = rand16(g, 40, 2, 64)
    sees = [np.tril(np.ones((40, 40), bool))]
    sees[0][:, 32:] = False
    want = expected(b, q, sees)
    out = attend(b, b.to_device(q4), q, "tree", [s[:, :32] for s in sees], words=1)
    assert q4.q4_device_status() == 0
    check(out, b, q, *want)


@pytest.mark.parametrize("kind", ["tree", "causal"])
@pytest.mark.parametrize("name", ODD)
def test_nan_reaches_what_sees_it_in_every_form(name, kind):
    f = ODD[name]
    g = np.random.default_rng(40 + len(name))
    draw = lambda r: [int(x) for x in g.integers(r[0], r[1] + 1, f["S"])]  # noqa: E731
    b = batch(g, draw(f["ctx"]), draw(f["n"]), f["Hkv"], f["d"], f["page"])
    if f.get("wide"):
        b.table = np.pad(b.table, ((0, 0), (0, 9000 // b.page)), constant_values=-1)
        b.max_pages = b.table.shape[1]
    for s in range(b.S):
        for j in np.flatnonzero(g.random(b.n[s]) < 0.15):
            p = b.ctx[s] + j
            for h in range(b.Hkv):
                b.v8[0, b.table[s, p // b.page], h, p % b.page, g.integers(0, b.d, 3)] = g.choice([0x7F, 0xFF], 3)
    b.set_values()
    q = rand16(g, b.rows, b.Hkv * f["G"], b.d)
    sees = seen_by(b, kind, g)
    with np.errstate(all="ignore"):
        a, A, B = expected(b, q, sees)
    got = attend(b, b.to_device(q4), q, kind, sees).cpu().numpy()[:b.rows].reshape(a.shape)
    assert q4.q4_device_status() == 0
    odd = np.isnan(a)
    assert odd.any() and not odd.all(axis=(1, 2)).any()
    assert np.array_equal(np.isnan(got), odd), np.argwhere(np.isnan(got) != odd)[:5]
    assert close(got, a, A, B)[~odd].all()


@pytest.mark.parametrize("d,G", [(128, 1), (128, 2), (64, 8), (128, 16), (64, 1)])
def test_keys_that_a_row_does_not_see_do_not_reach_it(d, G):
    g = np.random.default_rng(5)
    b = batch(g, [70, 0], [24, 11], 1, d, 16)
    for s, j in ((0, 7), (1, 4), (0, 23)):
        p = b.ctx[s] + j
        b.v8[0, b.table[s, p // 16], 0, p % 16, ::5] = 0x7F
        b.k8[0, b.table[s, p // 16], 0, p % 16, 3] = 0xFF
    b.set_values()
    q = rand16(g, b.rows, G, d)
    sees = seen_by(b, "tree", g)
    with np.errstate(all="ignore"):
        a, A, B = expected(b, q, sees)
    got = attend(b, b.to_device(q4), q, "tree", sees).cpu().numpy()[:b.rows].reshape(a.shape)
    assert q4.q4_device_status() == 0
    clean = np.concatenate([~sees[0][:, [7, 23]].any(1), ~sees[1][:, 4]])
    assert clean.any() and not clean.all()
    assert close(got, a, A, B)[clean].all()
    assert np.isnan(got[~clean]).all()  # a score of NaN


def test_agrees_with_the_fp16_attention_over_the_values_read_back():
    g = np.random.default_rng(8)
    b = batch(g, [700, 90], [2, 5], 2, 128, 16)
    c = b.to_device(q4)
    pool = [torch.zeros(x.shape, dtype=torch.float16, device="cuda") for x in b.d8[:2]]
    L = [x + y for x, y in zip(b.ctx, b.n)]
    start = torch_dev(np.array([0, L[0], sum(L)], np.int32))
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    k, v = (torch.empty(sum(L), 256, dtype=torch.float16, device="cuda") for _ in range(2))
    q4.q4_paged_read8(c, zero, start, sum(L), k, v)
    c16 = q4.PagedCache(*pool, b.n_pages, 16, 2, 128, b.dtable, 2, b.max_pages)
    q4.q4_paged_append(c16, zero, start, sum(L), k, v)
    q = rand16(g, 7, 8, 128)
    sees = seen_by(b, "causal", g)
    a, A, B = expected(b, q, sees)
    out = torch.empty(7, 1024, dtype=torch.float16, device="cuda")
    ws, n = workspace(128)
    q4.q4_tree_attention(c16, b.dctx, b.dstart, 7, torch_dev(q.reshape(7, -1)), 8, out, ws, n)
    assert close(out.cpu().numpy().reshape(a.shape), a, A, B).all()
    assert close(attend(b, c, q, "causal", sees).cpu().numpy()[:7].reshape(a.shape), a, A, B).all()
    assert q4.q4_device_status() == 0


def form(name, seed):
    f = FORMS[name]
    g = np.random.default_rng(seed)
    b = batch(g, f["ctx"], f["n"], f["Hkv"], f["d"], f["page"])
    return g, b, rand16(g, b.rows, f["Hkv"] * f["G"], f["d"])


@pytest.mark.parametrize("name", FORMS)
def test_forms_replay_with_other_sizes(name):
    g, b, q = form(name, 21)
    T, Hq, d = q.shape
    c = b.to_device(q4)
    dq, out = torch_dev(q.reshape(T, -1)), torch.empty(T, Hq * d, dtype=torch.float16, device="cuda")
    ws, n = workspace(d)
    run = lambda: q4.q4_tree_attention8(c, b.dctx, b.dstart, T, dq, Hq, out, ws, n)  # noqa: E731
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
            a, A, B = expected(b, q[:R], seen_by(b, "causal", g))
            assert close(got[:R].reshape(a.shape), a, A, B).all(), turn


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
    a, A, B = expected(b, q, sees)
    out = attend(b, c, q, "tree", sees)
    assert q4.q4_device_status() == -7
    got = out.cpu().numpy()[:b.rows].reshape(a.shape)
    ok = close(got, a, A, B)
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
        q4.q4_tree_attention8(c, b.dctx, b.dstart, T, dq, Hq, out, ws, n)

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
    b = batch(g, ctx, n, Hkv, d, page, spare=0)
    far = (1 << 31) // (Hkv * page * d) + 5  # pages before them
    b.to_device(q4)
    pools = []
    for x in b.d8:
        t = torch.empty((far + b.n_pages,) + tuple(x.shape[2:]), dtype=x.dtype, device="cuda")
        t[far:] = x[0]
        pools.append(t)
    table = np.where(b.table >= 0, b.table + far, -1).astype(np.int32)
    dtable = torch_dev(table)
    c = q4.PagedCache8(*pools, far + b.n_pages, page, Hkv, d, dtable, b.S, b.max_pages)
    q = rand16(g, b.rows, Hkv * G, d)
    sees = seen_by(b, "tree", g)
    want = expected(b, q, sees)
    out = attend(b, c, q, "tree", sees)
    assert q4.q4_device_status() == 0
    check(out, b, q, *want)
    # reading back, appending and accepting there
    L = b.ctx[0]
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.empty(L, Hkv * d, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    q4.q4_paged_read8(c, ints(0, 0), ints(0, L, L), L, k, v)
    assert np.array_equal(k.cpu().numpy().astype(np.float64), b.rows_of(b.k[0], 0, np.arange(L)).reshape(L, -1))
    rows = rand16(g, b.rows, Hkv * d)
    q4.q4_paged_append8(c, b.dctx, b.dstart, b.rows, torch_dev(rows), torch_dev(rows))
    got = torch.empty(b.rows, Hkv * d, dtype=torch.float16, device="cuda")
    q4.q4_paged_read8(c, b.dctx, b.dstart, b.rows, got)
    assert np.abs(got.cpu().numpy().astype(np.float64) - rows).max() <= np.abs(rows).max() * 2.0 ** -4
    last = b.n[0] - 1
    if last > 0:
        n_all = b.rows
        parents = [-1] + [0] * (b.n[0] - 1) + [-1] + [0] * (b.n[1] - 1)
        draft = list(range(n_all))
        sampled = [last] + [-1] * (n_all - 1)
        outs = [torch.empty(m, dtype=torch.int32, device="cuda") for m in (2, n_all, 2, 2)]
        q4.q4_tree_accept8(c, b.dctx, b.dstart, n_all, ints(*draft), ints(*parents), ints(*sampled), *outs)
        moved = torch.empty(2, Hkv * d, dtype=torch.float16, device="cuda")
        q4.q4_paged_read8(c, b.dctx, ints(0, 2, 2), 2, moved)
        assert torch.equal(moved[1], got[last])
    assert q4.q4_device_status() == 0


@pytest.mark.parametrize("kind", ["causal", "random"])
@pytest.mark.parametrize("name", MIXED)
def test_unlike_sequences_and_idle_places(name, kind):
    f = MIXED[name]
    g = np.random.default_rng(60 + len(name))
    b = batch(g, [int(x) for x in g.integers(0, 400, len(f["n"]))], f["n"], f["Hkv"], f["d"], f["page"])
    q = rand16(g, b.rows, f["Hkv"] * f["G"], f["d"])
    sees = seen_by(b, kind, g)
    want = expected(b, q, sees)
    out = attend(b, b.to_device(q4), q, kind, sees)
    assert q4.q4_device_status() == 0
    check(out, b, q, *want)


@pytest.mark.parametrize("n,G,page", [(1, 1, 64), (3, 4, 16), (20, 1, 7), (40, 2, 7), (40, 1, 64), (200, 1, 16), (9, 8, 128)])
def test_small_probabilities_beside_dominant_ones_in_every_form(n, G, page):
    # every 64th position has a score 17.0 above the others' (e^-17 = 2^-24.5) and
    # no value: what comes out is the small probabilities' share alone
    g = np.random.default_rng(44)
    b = batch(g, [3000], [n], 1, 128, page)
    at = np.arange(3000 + n)
    where = b.table[0][at // page], 0, at % page
    b.k_scales[0] = 1.0
    b.v_scales[0] = 16.0
    b.k8[0][where] = np.where(at[:, None] % 64 == 0, oracle.e4m3_codes(1.5), 0)
    b.v8[0][where] = np.where(at[:, None] % 64 == 0, 0, oracle.e4m3_codes(256 * (1 + 0.7 * g.random((3000 + n, 128)))))
    b.set_values()
    q = np.ones((n, G, 128), np.float16)
    sees = seen_by(b, "causal", g)
    a, A, B = expected(b, q, sees)
    assert np.all(a > 2.0 ** -8)
    check(attend(b, b.to_device(q4), q, "causal", sees), b, q, a, A, B)
    assert q4.q4_device_status() == 0


def test_bits_do_not_depend_on_the_run():
    g = np.random.default_rng(8)
    b = batch(g, [3000, 10, 777], [5, 64, 1], 2, 128, 16)
    q = rand16(g, b.rows, 8, 128)
    sees = seen_by(b, "tree", g)
    c = b.to_device(q4)
    first = attend(b, c, q, "tree", sees)
    for _ in range(5):
        assert torch.equal(first.view(torch.int16), attend(b, c, q, "tree", sees).view(torch.int16))
    assert q4.q4_device_status() == 0


def test_no_rows():
    g = np.random.default_rng(12)
    b = batch(g, [5, 6], [1, 1], 1, 64, 16)
    c = b.to_device(q4)
    b.dstart.zero_()
    out = torch.full((2, 64), -5.0, dtype=torch.float16, device="cuda")
    ws, n = workspace(64)
    for rows in (0, 2):
        q4.q4_tree_attention8(c, b.dctx, b.dstart, rows, torch.zeros_like(out), 1, out, ws, n)
        assert q4.q4_device_status() == 0
    assert bool((out == -5.0).all())


# tcgen05 jobs whose rows end in one CTA, and those that several share, with one softmax stream or two
NAN_FORMS = {
    "128 rows": dict(S=40, Hkv=2, G=4, n=(13, 30), ctx=(0, 300), d=128, page=16),
    "128 rows, heads of 64": dict(S=40, Hkv=2, G=4, n=(13, 30), ctx=(0, 300), d=64, page=16),
    "256 rows": dict(S=20, Hkv=2, G=4, n=(35, 64), ctx=(0, 300), d=128, page=48),
    "shared": dict(S=4, Hkv=1, G=4, n=(13, 64), ctx=(1500, 3000), d=128, page=32),
    "shared, heads of 64": dict(S=4, Hkv=1, G=4, n=(13, 64), ctx=(1500, 3000), d=64, page=32),
}


@pytest.mark.parametrize("name", NAN_FORMS)
def test_nan_among_every_lanes_columns_stays_in_its_column(name):
    # the columns of a row are stored by other lanes than the one that adds the NaN its row sees: every new row
    # has a NaN code in every fourth column, from another one on for each row, and every run gives the same bits
    f = NAN_FORMS[name]
    g = np.random.default_rng(50 + len(name))
    draw = lambda r: [int(x) for x in g.integers(r[0], r[1] + 1, f["S"])]  # noqa: E731
    b = batch(g, draw(f["ctx"]), draw(f["n"]), f["Hkv"], f["d"], f["page"])
    for s in range(b.S):
        for j in range(b.n[s]):
            p = b.ctx[s] + j
            b.v8[0, b.table[s, p // b.page], :, p % b.page, (j * 7 + s) % 4::4] = 0x7F if j % 2 else 0xFF
    b.set_values()
    q = rand16(g, b.rows, b.Hkv * f["G"], b.d)
    sees = [np.eye(n, dtype=bool) for n in b.n]  # a row sees itself: one column of four is NaN
    with np.errstate(all="ignore"):
        a, A, B = expected(b, q, sees)
    odd = np.isnan(a)
    assert odd.mean() == 0.25
    c = b.to_device(q4)
    first = None
    for _ in range(4):
        out = attend(b, c, q, "tree", sees)
        assert q4.q4_device_status() == 0
        first = out if first is None else first
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    got = first.cpu().numpy()[:b.rows].reshape(a.shape)
    assert np.array_equal(np.isnan(got), odd), np.argwhere(np.isnan(got) != odd)[:5]
    assert close(got, a, A, B)[~odd].all()


# every form of the launch, with a sequence of one row and no cached positions
QUERY_FORMS = {
    "clusters": dict(ctx=[120, 0, 250], n=[2, 1, 2], Hkv=2, G=2, d=128, page=16),
    "clusters, heads of 64": dict(ctx=[0, 700], n=[1, 3], Hkv=2, G=4, d=64, page=64),
    "clusters, pages of 7": dict(ctx=[120, 0, 250], n=[2, 1, 2], Hkv=2, G=2, d=128, page=7),
    "line": dict(ctx=[90, 0, 300, 17, 64] * 8, n=[1, 1, 3, 3, 1] * 8, Hkv=2, G=2, d=128, page=24),
    "line, heads of 64": dict(ctx=[90, 0, 300, 17, 64] * 8, n=[1, 1, 3, 3, 1] * 8, Hkv=2, G=5, d=64, page=12),
    "line, shared": dict(ctx=[9000, 0, 4000], n=[9, 1, 9], Hkv=2, G=4, d=128, page=16),
    "tcgen05": dict(ctx=[300, 0, 129], n=[40, 1, 64], Hkv=2, G=4, d=128, page=16),
    "tcgen05, heads of 64": dict(ctx=[300, 0, 129], n=[30, 1, 64], Hkv=2, G=4, d=64, page=7),
    "tcgen05, 256 rows": dict(ctx=[300, 0, 0], n=[140, 1, 200], Hkv=1, G=4, d=128, page=16),
    "tcgen05, shared": dict(ctx=[3000, 0], n=[40, 1], Hkv=1, G=4, d=128, page=16),
}


@pytest.mark.parametrize("kind", ["causal", "nothing"])
@pytest.mark.parametrize("name", QUERY_FORMS)
def test_queries_that_are_no_numbers_give_nan_in_every_form(name, kind):
    # an infinity whose products are all of the other sign (every score -inf), all of its own, of both signs or none
    # (a zero in each key), beside a NaN; a row of them that sees nothing gives zeros, and no other row is touched
    f = QUERY_FORMS[name]
    g = np.random.default_rng(80 + len(name))
    b = batch(g, f["ctx"], f["n"], f["Hkv"], f["d"], f["page"])
    for e, code in ((3, 0xB8), (8, 0x38), (21, 0x00)):  # -1, 1 and 0 in every key's element e
        b.k8[..., e] = code
    b.set_values()
    q = rand16(g, b.rows, f["Hkv"] * f["G"], f["d"])
    sees = seen_by(b, kind, g)
    want = expected(b, q, sees)
    odd = q.copy()
    bad = np.zeros(odd.shape[:2], bool)
    kinds = [(3, np.inf), (8, np.inf), (3, -np.inf), (8, -np.inf), (21, np.inf), (40, -np.inf), (63, np.nan), (f["d"] - 1, np.inf)]
    for i, r in enumerate(range(0, b.rows, 2)):
        for h in ((i * 3) % odd.shape[1], (i * 3 + 2) % odd.shape[1]):
            e, x = kinds[(i + h) % len(kinds)]
            odd[r, h, e], bad[r, h] = x, True
    one = b.start[b.n.index(1)]  # the sequence of one row
    odd[one, :, 3], bad[one] = np.inf, True
    out = attend(b, b.to_device(q4), odd, kind, sees)
    assert q4.q4_device_status() == 0
    got = out.cpu().numpy()[:b.rows].reshape(want[0].shape)
    looks = np.concatenate([m.any(1) | (c > 0) for m, c in zip(sees, b.ctx)])
    assert looks.any() and (kind == "causal" or not looks.all())
    assert np.isnan(got[bad & looks[:, None]]).all(), np.argwhere(~np.isnan(got).all(-1) & bad & looks[:, None])[:5]
    assert not got[~looks].any()
    assert close(got, *want)[~bad].all()


# sequences of 2^31 positions (one page, again and again): 4 units a tile of 128 positions for 16 rows, 10 (heads of
# 128) and 7 (of 64) for up to 128, 5 with the keys as they are; the first number of sequences that makes 2^31 units
@pytest.mark.parametrize("S,n,d,page", [(33, 1, 128, 1 << 22), (33, 9, 64, 1 << 22), (13, 64, 128, 8 * 499979), (19, 100, 64, 1 << 22),
                                        (26, 60, 128, 1 << 22)])
def test_calls_of_too_many_units_are_left_out(S, n, d, page):
    pages = ((1 << 31) - 128) // page
    codes = torch.zeros(1, 1, page, d, dtype=torch.uint8, device="cuda")
    scales = torch.ones(1, 1, -(-page // 16), device="cuda")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros(S, pages, dtype=torch.int32, device="cuda")
    c = q4.PagedCache8(codes, codes, scales, scales, 1, page, 1, d, table, S, pages)
    q = torch.zeros(S * n, d, dtype=torch.float16, device="cuda")
    out = torch.full_like(q, -5.0)
    ws, size = workspace(d)
    ctx = ints([page * pages - n] * S)
    q4.q4_tree_attention8(c, ctx, ints([n * i for i in range(S + 1)]), S * n, q, 1, out, ws, size)
    assert q4.q4_device_status() == -7
    assert bool((out == -5.0).all())
    # and the same call over less is computed
    ctx.fill_(5)
    q4.q4_tree_attention8(c, ctx, ints([n * i for i in range(S + 1)]), S * n, q, 1, out, ws, size)
    assert q4.q4_device_status() == 0
    assert not out.any()


@pytest.mark.parametrize("top", [2.25, 1.25])
@pytest.mark.parametrize("n,G,d,page", [(1, 2, 128, 16), (3, 4, 64, 64), (20, 4, 128, 64), (20, 4, 64, 16), (60, 4, 128, 16),
                                        (70, 4, 64, 24), (40, 2, 128, 7)])
def test_a_position_that_decides_its_row_late(n, G, d, page, top):
    # The first positions have scores of 0 (in units of log2) and no value, position 300 has `top` and a value, the others
    # next to no weight: the probability of position 300, of which 2^top / 2^12 is far from an fp16 number, decides the
    # row.  It is the row's greatest, so it enters the product as a power of two and is not rounded: what is left of
    # close()'s bound are exp2, the sums, the scores and the rounding of the output.
    g = np.random.default_rng(90)
    S = 9
    b = batch(g, [400] * S, [n] * S, 2, d, page)
    at = np.arange(400 + n)
    for s in range(S):
        where = 0, b.table[s][at // page], slice(None), at % page
        k = np.zeros((400 + n, 2, d))
        k[..., 0] = -30.0
        for h in range(2):
            k[:1 + 3 * s + h, h, 0] = 0.0
        k[300, :, 0] = top
        b.k8[where] = oracle.e4m3_codes(k)
        b.v8[where] = oracle.e4m3_codes(np.where((at < 40)[:, None, None], 0.0, 1 + g.random((400 + n, 2, d))))
    b.k_scales[...] = b.v_scales[...] = 1.0
    b.set_values()
    q = np.zeros((b.rows, 2 * G, d), np.float16)
    q[..., 0] = 1
    sees = seen_by(b, "causal", g)
    a, A, B = expected(b, q, sees, scale=np.log(2.0))
    got = attend(b, b.to_device(q4), q, "causal", sees, scale=float(np.log(2.0))).cpu().numpy()[:b.rows].reshape(a.shape)
    assert q4.q4_device_status() == 0
    ok = np.abs(got.astype(np.float64) - a) <= (4e-5 + 2.0 ** -19 * B) * A + ulp16(a) / 2
    assert ok.all(), (1 - ok.mean(), (np.abs(got - a) / a).max())
