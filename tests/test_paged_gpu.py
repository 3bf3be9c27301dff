"""GPU parity of the paged append and the tree acceptance against the fp64
oracle: both rotation layouts, every way a rotated part can lie in 16-byte
chunks, scaled frequencies, far positions, strides, empty sequences, page
sizes around a row count; what is not written stays as it was, bit for bit."""
import numpy as np
import pytest

import oracle
from helpers import torch_dev, ulp16
from serving_helpers import Batch, rand16, random_tree

torch = pytest.importorskip("torch")
import bit_quantized_gemv_q4_gb300 as q4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from bit_quantized_gemv_q4_gb300 import build
    build.build()


def frequencies(rot, **kw):
    f = torch.empty(rot // 2, dtype=torch.int64, device="cuda")
    q4.q4_rope_frequencies(f, rot, **kw)
    return f


@pytest.mark.parametrize("kw", [dict(), dict(theta=1e4), dict(factor=4.0), dict(factor=8.0, orig_len=8192),
                                dict(theta=5e5, factor=32.0, orig_len=4096, alpha=1.0, beta=4.0)])
@pytest.mark.parametrize("rot", [2, 62, 128])
def test_frequencies(kw, rot):
    got = frequencies(rot, **kw).cpu().numpy().view(np.uint64).astype(np.float64) * 2.0 ** -64
    args = dict(theta=1e6)
    args.update(kw)
    want = oracle.rope_turns(rot, **args)
    # two fp64 evaluations of the same power (a few 2^-53 each), and half a 2^-64
    assert np.all(np.abs(got - want) <= 1e-14 * want + 2.0 ** -64)


def rotation_bound(x, got_pos_turns):
    """|error| of a rotated pair before its fp16 rounding, per unit of the
    pair's norm: the angle (2^-32 turns left off, 2^-31 more where the float
    of the fraction rounds: 2 pi 2^-31 together under 3e-9 ... plus the
    float's 2^-25 of a half turn, 1e-7), sincospif (2 ulp, 2.4e-7), two fp32
    products and a sum (3 x 6e-8): below 1e-6."""
    return 1e-6


@pytest.mark.parametrize("d,Hq,Hkv,rot,inter,page", [
    (128, 16, 8, 128, False, 64), (128, 4, 1, 96, False, 16), (128, 8, 2, 64, True, 7), (128, 5, 5, 50, False, 1),
    (128, 4, 2, 22, True, 100), (64, 14, 2, 64, False, 16), (64, 4, 4, 2, False, 3), (64, 8, 1, 64, True, 64),
    (64, 3, 3, 62, True, 5), (128, 2, 1, 0, False, 16), (64, 0, 2, 32, False, 16)])
@pytest.mark.parametrize("far", [0, 1_000_003])
def test_append(d, Hq, Hkv, rot, inter, page, far):
    g = np.random.default_rng(rot + d + page + far)
    b = Batch(g, [0, 13, 5, 64, 30], [3, 1, 0, 40, 9], Hkv, d, page)
    k, v, q = rand16(g, b.rows, Hkv * d), rand16(g, b.rows, Hkv * d), rand16(g, b.rows, Hq * d)
    pos = np.concatenate([c + np.arange(n) for c, n in zip(b.ctx, b.n)]).astype(np.int32)
    rotary = (g.integers(0, 50, b.rows) + far).astype(np.int32) if far else pos
    kw = dict(theta=1e4, factor=4.0, orig_len=2048)
    turns = oracle.rope_turns(rot, **kw) if rot else np.zeros(0)
    c = b.to_device(q4)
    before = b.dk.clone(), b.dv.clone()
    tail = 3  # rows behind the last sequence
    pad = lambda x: torch.cat([torch_dev(x), torch.full((tail, x.shape[1]), 7.0, dtype=torch.float16, device="cuda")])
    dq = pad(q) if Hq else None
    qo = torch.full_like(dq, -3.0) if Hq else None
    q4.q4_paged_append(c, b.dctx, b.dstart, b.rows + tail, pad(k), pad(v), q=dq, q_out=qo, n_q_heads=Hq,
                       positions=torch_dev(np.concatenate([rotary, [0] * tail]).astype(np.int32)) if far else None,
                       freqs=frequencies(rot, **kw) if rot else None, rot_dim=rot,
                       layout=q4.Q4_ROPE_INTERLEAVED if inter else q4.Q4_ROPE_HALF, amplitude=1.25)
    assert q4.q4_device_status() == 0
    norm = lambda x: np.abs(np.asarray(x, np.float64)).max(-1, keepdims=True) * 2 * 1.25

    def check(got, x):
        want = oracle.rope_pairs(x, rotary, turns, inter, 1.25)
        err = np.abs(got.astype(np.float64) - want)
        assert np.all(err <= ulp16(want) / 2 + rotation_bound(None, None) * norm(x) * 1.001), err.max()
        assert np.array_equal(got[..., rot:], x[..., rot:])

    if Hq:
        out = qo.cpu().numpy()
        check(out[:b.rows].reshape(b.rows, Hq, d), q.reshape(b.rows, Hq, d))
        assert np.all(out[b.rows:] == -3.0)
    got_k, got_v = b.dk.cpu().numpy(), b.dv.cpu().numpy()
    ks, vs = k.reshape(b.rows, Hkv, d), v.reshape(b.rows, Hkv, d)
    new_k = np.concatenate([b.rows_of(got_k[0], s, b.ctx[s] + np.arange(n)) for s, n in enumerate(b.n)])
    new_v = np.concatenate([b.rows_of(got_v[0], s, b.ctx[s] + np.arange(n)) for s, n in enumerate(b.n)])
    check(new_k, ks)
    assert np.array_equal(new_v, vs)
    # everything else is untouched
    for pool, was in ((b.dk, before[0]), (b.dv, before[1])):
        same = (pool.view(torch.int16) == was.view(torch.int16)).cpu().numpy()
        for s in range(b.S):
            p = b.ctx[s] + np.arange(b.n[s])
            same[0, b.table[s][p // page], :, p % page] = True
        assert same.all()


def test_append_rows_of_a_fused_buffer_in_place():
    # q, k and v as columns of one product's output, queries turned in place
    g = np.random.default_rng(5)
    Hq, Hkv, d = 6, 2, 64
    b = Batch(g, [10, 0], [4, 7], Hkv, d, 16)
    c = b.to_device(q4)
    w = (Hq + 2 * Hkv) * d
    qkv = rand16(g, b.rows, w)
    buf = torch_dev(qkv)
    q, k, v = buf[:, :Hq * d], buf[:, Hq * d:(Hq + Hkv) * d], buf[:, (Hq + Hkv) * d:]
    q4.q4_paged_append(c, b.dctx, b.dstart, b.rows, k, v, q=q, q_out=q, n_q_heads=Hq, freqs=frequencies(d), rot_dim=d)
    assert q4.q4_device_status() == 0
    pos = np.concatenate([10 + np.arange(4), np.arange(7)])
    want = oracle.rope_pairs(qkv[:, :Hq * d].reshape(-1, Hq, d), pos, oracle.rope_turns(d))
    got = buf.cpu().numpy()
    assert np.all(np.abs(got[:, :Hq * d].reshape(-1, Hq, d) - want) <= ulp16(want) / 2 + 1e-5)
    assert np.array_equal(got[:, Hq * d:], qkv[:, Hq * d:])
    k_new = np.concatenate([b.rows_of(b.dk.cpu().numpy()[0], 0, 10 + np.arange(4)),
                            b.rows_of(b.dk.cpu().numpy()[0], 1, np.arange(7))])
    want = oracle.rope_pairs(qkv[:, Hq * d:(Hq + Hkv) * d].reshape(-1, Hkv, d), pos, oracle.rope_turns(d))
    assert np.all(np.abs(k_new - want) <= ulp16(want) / 2 + 1e-5)


def test_append_many_sequences():
    # more sequences than one level of the row search, most of them empty
    g = np.random.default_rng(6)
    n = [int(x) for x in g.integers(0, 3, 1500)]
    n[0] = n[-1] = 0
    b = Batch(g, [int(x) for x in g.integers(0, 20, 1500)], n, 1, 64, 8)
    c = b.to_device(q4)
    k, v = rand16(g, b.rows, 64), rand16(g, b.rows, 64)
    q4.q4_paged_append(c, b.dctx, b.dstart, b.rows, torch_dev(k), torch_dev(v))
    assert q4.q4_device_status() == 0
    kc, vc = b.dk.cpu().numpy(), b.dv.cpu().numpy()
    for s in range(b.S):
        at = b.ctx[s] + np.arange(n[s])
        assert np.array_equal(b.rows_of(kc[0], s, at)[:, 0], k[b.start[s]:b.start[s + 1]])
        assert np.array_equal(b.rows_of(vc[0], s, at)[:, 0], v[b.start[s]:b.start[s + 1]])


def test_append_past_32_bit_offsets():
    # a pool of more than 2^31 elements, the row at its end
    Hkv, d, page, n_pages = 8, 128, 64, 33000
    pool = torch.empty(2, n_pages, Hkv, page, d, dtype=torch.float16, device="cuda")
    assert pool[0].numel() > 2 ** 31
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    c = q4.PagedCache(pool[0], pool[1], n_pages, page, Hkv, d, table, 1, 1)
    k = torch.randn(1, Hkv * d, dtype=torch.float16, device="cuda")
    v = torch.randn(1, Hkv * d, dtype=torch.float16, device="cuda")
    q4.q4_paged_append(c, ints(63), ints(0, 1), 1, k, v)
    assert q4.q4_device_status() == 0
    assert torch.equal(pool[0, -1, :, 63].reshape(1, -1), k) and torch.equal(pool[1, -1, :, 63].reshape(1, -1), v)
    q = torch.randn(1, Hkv * d, dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(q4.q4_tree_attention_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    mask = torch.ones(1, 1, dtype=torch.int32, device="cuda")
    pool[:, -1, :, :63] = 0
    q4.q4_tree_attention(c, ints(63), ints(0, 1), 1, q, Hkv, out, ws, ws.numel(), mask=mask, mask_words=1)
    assert q4.q4_device_status() == 0
    kk, vv = pool[0, -1].permute(1, 0, 2).cpu().numpy(), pool[1, -1].permute(1, 0, 2).cpu().numpy()
    a, A = oracle.tree_attention(q.cpu().numpy().reshape(1, Hkv, d), kk, vv, np.ones((1, 64), bool))
    assert np.all(np.abs(out.cpu().numpy().reshape(a.shape) - a) <= 5.5e-4 * A + ulp16(a))


def test_append_bad_sizes_and_pages_write_nothing():
    g = np.random.default_rng(7)
    for what in ("page", "negative page", "ctx", "room", "start", "end"):
        b = Batch(g, [4, 9], [2, 3], 2, 64, 8)
        c = b.to_device(q4)
        before_k, before_v = b.dk.clone(), b.dv.clone()
        if what == "page":
            b.dtable[1, 1] = b.n_pages      # positions 9 .. 11 of the second sequence
        elif what == "negative page":
            b.dtable[1, 1] = -5
        elif what == "ctx":
            b.dctx[1] = -1
        elif what == "room":
            b.dctx[1] = 8 * b.max_pages - 2
        elif what == "start":
            b.dstart[:] = torch_dev(np.array([0, 5, 2], np.int32))
        else:
            b.dstart[2] = 6
        k, v = rand16(g, 5, 128), rand16(g, 5, 128)
        q4.q4_paged_append(c, b.dctx, b.dstart, 5, torch_dev(k), torch_dev(v))
        assert q4.q4_device_status() == -7, what
        p = np.arange(2)
        if what not in ("start", "end"):
            kc = b.dk.cpu().numpy()
            assert np.array_equal(b.rows_of(kc[0], 0, 4 + p), k[:2].reshape(2, 2, 64))
        # nothing outside the first sequence's rows changed
        for pool, was in ((b.dk, before_k), (b.dv, before_v)):
            same = (pool.view(torch.int16) == was.view(torch.int16)).cpu().numpy()
            first = 4 + np.arange(5 if what == "start" else 2)
            first = first[first // 8 < b.max_pages]
            same[0, b.table[0][first // 8], :, first % 8] = True
            assert same.all(), what
        assert q4.q4_device_status() == 0


# -------------------------------------------------------------- acceptance ---

def run_accept(b, c, draft, parents, sampled, layers, in_place=False):
    i32 = dict(dtype=torch.int32, device="cuda")
    acc, nxt = torch.full((b.S,), -9, **i32), torch.full((b.S,), -9, **i32)
    path = torch.full((b.rows + 2,), -9, **i32)
    ctx_out = b.dctx if in_place else torch.full((b.S,), -9, **i32)
    dev = lambda x: torch_dev(np.array(list(x) + [0, 0], np.int32))
    q4.q4_tree_accept(c, b.dctx, b.dstart, b.rows + 2, dev(draft), dev(parents), dev(sampled), acc, path, nxt, ctx_out,
                      n_layers=layers, layer_stride=b.dk[0].numel())
    return acc, path, nxt, ctx_out


@pytest.mark.parametrize("Hkv,d,page,layers,n,in_place", [
    (2, 64, 8, 1, [7, 1, 0, 33], False), (1, 128, 16, 3, [64, 20, 5, 100], True), (8, 128, 1, 2, [12], False),
    (3, 64, 50, 0, [9, 9], True), (2, 64, 64, 2, [400, 3], False)])
def test_accept(Hkv, d, page, layers, n, in_place):
    g = np.random.default_rng(sum(n) + page)
    b = Batch(g, [int(x) for x in g.integers(0, 40, len(n))], n, Hkv, d, page, layers=max(1, layers))
    draft, parents, sampled, paths = [], [], [], []
    for k in n:
        par = random_tree(g, k) if k else []
        tok = [int(x) for x in g.integers(0, 3, k)]      # few tokens: long paths, siblings that share one
        smp = [int(x) for x in g.integers(-1, 3, k)]
        if k > 60:                                         # one sequence walks a whole chain
            par[1:40] = range(39)
            tok[1:40] = smp[:39] = [1] * 39
        paths.append(oracle.tree_path(tok, par, smp))
        draft += tok
        parents += par
        sampled += smp
    c = b.to_device(q4)
    acc, path, nxt, ctx_out = run_accept(b, c, draft, parents, sampled, layers, in_place)
    assert q4.q4_device_status() == 0
    assert acc.tolist() == [len(p) for p in paths]
    want_path = [x for p, k in zip(paths, n) for x in p + [-1] * (k - len(p))]
    assert path.tolist() == want_path + [-9, -9]
    assert nxt.tolist() == [sampled[b.start[s] + p[-1]] if p else -1 for s, p in enumerate(paths)]
    assert ctx_out.tolist() == [x + len(p) for x, p in zip(b.ctx, paths)]
    for pool, dev in ((b.k, b.dk), (b.v, b.dv)):
        want = pool.copy()
        for s, p in enumerate(paths):
            for i, j in enumerate(p):
                a, z = b.ctx[s] + j, b.ctx[s] + i
                if layers:
                    want[:, b.table[s, z // page], :, z % page] = pool[:, b.table[s, a // page], :, a % page]
        assert np.array_equal(dev.cpu().numpy().view(np.uint16), want.view(np.uint16))


def test_accept_bad_parents_end_and_stay_inside():
    # parents ahead of their row, below -1, far outside: such rows continue nothing
    g = np.random.default_rng(9)
    b = Batch(g, [3], [6], 1, 64, 4)
    c = b.to_device(q4)
    acc, path, nxt, _ = run_accept(b, c, [5] * 6, [-1, 1, 4, 2**31 - 1, -(2**31), 0], [5] * 6, 1)
    assert q4.q4_device_status() == 0
    assert acc.tolist() == [2] and path.tolist()[:3] == [0, 5, -1] and nxt.tolist() == [5]


def test_accept_bad_sizes_and_pages():
    g = np.random.default_rng(10)
    b = Batch(g, [3, 8], [4, 4], 1, 64, 4)
    c = b.to_device(q4)
    chain = [-1, 0, 1, 2]
    b.dctx[0] = -4
    acc, path, nxt, ctx_out = run_accept(b, c, [1] * 8, chain * 2, [1] * 8, 1)
    assert q4.q4_device_status() == -7
    assert acc.tolist() == [-9, 4] and path.tolist()[:8] == [-9] * 4 + [0, 1, 2, 3] and ctx_out.tolist() == [-9, 12]
    b.dctx[0] = 3
    b.dtable[0, 1] = b.n_pages + 7
    before = b.dk.clone()
    acc, *_ = run_accept(b, c, [1, 2, 1, 1] + [1] * 4, [-1, 0, 0, 2] + chain, [1] * 8, 1)
    assert q4.q4_device_status() == -7 and acc.tolist() == [3, 4]
    assert torch.equal(b.dk.view(torch.int16), before.view(torch.int16))
    # more rows in a sequence than a tree may have
    n = 4097
    b = Batch(g, [0, 1], [n, 2], 1, 64, 64)
    c = b.to_device(q4)
    acc, *_ = run_accept(b, c, [1] * (n + 2), [i - 1 for i in range(n)] + [-1, 0], [1] * (n + 2), 1)
    assert q4.q4_device_status() == -7 and acc.tolist() == [-9, 2]


# ---------------------------------------- which sequences and rows are whose ---

def append_rows(b, c, k, v, rows):
    """One append of k, v (its queries a copy of k, left as -3 where nobody's); the pools before it, the queries out."""
    before = b.dk.clone(), b.dv.clone()
    qo = torch.full((rows, k.shape[1]), -3.0, dtype=torch.float16, device="cuda")
    q4.q4_paged_append(c, b.dctx, b.dstart, rows, torch_dev(k), torch_dev(v), q=torch_dev(k), q_out=qo, n_q_heads=b.Hkv)
    return before, qo.cpu().numpy()


def check_stored(b, k, v, before, qo, good):
    """The rows of the sequences in `good` {s: (first row, rows)} are stored, and nothing else."""
    mine = np.zeros(len(qo), bool)
    for s, (start, n) in good.items():
        at, rows = b.ctx[s] + np.arange(n), slice(start, start + n)
        mine[rows] = True
        for dev, x in ((b.dk, k), (b.dv, v)):
            assert np.array_equal(b.rows_of(dev.cpu().numpy()[0], s, at).reshape(n, -1), x[rows]), s
    assert np.array_equal(qo[mine], k[mine]) and np.all(qo[~mine] == -3.0)
    for dev, was in ((b.dk, before[0]), (b.dv, before[1])):
        same = (dev.view(torch.int16) == was.view(torch.int16)).cpu().numpy()
        for s, (_, n) in good.items():
            at = b.ctx[s] + np.arange(n)
            same[0, b.table[s][at // b.page], :, at % b.page] = True
        assert same.all()


def test_rows_before_the_first_sequence_belong_to_nobody():
    g = np.random.default_rng(41)
    b = Batch(g, [4, 9, 0], [2, 3, 1], 2, 64, 8)
    c = b.to_device(q4)
    b.dstart += 3
    k, v = rand16(g, 11, 128), rand16(g, 11, 128)
    before, qo = append_rows(b, c, k, v, 11)
    assert q4.q4_device_status() == 0
    check_stored(b, k, v, before, qo, {0: (3, 2), 1: (5, 3), 2: (8, 1)})
    # the attention and the acceptance take the same rows
    out = torch.full((11, 128), -3.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(q4.q4_tree_attention_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    q4.q4_tree_attention(c, b.dctx, b.dstart, 11, torch_dev(k), 2, out, ws, ws.numel())
    assert q4.q4_device_status() == 0
    got = out.cpu().numpy()
    assert np.all(got[:3] == -3.0) and np.all(got[9:] == -3.0)
    kc, vc = b.dk.cpu().numpy()[0], b.dv.cpu().numpy()[0]
    for s, (ctx, n) in enumerate(zip(b.ctx, b.n)):
        at, rows = np.arange(ctx + n), slice(3 + b.start[s], 3 + b.start[s + 1])
        a, A = oracle.tree_attention(k[rows].reshape(n, 2, 64), b.rows_of(kc, s, at), b.rows_of(vc, s, at),
                                     np.tril(np.ones((n, ctx + n), bool), ctx))
        assert np.all(np.abs(got[rows].reshape(a.shape) - a) <= 5.5e-4 * A + ulp16(a))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    acc, path, nxt, ctx_out = ints(9, 9, 9), ints(*[9] * 11), ints(9, 9, 9), ints(9, 9, 9)
    q4.q4_tree_accept(c, b.dctx, b.dstart, 11, ints(*[1] * 11), ints(9, 9, 9, -1, 0, -1, 0, 1, -1, 9, 9), ints(*[1] * 11),
                      acc, path, nxt, ctx_out)
    assert q4.q4_device_status() == 0
    assert acc.tolist() == [2, 3, 1] and path.tolist() == [9, 9, 9, 0, 1, 0, 1, 2, 0, 9, 9]


@pytest.mark.parametrize("S,bad", [(3, 1), (40, 39), (700, 650), (2, 0)])
def test_append_latches_a_bad_sequence_without_rows(S, bad):
    g = np.random.default_rng(42)
    n = [1 if s < 2 else 0 for s in range(S)]
    n[bad] = 0
    b = Batch(g, [5] * S, n, 1, 64, 8)
    c = b.to_device(q4)
    b.dctx[bad] = -2
    k, v = rand16(g, b.rows, 64), rand16(g, b.rows, 64)
    before, qo = append_rows(b, c, k, v, b.rows)
    assert q4.q4_device_status() == -7
    check_stored(b, k, v, before, qo, {s: (int(b.start[s]), n[s]) for s in range(S) if n[s]})
    assert q4.q4_device_status() == 0


@pytest.mark.parametrize("S", [3, 40, 1200])
def test_append_stores_good_sequences_around_bad_ones(S):
    # ends too large, starts out of order: only the sequence concerned is left out
    g = np.random.default_rng(43)
    n = [4] * S
    b = Batch(g, [int(x) for x in g.integers(0, 20, S)], n, 1, 64, 8)
    c = b.to_device(q4)
    start = b.start.copy()
    first = [0] if S == 3 else [int(x) for x in g.choice(S // 2, S // 8, replace=False) * 2]  # (their neighbours stay)
    good = {s: (int(start[s]), 4) for s in range(S)}
    for s in first:
        start[s + 1] = 99999  # s ends behind the rows, s + 1 begins there
        good.pop(s)
        good.pop(s + 1, None)
    b.dstart.copy_(torch_dev(start))
    k, v = rand16(g, b.rows + 3, 64), rand16(g, b.rows + 3, 64)
    before, qo = append_rows(b, c, k, v, b.rows + 3)
    assert q4.q4_device_status() == -7
    check_stored(b, k, v, before, qo, good)
    assert q4.q4_device_status() == 0


def test_calls_without_rows_take_empty_tensors():
    g = np.random.default_rng(51)
    b = Batch(g, [5, 6], [0, 0], 2, 64, 16)
    c = b.to_device(q4)
    h = lambda n: torch.empty(0, n, dtype=torch.float16, device="cuda")  # noqa: E731
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    ws = torch.empty(q4.q4_tree_attention_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    q4.q4_paged_append(c, b.dctx, b.dstart, 0, h(128), h(128), q=h(256), q_out=h(256), n_q_heads=4, positions=i)
    q4.q4_tree_attention(c, b.dctx, b.dstart, 0, h(256), 4, h(256), ws, ws.numel(), mask=i, mask_words=1)
    q4.q4_sample(torch.empty(0, 99, device="cuda"), q4.Q4_F32, 0, 99, i, top_k=i)
    two = lambda: torch.full((2,), -9, dtype=torch.int32, device="cuda")  # noqa: E731
    acc, nxt, ctx_out = two(), two(), two()
    q4.q4_tree_accept(c, b.dctx, b.dstart, 0, i, i, i, acc, i, nxt, ctx_out)
    assert q4.q4_device_status() == 0
    assert acc.tolist() == [0, 0] and nxt.tolist() == [-1, -1] and ctx_out.tolist() == [5, 6]
