"""GPU parity of the append with norms and of the 8-bit cache's append, reading
back and acceptance against the fp64 oracle: both rotation layouts, every way a
rotated part can lie in 16-byte chunks, blocks at every stage of filling, scales
that grow, page sizes that cut blocks short, sequences and pages that do not
fit; what is not written stays as it was, bit for bit."""
import numpy as np
import pytest

import oracle
from helpers import torch_dev, ulp16
from serving_helpers import Batch, Batch8, rand16, random_tree

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


# A head before its rounding, relative to its greatest rotated pair.  Rotation:
# under 1e-6 of the pair's norm (angle 3e-9, its float 1e-7, sincospif 2.4e-7,
# products and sum 1.8e-7).  Norm: the sum of 128 squares in 8 + 4 steps, mean,
# root, reciprocal and two products: under 20 x 2^-24 = 1.2e-6.
DELTA = 2.5e-6
AMPLITUDE = 1.25


def wanted(x, heads, d, rotary, turns, inter, norm, weight, eps):
    """(fp64 rows [rows, heads, d], their error before rounding)"""
    x = np.asarray(x, np.float64).reshape(-1, heads, d)
    y = oracle.head_norm(x, weight, eps) if norm else x
    z = oracle.rope_pairs(y, rotary, turns, inter, AMPLITUDE)
    size = np.abs(y).max(-1, keepdims=True) * 2 * AMPLITUDE
    err = np.where(np.arange(d) < 2 * len(turns), size, np.abs(y) if norm else 0.0) * DELTA
    return z, err


def step8(y, scale):
    """Half a step of e4m3 at y under a scale."""
    return scale * np.exp2(np.floor(np.log2(np.maximum(np.abs(y) / scale, 2.0 ** -6)))) * 2.0 ** -4


def check_block(y, err, values, scale, old):
    """New elements y of one block and head, what is stored for them, the block's scale, its former one or None."""
    y, top = oracle.cache8_limited(y), 0.0
    if y.size and not np.isnan(y).all():
        top = np.nanmax(np.abs(y))
    e = np.nanmax(err) if err.size else 0.0
    least, most = oracle.cache8_scale(max(0.0, top - e)), oracle.cache8_scale(top + e)  # (a border may be crossed either way)
    if old is not None:
        least, most = max(least, old), max(most, old)
    assert scale in (least, most), (scale, least, most)
    nan = np.isnan(y)
    assert np.array_equal(np.isnan(values), nan)
    ok = np.abs(values - y)[~nan] <= (step8(y, scale) + err)[~nan]
    assert ok.all(), (np.abs(values - y)[~nan][~ok][:4], y[~nan][~ok][:4], scale)


def check_append8(b, before, after, k, ek, v, rows_of_seq=None):
    """Every block that a sequence's new rows touch, and that nothing else has changed."""
    touched = [np.zeros(x.shape, bool) for x in before]
    for s in (range(b.S) if rows_of_seq is None else rows_of_seq):
        p, end = b.ctx[s], b.ctx[s] + b.n[s]
        while p < end:
            page, at = b.table[s, p // b.page], p % b.page
            lo = at // 16 * 16
            stop = min(p - at + min(lo + 16, b.page), end)
            r = slice(b.start[s] + p - b.ctx[s], b.start[s] + stop - b.ctx[s])
            a0, a1 = at, at + stop - p
            for i, (y, err) in enumerate(((k, ek), (v, np.zeros_like(v)))):
                for h in range(b.Hkv):
                    old = float(before[2 + i][0, page, h, lo // 16]) if at > lo else None
                    scale = float(after[2 + i][0, page, h, lo // 16])
                    got = oracle.e4m3_values(after[i][0, page, h, a0:a1]) * scale
                    check_block(y[r, h], err[r, h], got, scale, old)
                    if old is not None:
                        was = before[i][0, page, h, lo:at]
                        want = was if old == scale else oracle.cache8_rescale(was, old, scale)
                        assert np.array_equal(after[i][0, page, h, lo:at], want)
                touched[i][0, page, :, lo:a1] = True
                touched[2 + i][0, page, :, lo // 16] = True
            p = stop
    for x, y, t in zip(before, after, touched):
        assert np.array_equal(x[~t].view(np.uint8), y[~t].view(np.uint8))


SHAPES = [
    # d, Hq, Hkv, rot, neighbours, page
    (128, 16, 8, 128, False, 64), (128, 4, 1, 96, False, 16), (128, 8, 2, 64, True, 7), (128, 5, 5, 50, False, 1),
    (128, 4, 2, 22, True, 100), (64, 14, 2, 64, False, 16), (64, 4, 4, 2, False, 3), (64, 8, 1, 64, True, 40),
    (64, 3, 3, 62, True, 5), (128, 2, 1, 0, False, 24), (64, 0, 2, 34, False, 16), (128, 7, 3, 32, False, 33)]


def call(q4_call, b, c, q, k, v, Hq, rot, inter, rotary, norm, tail=3, q_out=None):
    pad = lambda x: torch.cat([torch_dev(x), torch.full((tail, x.shape[1]), 7.0, dtype=torch.float16, device="cuda")])
    dq = pad(q) if Hq else None
    qo = torch.full_like(dq, -3.0) if Hq else None
    q4_call(c, b.dctx, b.dstart, b.rows + tail, pad(k), pad(v), norm=norm, q=dq, q_out=qo, n_q_heads=Hq,
            positions=None if rotary is None else torch_dev(np.concatenate([rotary, [0] * tail]).astype(np.int32)),
            freqs=frequencies(rot, theta=1e4) if rot else None, rot_dim=rot,
            layout=q4.Q4_ROPE_INTERLEAVED if inter else q4.Q4_ROPE_HALF, amplitude=AMPLITUDE)
    return qo


def setup(kind, shape, ctx, n, seed, far=0, spread=True):
    d, Hq, Hkv, rot, inter, page = shape
    g = np.random.default_rng(seed)
    b = kind(g, ctx, n, Hkv, d, page)
    k, v, q = rand16(g, b.rows, Hkv * d), rand16(g, b.rows, Hkv * d), rand16(g, b.rows, Hq * d)
    if spread:  # rows of unlike size, so that scales grow and do not
        size = np.exp(g.standard_normal((b.rows, 1)) * 1.5)
        k, v = (k * size).astype(np.float16), (v * size).astype(np.float16)
    pos = np.concatenate([c + np.arange(m) for c, m in zip(b.ctx, b.n)] + [np.zeros(0)]).astype(np.int32)
    rotary = (g.integers(0, 50, b.rows) + far).astype(np.int32) if far else pos
    wq, wk = (1 + 0.4 * g.standard_normal((2, d))).astype(np.float16)
    return g, b, q, k, v, rotary, wq, wk


RAGGED = ([0, 13, 5, 64, 30, 17], [3, 1, 0, 40, 9, 1])


def check_q(qo, q, b, Hq, d, rotary, turns, inter, norm, wq, eps):
    if not Hq:
        return
    out = qo.cpu().numpy()
    want, err = wanted(q, Hq, d, rotary, turns, inter, norm, wq, eps)
    assert np.all(np.abs(out[:b.rows].reshape(want.shape) - want) <= ulp16(want) / 2 + err)
    assert np.all(out[b.rows:] == -3.0)


@pytest.mark.parametrize("norms", [(True, True), (True, False), (False, True), (False, False), None])
@pytest.mark.parametrize("shape", SHAPES)
def test_append_norm(shape, norms):
    d, Hq, Hkv, rot, inter, page = shape
    far = 1_000_003 if norms == (True, False) else 0
    g, b, q, k, v, rotary, wq, wk = setup(Batch, shape, *RAGGED, seed=rot + d + page, far=far)
    eps = 1e-3
    qn, kn = norms or (False, False)
    norm = None
    if norms:
        if norms == (True, True):
            norm = q4.HeadNorm(torch_dev(wq), torch_dev(wk), eps)
        else:  # no weights: ones
            wq = wk = None
            norm = q4.HeadNorm(None, None, eps, q=qn, k=kn)
    c = b.to_device(q4)
    before = b.dk.clone(), b.dv.clone()
    qo = call(q4.q4_paged_append_norm, b, c, q, k, v, Hq, rot, inter, rotary if far else None, norm)
    assert q4.q4_device_status() == 0
    turns = oracle.rope_turns(rot, 1e4) if rot else np.zeros(0)
    check_q(qo, q, b, Hq, d, rotary, turns, inter, qn, wq, eps)
    want, err = wanted(k, Hkv, d, rotary, turns, inter, kn, wk, eps)
    got_k, got_v = b.dk.cpu().numpy(), b.dv.cpu().numpy()
    at = [b.ctx[s] + np.arange(m) for s, m in enumerate(b.n)]
    new_k = np.concatenate([b.rows_of(got_k[0], s, p) for s, p in enumerate(at)])
    new_v = np.concatenate([b.rows_of(got_v[0], s, p) for s, p in enumerate(at)])
    assert np.all(np.abs(new_k.astype(np.float64) - want) <= ulp16(want) / 2 + err)
    assert np.array_equal(new_v, v.reshape(new_v.shape))
    for pool, was in ((b.dk, before[0]), (b.dv, before[1])):
        same = (pool.view(torch.int16) == was.view(torch.int16)).cpu().numpy()
        for s, p in enumerate(at):
            same[0, b.table[s][p // page], :, p % page] = True
        assert same.all()


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_append8(shape, norm):
    d, Hq, Hkv, rot, inter, page = shape
    far = 0 if norm else 1_000_003
    g, b, q, k, v, rotary, wq, wk = setup(Batch8, shape, *RAGGED, seed=rot + d + page, far=far)
    c = b.to_device(q4)
    before = b.from_device()
    qo = call(q4.q4_paged_append8, b, c, q, k, v, Hq, rot, inter, rotary if far else None,
              q4.HeadNorm(torch_dev(wq), torch_dev(wk), 1e-3) if norm else None)
    assert q4.q4_device_status() == 0
    turns = oracle.rope_turns(rot, 1e4) if rot else np.zeros(0)
    check_q(qo, q, b, Hq, d, rotary, turns, inter, norm, wq, 1e-3)
    want, err = wanted(k, Hkv, d, rotary, turns, inter, norm, wk, 1e-3)
    check_append8(b, before, b.from_device(), want, err, v.reshape(want.shape).astype(np.float64))


@pytest.mark.parametrize("ctx,n", [
    ([3, 0, 100], [500, 11, 30]), ([7] * 300, [1, 2, 0] * 100), ([11, 250], [1500, 700]), ([15, 16, 17, 1], [520, 513, 512, 600])])
@pytest.mark.parametrize("page", [16, 24, 64, 5])
def test_append8_many_rows(ctx, n, page):
    # every size of a window of rows, runs that begin in one window and end in the next
    shape = (64, 2, 1, 64, False, page)
    g, b, q, k, v, rotary, wq, wk = setup(Batch8, shape, ctx, n, seed=page + len(ctx))
    c = b.to_device(q4)
    before = b.from_device()
    qo = call(q4.q4_paged_append8, b, c, q, k, v, 2, 64, False, None, q4.HeadNorm(torch_dev(wq), torch_dev(wk), 1e-3))
    assert q4.q4_device_status() == 0
    turns = oracle.rope_turns(64, 1e4)
    check_q(qo, q, b, 2, 64, rotary, turns, False, True, wq, 1e-3)
    want, err = wanted(k, 1, 64, rotary, turns, False, True, wk, 1e-3)
    check_append8(b, before, b.from_device(), want, err, v.reshape(want.shape).astype(np.float64))


@pytest.mark.parametrize("d", [64, 128])
def test_append8_token_by_token(d):
    # a block fills up over many calls, its scale growing now and then; each step against the state before it
    g = np.random.default_rng(d)
    b = Batch8(g, [0, 14, 37], [40, 40, 40], 2, d, 24)
    c = b.to_device(q4)
    full = list(b.n)
    grew = 0
    ctx0 = list(b.ctx)
    for i in range(full[0]):
        b.ctx, b.n, b.rows = [x + i for x in ctx0], [1, 1, 1], 3
        b.start = np.arange(4, dtype=np.int32)
        b.dctx, b.dstart = torch_dev(np.array(b.ctx, np.int32)), torch_dev(b.start)
        size = np.exp(g.standard_normal((3, 1)))
        k, v = (rand16(g, 3, 2 * d) * size).astype(np.float16), (rand16(g, 3, 2 * d) * size).astype(np.float16)
        before = b.from_device()
        q4.q4_paged_append8(c, b.dctx, b.dstart, 3, torch_dev(k), torch_dev(v))
        after = b.from_device()
        y = k.reshape(3, 2, d).astype(np.float64)
        check_append8(b, before, after, y, np.zeros_like(y), v.reshape(3, 2, d).astype(np.float64))
        grew += sum(int((x[2 + j] != y[2 + j]).sum()) for j in range(2) for x, y in ((before, after),))
    assert q4.q4_device_status() == 0
    assert grew > 20


@pytest.mark.parametrize("d", [64, 128])
def test_append8_extremes(d):
    # infinities, NaN, zeros, the largest and the smallest numbers; blocks of zeros take the least scale
    g = np.random.default_rng(d + 1)
    b = Batch8(g, [0, 20], [64, 40], 1, d, 16)
    x = rand16(g, b.rows, d)
    x[3, ::7], x[5, 1], x[20] = np.inf, -np.inf, np.nan
    x[33, 2], x[40, ::5] = np.nan, 65504.0
    x[48:64] = 0.0
    x[64:76] = (g.integers(1, 60, (12, d)) * 2.0 ** -24).astype(np.float16)
    x[80:90] *= np.float16(1e-4)
    c = b.to_device(q4)
    before = b.from_device()
    q4.q4_paged_append8(c, b.dctx, b.dstart, b.rows, torch_dev(x), torch_dev(-x))
    assert q4.q4_device_status() == 0
    y = x.reshape(-1, 1, d).astype(np.float64)
    after = b.from_device()
    check_append8(b, before, after, y, np.zeros_like(y), -y)
    # all of it reads back as finite fp16, or the NaN that went in
    out = torch.empty(64, d, dtype=torch.float16, device="cuda")
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q4.q4_paged_read8(c, ints(0, 0), ints(0, 64, 64), 64, k=out)
    assert q4.q4_device_status() == 0
    assert np.array_equal(np.isnan(out.cpu().numpy()), np.isnan(x[:64])) and not np.isinf(out.cpu().numpy()).any()


def test_norm_of_zeros_without_eps_stays_zero():
    g = np.random.default_rng(2)
    b = Batch8(g, [0], [3], 1, 64, 16)
    c = b.to_device(q4)
    z = torch.zeros(3, 64, dtype=torch.float16, device="cuda")
    q = z.clone()
    q4.q4_paged_append8(c, b.dctx, b.dstart, 3, z, z, norm=q4.HeadNorm(None, None, 0.0), q=q, q_out=q, n_q_heads=1,
                        freqs=frequencies(64), rot_dim=64)
    assert q4.q4_device_status() == 0
    assert not q.any()
    assert not oracle.e4m3_values(b.from_device()[0][0, b.table[0, 0], 0, :3]).any()  # (either sign of zero)


@pytest.mark.parametrize("which", ["norm", "8"])
@pytest.mark.parametrize("rot", [64, 50])
def test_append_rows_of_a_fused_buffer_in_place(which, rot):
    # q, k and v as columns of one product's output, queries turned in place
    g = np.random.default_rng(5)
    Hq, Hkv, d = 6, 2, 64
    b = (Batch if which == "norm" else Batch8)(g, [10, 0], [4, 7], Hkv, d, 16)
    c = b.to_device(q4)
    w = (Hq + 2 * Hkv) * d
    qkv = rand16(g, b.rows, w)
    buf = torch_dev(qkv)
    q, k, v = buf[:, :Hq * d], buf[:, Hq * d:(Hq + Hkv) * d], buf[:, (Hq + Hkv) * d:]
    f = q4.q4_paged_append_norm if which == "norm" else q4.q4_paged_append8
    f(c, b.dctx, b.dstart, b.rows, k, v, norm=q4.HeadNorm(eps=1e-3), q=q, q_out=q, n_q_heads=Hq,
      freqs=frequencies(rot, theta=1e4), rot_dim=rot, amplitude=AMPLITUDE)
    assert q4.q4_device_status() == 0
    pos = np.concatenate([10 + np.arange(4), np.arange(7)])
    want, err = wanted(qkv[:, :Hq * d], Hq, d, pos, oracle.rope_turns(rot, 1e4), False, True, None, 1e-3)
    got = buf.cpu().numpy()
    assert np.all(np.abs(got[:, :Hq * d].reshape(want.shape) - want) <= ulp16(want) / 2 + err)
    assert np.array_equal(got[:, Hq * d:], qkv[:, Hq * d:])


def test_append8_around_bad_sequences_and_pages():
    # a sequence that does not fit is left out, good ones around it are stored; a page outside the pool holds nothing
    g = np.random.default_rng(9)
    b = Batch8(g, [5, 8, 3, 20], [6, 4, 7, 5], 2, 64, 16)
    c = b.to_device(q4)
    b.dctx[1] = -2
    b.table[2, 0] = b.n_pages + 3
    b.dtable[2, 0] = b.n_pages + 3
    before = b.from_device()
    k, v = rand16(g, b.rows, 128), rand16(g, b.rows, 128)
    q = torch_dev(rand16(g, b.rows, 64))
    qo = torch.full_like(q, 9.0)
    q4.q4_paged_append8(c, b.dctx, b.dstart, b.rows, torch_dev(k), torch_dev(v), q=q, q_out=qo, n_q_heads=1)
    assert q4.q4_device_status() == -7
    y = k.reshape(-1, 2, 64).astype(np.float64)
    check_append8(b, before, b.from_device(), y, np.zeros_like(y), v.reshape(-1, 2, 64).astype(np.float64), [0, 3])
    same = (qo == q).all(1).cpu().numpy()
    assert same[:6].all() and same[10:].all() and bool((qo[6:10] == 9.0).all())


@pytest.mark.parametrize("d", [64, 128])
def test_append8_starts_out_of_order_stay_in_their_pages(d):
    # sequences 0 (rows 0 .. 15) and 2 (rows 3 .. 19) overlap, 1 and 3 end before they begin: what is stored is not
    # defined, where it is stored is
    g = np.random.default_rng(10)
    b = Batch8(g, [0, 0, 0, 0], [16, 16, 17, 16], 2, d, 16, spare=6)
    c = b.to_device(q4)
    b.dstart.copy_(torch.tensor([0, 16, 3, 20, 2], dtype=torch.int32))
    before = b.from_device()
    k, v, q = torch_dev(rand16(g, b.rows, 2 * d)), torch_dev(rand16(g, b.rows, 2 * d)), torch_dev(rand16(g, b.rows, d))
    qo = torch.full_like(q, 9.0)
    q4.q4_paged_append8(c, b.dctx, b.dstart, b.rows, k, v, q=q, q_out=qo, n_q_heads=1)
    assert q4.q4_device_status() == -7
    mine = np.zeros(b.n_pages, bool)
    mine[b.table[0][:1]] = mine[b.table[2][:2]] = True
    for x, y in zip(before, b.from_device()):
        assert np.array_equal(x[:, ~mine].view(np.uint8), y[:, ~mine].view(np.uint8))
    assert bool((qo[20:] == 9.0).all())
    assert bool(((qo == 9.0) | (qo == q))[:20].all())


def test_append8_many_sequences():
    # more sequences than one level of the row search, most of them empty
    g = np.random.default_rng(6)
    n = [int(x) for x in g.integers(0, 3, 1500)]
    n[0] = n[-1] = 0
    b = Batch8(g, [int(x) for x in g.integers(0, 20, 1500)], n, 1, 64, 8)
    c = b.to_device(q4)
    before = b.from_device()
    k, v = rand16(g, b.rows, 64), rand16(g, b.rows, 64)
    q4.q4_paged_append8(c, b.dctx, b.dstart, b.rows, torch_dev(k), torch_dev(v))
    assert q4.q4_device_status() == 0
    y = k.reshape(-1, 1, 64).astype(np.float64)
    check_append8(b, before, b.from_device(), y, np.zeros_like(y), v.reshape(-1, 1, 64).astype(np.float64))
    out = torch.empty(b.rows, 64, dtype=torch.float16, device="cuda")
    q4.q4_paged_read8(c, b.dctx, b.dstart, b.rows, v=out)
    pool = b.values(b.from_device()[1], b.from_device()[3])[0]
    want = np.concatenate([b.rows_of(pool, s, b.ctx[s] + np.arange(m)) for s, m in enumerate(b.n)]).reshape(b.rows, 64)
    assert np.array_equal(out.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("rows", [3, 40, 900])
def test_append8_replays_with_other_sizes(rows):
    # one captured call; the sizes change on the device, down to nobody having a row
    g = np.random.default_rng(rows)
    b = Batch8(g, [40, 40], [rows, rows], 2, 64, 16)  # (pages for every size below)
    c = b.to_device(q4)
    k, v = rand16(g, rows, 128), rand16(g, rows, 128)
    dk, dv = torch_dev(k), torch_dev(v)
    run = lambda: q4.q4_paged_append8(c, b.dctx, b.dstart, rows, dk, dv)  # noqa: E731
    b.dstart.copy_(torch_dev(np.array([0, rows, rows], np.int32)))
    side = torch.cuda.Stream()
    keep = [x.clone() for x in b.d8]
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for ctx, n in (([30, 5], [rows, 0]), ([0, 17], [rows // 3, rows - rows // 3]), ([7, 9], [0, 0]), ([16, 15], [1, rows - 1])):
        b.ctx, b.n = ctx, n
        b.start = np.array([0, n[0], sum(n)], np.int32)
        b.dctx.copy_(torch_dev(np.array(ctx, np.int32)))
        b.dstart.copy_(torch_dev(b.start))
        for x, y in zip(b.d8, keep):
            x.copy_(y)
        before = b.from_device()
        graph.replay()
        assert q4.q4_device_status() == 0
        y = k.reshape(-1, 2, 64).astype(np.float64)
        check_append8(b, before, b.from_device(), y, np.zeros_like(y), v.reshape(-1, 2, 64).astype(np.float64))


# ------------------------------------------------------------------ read back ---

@pytest.mark.parametrize("d,Hkv,page", [(128, 8, 64), (128, 3, 24), (64, 1, 7), (64, 5, 1), (128, 1, 100)])
def test_read8(d, Hkv, page):
    g = np.random.default_rng(d + page)
    b = Batch8(g, [0, 90, 13, 40], [50, 3, 0, 70], Hkv, d, page)
    c = b.to_device(q4)
    w, tail = Hkv * d, 2
    k = torch.full((b.rows + tail, w + 8), 5.0, dtype=torch.float16, device="cuda")
    v = torch.full((b.rows + tail, w), 5.0, dtype=torch.float16, device="cuda")
    q4.q4_paged_read8(c, b.dctx, b.dstart, b.rows + tail, k[:, :w], v)
    assert q4.q4_device_status() == 0
    for got, pool in ((k.cpu().numpy()[:, :w], b.k), (v.cpu().numpy(), b.v)):
        want = np.concatenate([b.rows_of(pool[0], s, b.ctx[s] + np.arange(m)) for s, m in enumerate(b.n)]).reshape(b.rows, w)
        assert np.array_equal(got[:b.rows].astype(np.float64), want)
        assert np.all(got[b.rows:] == 5.0)
    assert bool((k[:, w:] == 5.0).all())
    only = torch.empty(b.rows, w, dtype=torch.float16, device="cuda")
    q4.q4_paged_read8(c, b.dctx, b.dstart, b.rows, v=only)
    assert torch.equal(only, v[:b.rows])
    assert q4.q4_device_status() == 0


def test_read8_bad_pages_and_sequences():
    g = np.random.default_rng(3)
    b = Batch8(g, [4, 0, 9], [5, 20, 6], 2, 64, 16)
    c = b.to_device(q4)
    b.dtable[1, 1] = -1          # positions 16 .. read as zeros
    b.dctx[2] = 1 << 20          # does not fit: left out
    k = torch.full((b.rows, 128), 5.0, dtype=torch.float16, device="cuda")
    v = k.clone()
    q4.q4_paged_read8(c, b.dctx, b.dstart, b.rows, k, v)
    assert q4.q4_device_status() == -7
    k = k.cpu().numpy().astype(np.float64)
    assert np.array_equal(k[:5], b.rows_of(b.k[0], 0, 4 + np.arange(5)).reshape(5, -1))
    assert np.array_equal(k[5:21], b.rows_of(b.k[0], 1, np.arange(16)).reshape(16, -1))
    assert not k[21:25].any() and np.all(k[25:] == 5.0)


# ----------------------------------------------------------------- acceptance ---

def accept(b, c, draft, parents, sampled, layers, strides):
    i32 = lambda x: torch_dev(np.asarray(x, np.int32))
    out = [torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (b.S, max(1, b.rows), b.S, b.S)]
    q4.q4_tree_accept8(c, b.dctx, b.dstart, b.rows, i32(draft), i32(parents), i32(sampled), *out, n_layers=layers,
                       layer_stride=strides[0], scale_stride=strides[1])
    return [x.cpu().numpy() for x in out]


@pytest.mark.parametrize("d,Hkv,page,layers", [(128, 2, 16, 3), (64, 3, 24, 2), (128, 1, 7, 1), (64, 1, 1, 2),
                                               (128, 8, 64, 5), (64, 2, 100, 1)])
def test_accept8(d, Hkv, page, layers):
    g = np.random.default_rng(page + d)
    ctx, n = [0, 14, 30, 5, 61, 3], [1, 20, 64, 0, 40, 300]
    b = Batch8(g, ctx, n, Hkv, d, page, layers=layers)
    c = b.to_device(q4)
    draft, parents, sampled, paths = [], [], [], []
    for s, m in enumerate(n):
        p = random_tree(g, m, fan=2) if m else []
        tok = [100 * s + j for j in range(m)]
        smp = g.integers(-5, 0, m).tolist()
        at = m - 1  # walk some row's ancestors
        chain = []
        while at > 0:
            chain.append(at)
            at = p[at]
        for j in chain:
            smp[p[j]] = tok[j]
        draft, parents, sampled = draft + tok, parents + p, sampled + smp
        paths.append(oracle.tree_path(tok, p, smp))
    before = b.from_device()
    acc, path, nxt, ctx_out = accept(b, c, draft, parents, sampled, layers, (b.k8[0].size, b.k_scales[0].size))
    assert q4.q4_device_status() == 0
    assert acc.tolist() == [len(p) for p in paths]
    assert ctx_out.tolist() == [x + len(p) for x, p in zip(ctx, paths)]
    for s, p in enumerate(paths):
        assert path[b.start[s]:b.start[s + 1]].tolist() == p + [-1] * (n[s] - len(p))
        assert nxt[s] == (sampled[b.start[s] + p[-1]] if p else -1)
    want = [x.copy() for x in before]
    for s, p in enumerate(paths):
        for i in range(2):
            oracle.cache8_accept(want[i], want[2 + i], b.table[s], ctx[s], n[s], p)
    for x, y in zip(want, b.from_device()):
        assert np.array_equal(x.view(np.uint8), y.view(np.uint8))
    assert any((x != y).any() for x, y in zip(before[2:], want[2:]) if page > 1) or page == 1


def test_accept8_without_layers_moves_nothing_and_bad_pages_hold_nothing():
    g = np.random.default_rng(1)
    b = Batch8(g, [14, 0], [6, 6], 1, 64, 16)
    c = b.to_device(q4)
    before = b.from_device()
    args = ([0, 1, 2, 3, 4, 5] * 2, [-1, 0, 0, 1, 2, 4] * 2, [2, 0, 4, 0, 5, 7] * 2)  # path 0 2 4 5
    acc, path, nxt, ctx = accept(b, c, *args, 0, (0, 0))
    assert acc.tolist() == [4, 4] and ctx.tolist() == [18, 4] and nxt.tolist() == [7, 7]
    assert path.tolist() == [0, 2, 4, 5, -1, -1] * 2
    for x, y in zip(before, b.from_device()):
        assert np.array_equal(x.view(np.uint8), y.view(np.uint8))
    assert q4.q4_device_status() == 0
    # the first sequence's second page is outside the pool: its rows 2 .. have no memory, so nothing moves there
    b.dtable[0, 1] = 1 << 30
    accept(b, c, *args, 1, (0, 0))
    assert q4.q4_device_status() == -7
    want = [x.copy() for x in before]
    for i in range(2):
        oracle.cache8_accept(want[i], want[2 + i], b.table[1], 0, 6, [0, 2, 4, 5])
    after = b.from_device()
    for x, y in zip(want, after):
        assert np.array_equal(x.view(np.uint8), y.view(np.uint8))


# ------------------------------------------------------------- scales that grow ---

@pytest.mark.parametrize("d,page", [(64, 24), (128, 16), (128, 7), (64, 100)])
def test_append8_twice_as_large_each_time(d, page):
    # every token is twice the one before: a block that goes on takes twice its scale each time, in every head
    g = np.random.default_rng(d + page)
    S, H, steps = 11, 2, 20
    ctx0 = [int(x) for x in g.integers(0, 60, S)]
    b = Batch8(g, [0] * S, [c + steps for c in ctx0], H, d, page)  # (pages for all of it)
    c = b.to_device(q4)
    b.d8[2].fill_(2.0 ** -15)
    b.d8[3].fill_(2.0 ** -15)
    base = [rand16(g, S, H * d) for _ in range(2)]
    base = [(x * np.float16(2.0 ** -12) + np.float16(2.0 ** -13) * np.sign(x)).astype(np.float16) for x in base]
    base = [np.where(x == 0, np.float16(2.0 ** -13), x) for x in base]
    for x in base:
        assert 2.0 ** 20 * np.abs(x.astype(np.float64)).max() < 61440
    b.n, b.rows = [1] * S, S
    b.start = np.arange(S + 1, dtype=np.int32)
    b.dstart.copy_(torch_dev(b.start))
    grown = [0, 0]
    for i in range(steps):
        b.ctx = [x + i for x in ctx0]
        b.dctx.copy_(torch_dev(np.array(b.ctx, np.int32)))
        k, v = ((x.astype(np.float64) * 2.0 ** i).astype(np.float16) for x in base)
        before = b.from_device()
        q4.q4_paged_append8(c, b.dctx, b.dstart, S, torch_dev(k), torch_dev(v))
        after = b.from_device()
        check_append8(b, before, after, k.reshape(S, H, d).astype(np.float64), np.zeros((S, H, d)),
                      v.reshape(S, H, d).astype(np.float64))
        for s in range(S):
            at = b.ctx[s] % page
            if i == 0 or at % 16 == 0:
                continue  # a block's first token, or one behind positions that this test has not stored
            for j in range(2):
                was, now = (x[2 + j][0, b.table[s, b.ctx[s] // page], :, at // 16] for x in (before, after))
                low = now == 2.0 ** -15  # (the least scale holds for the first ones)
                assert np.array_equal(now[~low], 2 * was[~low])
                grown[j] += int((~low).sum())
    assert q4.q4_device_status() == 0
    assert min(grown) > S * steps  # of 2 S (steps - 1), less the blocks' first tokens and the least scales


@pytest.mark.parametrize("d,Hkv,page,layers", [(128, 2, 16, 3), (64, 3, 32, 1), (64, 1, 48, 2)])
def test_accept8_rows_from_blocks_of_greater_scales(d, Hkv, page, layers):
    # positions 16 .. of each sequence are 32 times larger: rows that move from there into the first block of the new
    # ones take it to their scale, and its other rows are rewritten
    g = np.random.default_rng(7 + d)
    ctx, n = [3, 10, 0], [40, 30, 64]
    b = Batch8(g, ctx, n, Hkv, d, page, layers=layers, spread=0.2)
    for s in range(3):
        for p in range(16, ctx[s] + n[s], 16):
            at = (slice(None), b.table[s, p // page], slice(None), p % page // 16)
            b.k_scales[at] *= 32.0
            b.v_scales[at] *= 32.0
    c = b.to_device(q4)
    draft, parents, sampled, paths = [], [], [], []
    for s in range(3):
        far = [20 + j for j in range(4)]  # 0 -> 20 -> 21 -> 22 -> 23: places 1 .. 4
        p = [-1] + [0] * (n[s] - 1)
        smp = [-1] * n[s]
        for a, i in zip([0] + far, far):
            p[i], smp[a] = a, i
        draft, parents, sampled = draft + list(range(n[s])), parents + p, sampled + smp
        paths.append([0] + far)
    before = b.from_device()
    acc = accept(b, c, draft, parents, sampled, layers, (b.k8[0].size, b.k_scales[0].size))[0]
    assert q4.q4_device_status() == 0
    assert acc.tolist() == [5, 5, 5]
    want, after = [x.copy() for x in before], b.from_device()
    for s in range(3):
        for i in range(2):
            oracle.cache8_accept(want[i], want[2 + i], b.table[s], ctx[s], n[s], paths[s])
            block = (slice(None), b.table[s, 0], slice(None), 0)
            assert np.all(after[2 + i][block] > before[2 + i][block])
    for x, y in zip(want, after):
        assert np.array_equal(x.view(np.uint8), y.view(np.uint8))


def test_append_norm_past_32_bit_offsets():
    # pools of more than 2^31 elements: the pages in use lie at the far end
    d, Hq, Hkv, rot, page = 128, 4, 2, 128, 64
    g, b, q, k, v, rotary, wq, wk = setup(Batch, (d, Hq, Hkv, rot, False, page), [200, 77, 0], [3, 1, 70], seed=6)
    far = (1 << 31) // (Hkv * page * d) + 5  # pages before them
    b.to_device(q4)
    pools = []
    for x in (b.k, b.v):
        t = torch.empty((far + b.n_pages,) + x.shape[2:], dtype=torch.float16, device="cuda")
        t[far:] = torch_dev(x[0])
        pools.append(t)
    table = torch_dev(np.where(b.table >= 0, b.table + far, -1).astype(np.int32))
    c = q4.PagedCache(*pools, far + b.n_pages, page, Hkv, d, table, b.S, b.max_pages)
    qo = call(q4.q4_paged_append_norm, b, c, q, k, v, Hq, rot, False, None, q4.HeadNorm(torch_dev(wq), torch_dev(wk), 1e-3))
    assert q4.q4_device_status() == 0
    turns = oracle.rope_turns(rot, 1e4)
    check_q(qo, q, b, Hq, d, rotary, turns, False, True, wq, 1e-3)
    want, err = wanted(k, Hkv, d, rotary, turns, False, True, wk, 1e-3)
    got = [x[far:].cpu().numpy() for x in pools]
    at = [b.ctx[s] + np.arange(m) for s, m in enumerate(b.n)]
    new_k, new_v = (np.concatenate([b.rows_of(x, s, p) for s, p in enumerate(at)]) for x in got)
    assert np.all(np.abs(new_k.astype(np.float64) - want) <= ulp16(want) / 2 + err)
    assert np.array_equal(new_v, v.reshape(new_v.shape))
    for pool, was in zip(got, (b.k[0], b.v[0])):
        for s, p in enumerate(at):
            was[b.table[s][p // page], :, p % page] = pool[b.table[s][p // page], :, p % page]
        assert np.array_equal(pool.view(np.uint16), was.view(np.uint16))
