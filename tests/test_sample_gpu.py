"""GPU sampling against the fp64 oracle: the token has to be the oracle's
exactly, its probability to fp32's last bits.  Limits alone and together,
ties, masked rows, extreme logits and temperatures, vocabularies around the
sizes the kernel works in, strides and both element types."""
import math

import numpy as np
import pytest

import oracle
from helpers import torch_dev

torch = pytest.importorskip("torch")
import bit_quantized_gemv_q4_gb300 as q4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from bit_quantized_gemv_q4_gb300 import build
    build.build()


def sample(x, ld=0, vocab=None, want_probs=True, **kw):
    x = np.asarray(x)
    rows, V = x.shape[0], vocab or x.shape[1]
    f = lambda v, t: None if v is None else torch_dev(np.broadcast_to(np.asarray(v, t), (rows,)).copy())
    tok = torch.full((rows + 1,), -7, dtype=torch.int32, device="cuda")
    pr = torch.full((rows + 1,), -7.0, device="cuda") if want_probs else None
    q4.q4_sample(torch_dev(x), q4.Q4_F16 if x.dtype == np.float16 else q4.Q4_F32, rows, V, tok,
                 temperature=f(kw.get("temperature"), np.float32), top_k=f(kw.get("top_k"), np.int32),
                 top_p=f(kw.get("top_p"), np.float32), min_p=f(kw.get("min_p"), np.float32),
                 u=f(kw.get("u"), np.float32), probs=pr, ld=ld)
    assert q4.q4_device_status() == 0
    assert tok[rows] == -7 and (pr is None or pr[rows] == -7.0)
    return tok[:rows].tolist(), None if pr is None else pr[:rows].cpu().numpy().astype(np.float64)


def check(x, **kw):
    tok, pr = sample(x, **kw)
    for r in range(x.shape[0]):
        one = {k: None if v is None else np.broadcast_to(np.asarray(v, np.int32 if k == "top_k" else np.float32),
                                                        (x.shape[0],))[r] for k, v in kw.items()}
        one = {k: (int(v) if k == "top_k" else float(v)) for k, v in one.items() if v is not None}
        t, p = oracle.sample(x[r], **one)
        assert tok[r] == t, (r, one, tok[r], t, pr[r], p)
        # a weight carries 2^-30 of itself and 2^-45 of the greatest (a token
        # far below it has few bits), the quotient's fp32 rounding 2^-24
        assert abs(pr[r] - p) <= 2.0 ** -23 * p + 2.0 ** -43, (r, pr[r], p)


def rows16(g, n, V, spread=3.0, dtype=np.float32):
    return (g.standard_normal((n, V)) * spread).astype(dtype)


@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("V", [1, 2, 3, 31, 33, 1000, 1023, 1025, 4099, 50257])
def test_vocabularies_and_limits(V, dtype):
    g = np.random.default_rng(V)
    n = 24
    x = rows16(g, n, V, dtype=dtype)
    u = g.random(n).astype(np.float32)
    check(x, u=u)
    check(x, u=u, temperature=g.uniform(0.3, 2.0, n))
    check(x, u=u, top_k=g.integers(-1, 60, n))
    check(x, u=u, top_p=g.uniform(0.0, 1.1, n))
    check(x, u=u, min_p=g.uniform(-0.1, 0.5, n))
    check(x, u=u, temperature=g.choice([0.0, 0.7, 1.0, 1.5], n), top_k=g.choice([0, 5, 50], n),
          top_p=g.choice([1.0, 0.9, 0.5], n), min_p=g.choice([0.0, 0.1], n))
    check(x)
    check(x, temperature=0.0, u=0.9)


@pytest.mark.parametrize("dtype", [np.float32, np.float16])
def test_large_vocabulary(dtype):
    g = np.random.default_rng(2)
    x = rows16(g, 6, 151936, 2.5, dtype)
    x[:, 1000:1010] += 9
    u = np.array([0.0, 0.3, 0.62, 0.9, 0.97, 0.999], np.float32)
    check(x, u=u)
    check(x, u=u, temperature=1.3, top_p=0.97)
    check(x, u=u, top_k=100000, min_p=1e-5)
    check(rows16(g, 2, 1 << 19, 1.0, dtype), u=[0.4, 0.8])


def test_ties_go_to_the_lowest_index():
    x = np.zeros((8, 4000), np.float32)
    x[:, 7] = -0.0
    x[4:, 100:300] = 1.0
    x[4:, 200] = np.float32(1.0)
    u = np.array([0.0, 0.25, 0.5, 0.99999994] * 2, np.float32)
    check(x, u=u)
    check(x, u=u, top_k=37)
    check(x, u=u, top_p=0.25)
    check(x, u=u, top_k=201, top_p=0.9)
    check(x, u=u, min_p=1.0)
    check(x)
    # few distinct values, many of each
    g = np.random.default_rng(3)
    y = g.integers(-3, 3, (16, 5000)).astype(np.float32)
    u = g.random(16).astype(np.float32)
    check(y, u=u)
    check(y, u=u, top_k=1300, top_p=0.8)


def test_neighbouring_floats():
    # logits one ulp apart: the order is exact although the weights hardly differ
    base = np.float32(3.0)
    x = np.empty((6, 2000), np.float32)
    v = base
    for i in range(2000):
        x[:, (i * 1237) % 2000] = v
        v = np.nextafter(v, np.float32(10), dtype=np.float32)
    u = np.array([0.0, 0.1, 0.5, 0.501, 0.9, 0.9999], np.float32)
    check(x, u=u)
    check(x, u=u, top_k=700)
    check(x, u=u, top_p=0.3)


def test_masked_and_extreme_logits():
    g = np.random.default_rng(4)
    low = np.finfo(np.float32).min
    x = rows16(g, 12, 3001)
    x[0] = -np.inf
    x[1] = np.nan
    x[2, 1:] = -np.inf
    x[3] = low
    x[4, ::2] = low
    x[5, 100:] = -np.inf
    x[6, 5] = np.inf
    x[7, 9:2000:3] = np.inf
    x[8, :50] = np.nan
    x[9, 17] = 3e38
    x[10] = -3e38
    x[10, 5] = -2.9e38
    x[11] *= 1e4
    u = np.full(12, 0.7, np.float32)
    check(x, u=u)
    check(x, u=u, top_k=40, top_p=0.8, min_p=0.05)
    check(x, u=u, top_p=0.0)
    check(x)
    h = rows16(g, 4, 777, dtype=np.float16)
    h[0] = -65504.0
    h[1, 3] = np.inf
    h[2, 5:] = -np.inf
    h[3, :] = -np.inf
    check(h, u=0.4, top_k=3)
    check(h, u=0.4)


def test_extreme_settings():
    g = np.random.default_rng(5)
    x = rows16(g, 8, 2000)
    x[:, 3] = x[:, 4] = 20.0
    for t in (1e-40, 1e-30, 1e-4, 1e4, 1e30, float("inf")):
        check(x, u=g.random(8), temperature=t)
    check(x, u=g.random(8), temperature=-1.0)
    check(x, u=g.random(8), top_k=2**31 - 1)
    check(x, u=g.random(8), top_k=-(2**31))
    check(x, u=g.random(8), top_p=-3.0)
    check(x, u=g.random(8), top_p=1e-30)
    check(x, u=[0.0, -1.0, 1.0, 2.0, 0.99999994, 1e-30, 0.5, 0.25])
    nan = float("nan")
    a, _ = sample(x, u=0.5, top_p=nan, min_p=nan)
    b, _ = sample(x, u=0.5)
    assert a == b
    assert sample(x, u=0.5, temperature=nan)[0] == sample(x)[0]
    assert sample(x, u=nan)[0] == sample(x, u=0.0)[0]


def test_strided_rows_and_no_probs():
    g = np.random.default_rng(6)
    for dtype in (np.float32, np.float16):
        x = rows16(g, 5, 1037, dtype=dtype)
        u = g.random(5).astype(np.float32)
        tok, pr = sample(x, ld=1037, vocab=1001, u=u)
        for r in range(5):
            t, p = oracle.sample(x[r, :1001], u=float(u[r]))
            assert tok[r] == t and abs(pr[r] - p) < 1e-6
        assert sample(x, ld=1037, vocab=1001, u=u, want_probs=False)[0] == tok


def test_shares_follow_the_probabilities():
    # 4096 even numbers of [0, 1): each token gets its share of them to within one
    x = np.log(np.array([0.5, 0.25, 0.125, 0.0625, 0.0625])).astype(np.float32)
    u = (np.arange(4096) + 0.5) / 4096
    tok, _ = sample(np.broadcast_to(x, (4096, 5)).copy(), u=u)
    assert np.all(np.abs(np.bincount(tok, minlength=5) / 4096 - np.exp(x)) <= 1.5 / 4096)


def test_one_call_on_another_stream_and_in_a_graph():
    g = np.random.default_rng(7)
    x = torch_dev(rows16(g, 4, 9000))
    u = torch.tensor([0.1, 0.4, 0.7, 0.95], device="cuda")
    tok = torch.empty(4, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    q4.q4_sample(x, q4.Q4_F32, 4, 9000, tok, u=u, stream=s)
    s.synchronize()
    first = tok.tolist()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.q4_sample(x, q4.Q4_F32, 4, 9000, tok, u=u)
    tok.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert tok.tolist() == first
    u.copy_(torch.tensor([0.9, 0.2, 0.1, 0.5], device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert tok.tolist() == [oracle.sample(x[i].cpu().numpy(), u=float(u[i]))[0] for i in range(4)]


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("kind", ["normal", "rounded", "equal", "masked", "ramp", "wide", "one peak"])
def test_all_limits_in_turn_over_kinds_of_rows(kind, dtype):
    """Every row with settings of its own: flat and peaked rows, the nucleus's end
    and the token in the list, below it and among equals."""
    g = np.random.default_rng(len(kind) * 10 + len(dtype))
    for V in (37, 2500, 9001):
        R = 12
        x = g.standard_normal((R, V)) * np.exp(g.uniform(-4, 3, (R, 1)))
        if kind == "rounded":
            x = np.round(x * 4) / 4
        elif kind == "equal":
            x[:] = x[:, :1]
        elif kind == "masked":
            x[g.random((R, V)) < 0.7] = -np.inf
        elif kind == "ramp":
            x += np.linspace(0, 40, V)
        elif kind == "wide":
            x *= 100
        elif kind == "one peak":
            x[:, V // 3] += 20
        x = x.astype(np.float16 if dtype == "f16" else np.float32)
        T = np.where(g.random(R) < 0.5, 1.0, np.exp(g.uniform(-4, 4, R))).astype(np.float32)
        k = np.where(g.random(R) < 0.5, 0, g.integers(1, V + 5, R)).astype(np.int32)
        p = np.where(g.random(R) < 0.4, 1.0, g.random(R)).astype(np.float32)
        m = np.where(g.random(R) < 0.5, 0.0, np.exp(g.uniform(-10, 0, R))).astype(np.float32)
        u = g.random(R).astype(np.float32)
        tok, pr = sample(x, temperature=T, top_k=k, top_p=p, min_p=m, u=u)
        for r in range(R):
            t, q = oracle.sample(x[r], float(T[r]), int(k[r]), float(p[r]), float(m[r]), float(u[r]))
            assert tok[r] == t, (V, r, tok[r], t)
            assert abs(pr[r] - q) <= 2.0 ** -23 * q + 2.0 ** -43, (V, r, pr[r], q)  # (as in check)


@pytest.mark.parametrize("top", [8.0078125, 12.0, 2.5])
@pytest.mark.parametrize("V", [3000, 20001])
def test_half_logits_far_smaller_than_the_greatest(top, V):
    """Logits whose difference to the greatest no float holds: multiples of 2^-24
    under a greatest logit of 2.5 to 12.  Left out, the lost bits come to 2^-21 of
    such a weight; check allows 2^-23."""
    g = np.random.default_rng(V)
    for low in (7, -7, 5, None):
        x = np.empty((6, V), np.float16)
        x[:] = (np.full((6, V), low) if low else g.integers(-7, 8, (6, V))) * 2.0 ** -24
        x[:, V // 2] = top
        u = ((np.arange(6) + 0.5) / 6).astype(np.float32)
        u[3:] = 1 - (1 - u[3:]) * np.float32(0.02)
        check(x, u=u)
        check(x, u=u, top_p=0.9999)
        check(x, u=u, top_k=2000)


def test_equal_weights_of_the_longest_part_add_up():
    """Rows that begin one half behind a 16-byte boundary give the last of four
    CTAs 2^17 + 7 equal logits below the list; at these temperatures (found by
    evaluating the weight's operations in exact arithmetic) the 15 low bits of their
    weight are all set, which no 32-bit sum of as many holds."""
    V, R = 1 << 19, 48  # (as many rows as leave four CTAs to each)
    temps = [0.7507458329200745, 0.7530942559242249, 0.7561022043228149, 0.7603664398193359, 0.7634600400924683,
             0.7695407867431641]
    x = np.full((R, V + 1), -np.inf, np.float16)
    x[:, 0] = 0.0
    rows = list(range(7, R, 8))
    for r in rows:
        x[r, 1:1601:8] = 0.0
        x[r, 1 + 8 * ((V // 8 - 1) * 3 // 4):] = -1.0
    T, u = np.ones(R, np.float32), np.full(R, 0.5, np.float32)
    T[rows], u[rows] = temps, [0.3, 0.5, 0.9, 0.99, 0.999, 0.99999]
    tok, pr = sample(x, ld=V + 1, vocab=V, temperature=T, u=u)
    for r in rows:
        t, p = oracle.sample(x[r, :V], float(T[r]), u=float(u[r]))
        assert tok[r] == t, (r, tok[r], t)
        assert abs(pr[r] - p) <= 2.0 ** -23 * p + 2.0 ** -43
