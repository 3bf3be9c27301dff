"""GPU parity of the attention over the 8-bit paged cache in the form for page
tables of many positions (heads of 128, pages of whole blocks, 49 .. 168 rows per
kv head): its keys meet the products as the codes they are, its queries in three
8-bit parts."""
import numpy as np
import pytest

import oracle
import test_tree_attention8_gpu as short
from helpers import torch_dev
from serving_helpers import rand16
from test_tree_attention_gpu import seen_by

torch = pytest.importorskip("torch")
import bit_quantized_gemv_q4_gb300 as q4  # noqa: E402

pytestmark = pytest.mark.gpu
POSITIONS = 4096  # of a page table, from which on the form is taken

make, reckon = short.batch, short.expected


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from bit_quantized_gemv_q4_gb300 import build
    build.build()


def long(g, ctx, n, Hkv, d, page, **kw):
    b = make(g, ctx, n, Hkv, d, page, **kw)
    more = max(0, -(-POSITIONS // page) - b.max_pages)
    b.table = np.pad(b.table, ((0, 0), (0, more)), constant_values=-1)
    b.max_pages = b.table.shape[1]
    return b


# A query's elements lose at most 2^-10 of what its greatest (counted as 2^-14 if
# it is less) makes 128 or more: 2^-17 of the greatest.  With C the row's greatest
# sum of |k| times that and the scale, a probability and the sum it is divided by
# move by 2^-17 C each: 2^-19 x 8 C together.
def expected(b, q, sees, scale=None):
    a, A, B = reckon(b, q, sees, scale)
    f = 1 / np.sqrt(b.d) if scale is None else scale
    G = q.shape[1] // b.Hkv
    for s in range(b.S):
        rows, L = slice(b.start[s], b.start[s + 1]), b.ctx[s] + b.n[s]
        if L == 0 or b.n[s] == 0:
            continue
        sums = np.nansum(np.abs(b.rows_of(b.k[0], s, np.arange(L))), -1).max(0)  # [Hkv]
        top = np.maximum(np.nanmax(np.abs(q[rows].astype(np.float64)), -1), 2.0 ** -14)
        B[rows] += 8 * f * (top * np.repeat(sums, G))[..., None]
    return a, A, B


@pytest.fixture
def as_long(monkeypatch):
    monkeypatch.setattr(short, "batch", long)
    monkeypatch.setattr(short, "expected", expected)


CASES = [
    # Hkv, G, page, ctx, n: jobs of up to 128 rows, of more, of both; boxes of 16 and 32 rows
    (2, 4, 16, [500, 130, 0], [13, 14, 15]),
    (2, 4, 64, [300, 0, 40, 7], [40, 33, 64, 0]),
    (1, 8, 48, [700, 5], [40, 0]),
    (2, 2, 32, [5, 129, 1000, 0], [120, 130, 60, 0]),
    (1, 1, 128, [2100, 0], [300, 0]),
    (1, 16, 16, [127], [9]),
    (3, 7, 16, [0, 1, 64, 3], [9, 0, 17, 30]),
    (1, 2, 240, [1900, 3], [64, 65]),
    (8, 1, 112, [640, 33, 255], [49, 128, 129]),
]


@pytest.mark.parametrize("kind", ["causal", "tree", "random", "nothing"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, kind):
    Hkv, G, page, ctx, n = CASES[case]
    g = np.random.default_rng(300 + case)
    b = long(g, ctx, n, Hkv, 128, page)
    q = rand16(g, b.rows, Hkv * G, 128)
    sees = seen_by(b, kind, g)
    want = expected(b, q, sees)
    out = short.attend(b, b.to_device(q4), q, kind, sees)
    assert q4.q4_device_status() == 0
    short.check(out, b, q, *want)


@pytest.mark.parametrize("page,n", [(16, [50, 40]), (64, [40, 70]), (16, [100, 50])])
def test_blocks_of_unlike_scales(as_long, page, n):
    short.test_blocks_of_unlike_scales(page, n)


@pytest.mark.parametrize("what", ["page", "ctx", "room"])
def test_a_bad_sequence_is_left_out(as_long, what):
    short.test_forms_leave_a_bad_sequence_out("tcgen05", what)


def test_replays_with_other_sizes(as_long):
    short.test_forms_replay_with_other_sizes("tcgen05")


def test_calls_side_by_side(as_long):
    short.test_calls_side_by_side_and_graphs_that_share_a_workspace()


@pytest.mark.parametrize("n,G,page", [(40, 2, 16), (150, 1, 16), (20, 8, 128)])
def test_small_probabilities_beside_dominant_ones(as_long, n, G, page):
    short.test_small_probabilities_beside_dominant_ones_in_every_form(n, G, page)


@pytest.mark.parametrize("n", [20, 40])
def test_queries_of_every_magnitude(n):
    # rows from fp16's least numbers to its greatest, rows of zeros, and rows whose elements lie 2^20 apart
    g = np.random.default_rng(n)
    b = long(g, [300], [n], 1, 128, 16)
    b.k_scales[...] = np.where(np.isnan(b.k_scales), np.nan, 2.0 ** -15)
    b.set_values()
    q = rand16(g, n, 4, 128).astype(np.float64)
    q *= 2.0 ** g.integers(-24, 14, (n, 4, 1))
    q[::5] *= 2.0 ** g.integers(-20, 1, q[::5].shape)
    q[::7] = 0
    q = np.clip(q, -65504, 65504).astype(np.float16)
    sees = seen_by(b, "causal", g)
    want = expected(b, q, sees)
    out = short.attend(b, b.to_device(q4), q, "causal", sees)
    assert q4.q4_device_status() == 0
    short.check(out, b, q, *want)


@pytest.mark.parametrize("n", [20, 40])
def test_queries_that_are_no_numbers_stay_in_their_rows(n):
    g = np.random.default_rng(n)
    b = long(g, [300], [n], 1, 128, 16)
    q = rand16(g, n, 4, 128)
    sees = seen_by(b, "causal", g)
    a, A, B = expected(b, q, sees)
    odd = q.copy()
    odd[3, 1, 5], odd[7, 0, 127], odd[n - 1, 2, 0] = np.nan, np.inf, -np.inf
    out = short.attend(b, b.to_device(q4), odd, "causal", sees)
    assert q4.q4_device_status() == 0
    got = out.cpu().numpy()[:n].reshape(a.shape)
    bad = np.zeros((n, 4), bool)
    bad[3, 1] = bad[7, 0] = bad[n - 1, 2] = True
    assert np.isnan(got[bad]).all()
    assert short.close(got[~bad], a[~bad], A[~bad], B[~bad]).all()


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("n", [20, 40])
def test_codes_that_are_no_numbers_reach_who_sees_them(n, what):
    g = np.random.default_rng(70 + n)
    b = long(g, [130, 200], [n, n], 2, 128, 32)
    place = lambda p: (0, b.table[1, p // 32], 1, p % 32)  # noqa: E731
    codes = getattr(b, what + "8")
    codes[place(200 + 4)][3] = 0x7F  # a new row of sequence 1, kv head 1: of its rows those that see row 4
    b.set_values()
    q = rand16(g, b.rows, 8, 128)
    sees = seen_by(b, "causal", g)
    out = short.attend(b, b.to_device(q4), q, "causal", sees).cpu().numpy()[:2 * n].reshape(2 * n, 8, 128)
    assert q4.q4_device_status() == 0
    reached = np.zeros(out.shape, bool)
    reached[n + 4:, 4:, :] = what == "k"
    reached[n + 4:, 4:, 3] = True
    assert np.array_equal(np.isnan(out), reached)
    codes[place(204)][3] = oracle.e4m3_codes(1.0)
    b.set_values()
    a, A, B = expected(b, q, sees)
    fine = ~reached
    if what == "k":
        fine[n + 4:, 4:] = False
    assert short.close(out, a, A, B)[fine].all()


@pytest.mark.parametrize("name", ["128 rows", "shared"])
def test_nan_among_every_lanes_columns(as_long, name):
    short.test_nan_among_every_lanes_columns_stays_in_its_column(name)


@pytest.mark.parametrize("kind", ["causal", "nothing"])
@pytest.mark.parametrize("name", ["tcgen05", "tcgen05, shared"])
def test_queries_that_are_no_numbers(as_long, name, kind):
    short.test_queries_that_are_no_numbers_give_nan_in_every_form(name, kind)


@pytest.mark.parametrize("kind", ["causal", "tree"])
@pytest.mark.parametrize("name", ["tcgen05, short", "tcgen05, shared"])
def test_nan_reaches_what_sees_it(as_long, name, kind):
    short.test_nan_reaches_what_sees_it_in_every_form(name, kind)


def test_pages_past_32_bit_offsets(as_long):
    short.test_pages_past_32_bit_offsets(64, [40, 3], 4)


def test_bits_do_not_depend_on_the_run(as_long):
    short.test_bits_do_not_depend_on_the_run()


@pytest.mark.parametrize("top", [2.25, 1.25])
@pytest.mark.parametrize("n,G,page", [(20, 4, 64), (40, 4, 16)])
def test_a_position_that_decides_its_row_late(as_long, n, G, page, top):
    short.test_a_position_that_decides_its_row_late(n, G, 128, page, top)
