"""Host-side checks of the paged-cache and sampling calls that need no GPU:
struct layouts, refusals (no pointer is dereferenced), the page division."""
import ctypes
import os
import random
import subprocess

import pytest

import bit_quantized_gemv_q4_gb300 as q4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return q4.lib()


STRUCTS = ["q4_paged_cache", "q4_rope_desc", "q4_paged_append_desc", "q4_tree_attention_desc", "q4_tree_accept_desc",
           "q4_sample_desc"]


def test_struct_layouts_match_c(tmp_path):
    lines = []
    for t in STRUCTS:
        lines.append(f'printf("{t} %zu\\n", sizeof({t}));')
        for f, *_ in getattr(q4, t)._fields_:
            lines.append(f'printf("{t}.{f} %zu\\n", offsetof({t}, {f}));')
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"q4.h\"\nint main(void) {\n" +
                   "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for ln in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        key, val = ln.rsplit(" ", 1)
        t, _, f = key.partition(".")
        got = getattr(getattr(q4, t), f).offset if f else ctypes.sizeof(getattr(q4, t))
        assert got == int(val), key


def cache(**kw):
    c = dict(k=FAKE, v=FAKE, page_table=FAKE, n_pages=8, page_size=16, n_kv_heads=2, head_dim=128, n_seqs=2, max_pages=4)
    c.update(kw)
    return q4.q4_paged_cache(*[c[f] for f, _ in q4.q4_paged_cache._fields_])


CACHE_BAD = [("k", None, -1), ("v", None, -1), ("page_table", None, -1), ("n_pages", 0, -1), ("page_size", 0, -1),
             ("n_kv_heads", 0, -1), ("n_seqs", 0, -1), ("max_pages", 0, -1), ("head_dim", 96, -2), ("k", FAKE + 8, -3),
             ("v", FAKE + 2, -3), ("page_size", 1 << 29, -2)]


def refuse(call, base, bad):
    for f, v, want in bad:
        d = type(base).from_buffer_copy(base)
        setattr(d, f, v)
        assert call(ctypes.byref(d), None) == want, (f, v)
        assert q4.lib().q4_last_error() != b""
    if hasattr(base, "cache"):
        for f, v, want in CACHE_BAD:
            d = type(base).from_buffer_copy(base)
            d.cache = cache(**{f: v})
            assert call(ctypes.byref(d), None) == want, (f, v)
        for f in ("ctx_len", "row_start"):
            d = type(base).from_buffer_copy(base)
            setattr(d, f, None)
            assert call(ctypes.byref(d), None) == -1
        d = type(base).from_buffer_copy(base)
        d.rows = -1
        assert call(ctypes.byref(d), None) == -1
    assert call(None, None) == -1


def test_append_refusals(L):
    d = q4.q4_paged_append_desc(cache(), FAKE, FAKE, 4, None, FAKE, FAKE, 0, 0, FAKE, FAKE, 0, 0, 4, FAKE, 128, 0, 1.0)
    refuse(L.q4_paged_append, d, [
        ("k", None, -1), ("v", None, -1), ("q", None, -1), ("q_out", None, -1), ("n_q_heads", 0, -1),
        ("rot_dim", 130, -1), ("rot_dim", 63, -1), ("rot_dim", -2, -1), ("rot_dim", 0, -1), ("freqs", None, -1),
        ("layout", 2, -1), ("amplitude", -1.0, -1), ("amplitude", float("nan"), -1), ("freqs", FAKE + 4, -3),
        ("k", FAKE + 8, -3), ("v", FAKE + 8, -3), ("q", FAKE + 8, -3), ("q_out", FAKE + 8, -3), ("ldk", 255, -1),
        ("ldk", 260, -3), ("ldv", 8, -1), ("ldq", 511, -1), ("ldqo", 513, -3), ("ldq", 1024, -1),
        ("n_q_heads", 1 << 20, -2)])


def test_attention_refusals(L):
    need = L.q4_tree_attention_workspace_bytes(128)
    assert 0 < need <= 256 << 20 and 0 < L.q4_tree_attention_workspace_bytes(64) <= need
    assert L.q4_tree_attention_workspace_bytes(96) == 0
    d = q4.q4_tree_attention_desc(cache(), FAKE, FAKE, 4, FAKE, 1, FAKE, FAKE, 0, 0, 4, 0.0, FAKE, need)
    refuse(L.q4_tree_attention, d, [
        ("q", None, -1), ("out", None, -1), ("workspace", None, -1), ("workspace_bytes", need - 1, -1),
        ("workspace", FAKE + 16, -3), ("n_q_heads", 1, -1), ("n_q_heads", 5, -1), ("mask_words", 0, -1),
        ("mask", FAKE + 2, -3), ("scale", -1.0, -1), ("scale", float("inf"), -1), ("scale", float("nan"), -1),
        ("scale", 1e-38, -1), ("ldq", 500, -1), ("ldo", 516, -3), ("q", FAKE + 8, -3), ("out", FAKE + 4, -3),
        ("rows", 2**31 - 1, -2)])


def test_accept_refusals(L):
    d = q4.q4_tree_accept_desc(cache(), FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 8 * 16 * 2 * 128)
    refuse(L.q4_tree_accept, d, [(f, None, -1) for f in ("draft", "parents", "sampled", "accepted", "path",
                                                         "next_token", "ctx_out")] +
           [("n_layers", -1, -1), ("layer_stride", 8 * 16 * 2 * 128 - 8, -1), ("layer_stride", 8 * 16 * 2 * 128 + 4, -3)])


def test_sample_refusals(L):
    d = q4.q4_sample_desc(FAKE, 0, 3, 1000, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    refuse(L.q4_sample, d, [("logits", None, -1), ("tokens", None, -1), ("dtype", 2, -1), ("rows", -1, -1),
                            ("vocab", 0, -1), ("vocab", (1 << 19) + 1, -2), ("ld", 999, -1), ("logits", FAKE + 2, -3)])


def test_frequencies_refusals(L):
    d = q4.q4_rope_desc(128, 4096, 1e6, 8.0, 1.0, 32.0)
    call = lambda p, s: L.q4_rope_frequencies(p, FAKE, s)
    refuse(call, d, [("rot_dim", 0, -1), ("rot_dim", 3, -1), ("rot_dim", 2048, -1), ("theta", 1.0, -1),
                     ("theta", float("nan"), -1), ("theta", float("inf"), -1), ("factor", 0.5, -1),
                     ("factor", float("inf"), -1), ("orig_len", -1, -1), ("alpha", -1.0, -1), ("beta", 1.0, -1),
                     ("beta", float("nan"), -1)])
    assert L.q4_rope_frequencies(ctypes.byref(d), None, None) == -1
    assert L.q4_rope_frequencies(ctypes.byref(d), FAKE + 4, None) == -3


def test_page_division_is_exact():
    # the kernels' quotient: n m >> (31 + s), m = ceil(2^(31+s) / d), s = ceil(log2 d)
    r = random.Random(1)
    ds = list(range(1, 300)) + [2**k + e for k in range(9, 31) for e in (-1, 0, 1)] + [2**31 - 1]
    for d in ds:
        s = (d - 1).bit_length()
        m = -(-(1 << (31 + s)) // d)
        assert m < 1 << 32
        for n in [0, d - 1, d, 2 * d - 1, (2**31 - 1) // d * d, (2**31 - 1) // d * d - 1, 2**31 - 1] + [
                r.randrange(2**31) for _ in range(50)]:
            if 0 <= n < 2**31:
                assert n * m >> (31 + s) == n // d, (n, d)


def test_binding_checks_its_tensors(L):
    torch = pytest.importorskip("torch")
    host = torch.zeros(64, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device memory"):
        q4.q4_sample(host, q4.Q4_F32, 1, 64, host)
    with pytest.raises(ValueError, match="CUDA device memory"):
        q4.q4_tree_accept(q4.PagedCache(FAKE, FAKE, 8, 16, 2, 128, host, 2, 4), FAKE, FAKE, 4, *[FAKE] * 7)


def test_binding_without_a_device_gives_the_library_s_error(L):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("there is a device")
    with pytest.raises(q4.Q4Error, match="NO_DEVICE"):
        q4.q4_sample(FAKE, q4.Q4_F32, 1, 64, FAKE)
    with pytest.raises(q4.Q4Error, match="vocab"):
        q4.q4_sample(FAKE, q4.Q4_F32, 1, 0, FAKE)


def test_positions_leave_room_for_a_tile_below_2_31(L):
    # the attention rounds a sequence's length up to tiles of 128 positions in 32 bits
    append = q4.q4_paged_append_desc(cache(), FAKE, FAKE, 0, None, FAKE, FAKE, 0, 0, None, None, 0, 0, 0, None, 0, 0, 1.0)
    attend = q4.q4_tree_attention_desc(cache(), FAKE, FAKE, 0, None, 0, FAKE, FAKE, 0, 0, 4, 0.0, FAKE,
                                       L.q4_tree_attention_workspace_bytes(128))
    accept = q4.q4_tree_accept_desc(cache(), FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0)
    for pages, size in ((4, (1 << 29) - 31), ((1 << 25) - 1, 64), ((1 << 31) - 127, 1), (1, (1 << 31) - 1)):
        for call, d in ((L.q4_paged_append, append), (L.q4_tree_attention, attend), (L.q4_tree_accept, accept)):
            d.cache = cache(max_pages=pages, page_size=size)
            assert call(ctypes.byref(d), None) == -2, (pages, size)
    for pages, size in ((4, (1 << 29) - 32), ((1 << 25) - 2, 64), ((1 << 31) - 128, 1), (1, (1 << 31) - 128)):
        # (no rows: with a device the call ends before it reads anything)
        for call, d in ((L.q4_paged_append, append), (L.q4_tree_attention, attend)):
            d.cache = cache(max_pages=pages, page_size=size)
            assert call(ctypes.byref(d), None) in (0, -6), (pages, size, L.q4_last_error())
            n = pages * size  # the last tile's end
            assert (n + 127) // 128 * 128 < 1 << 31


def test_heads_and_sequences_that_pass_32_bits_are_refused(L):
    # (a layer's columns of 16 bytes, the searches over the sequences and the grids are counted in 32 bits)
    append = q4.q4_paged_append_desc(cache(), FAKE, FAKE, 0, None, FAKE, FAKE, 0, 0, None, None, 0, 0, 0, None, 0, 0, 1.0)
    attend = q4.q4_tree_attention_desc(cache(), FAKE, FAKE, 0, None, 0, FAKE, FAKE, 0, 0, 1 << 26, 0.0, FAKE,
                                       L.q4_tree_attention_workspace_bytes(128))
    accept = q4.q4_tree_accept_desc(cache(), FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 0)
    for bad in (dict(n_kv_heads=(1 << 17) + 1), dict(n_kv_heads=1 << 26), dict(n_seqs=(1 << 27) + 1),
                dict(n_seqs=(1 << 31) - 1)):
        for call, d in ((L.q4_paged_append, append), (L.q4_tree_attention, attend), (L.q4_tree_accept, accept)):
            d.cache = cache(**bad)
            assert call(ctypes.byref(d), None) == -2, bad


def test_misaligned_arrays_are_refused(L):
    # (a kernel that reads them would fault)
    need = L.q4_tree_attention_workspace_bytes(128)
    append = q4.q4_paged_append_desc(cache(), FAKE, FAKE, 4, FAKE, FAKE, FAKE, 0, 0, FAKE, FAKE, 0, 0, 4, FAKE, 128, 0, 1.0)
    attend = q4.q4_tree_attention_desc(cache(), FAKE, FAKE, 4, FAKE, 1, FAKE, FAKE, 0, 0, 4, 0.0, FAKE, need)
    accept = q4.q4_tree_accept_desc(cache(), FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 0)
    sample = q4.q4_sample_desc(FAKE, 0, 3, 1000, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    for call, base, names in (
            (L.q4_paged_append, append, ["ctx_len", "row_start", "positions"]),
            (L.q4_tree_attention, attend, ["ctx_len", "row_start", "mask"]),
            (L.q4_tree_accept, accept, ["ctx_len", "row_start", "draft", "parents", "sampled", "accepted", "path",
                                        "next_token", "ctx_out"]),
            (L.q4_sample, sample, ["temperature", "top_k", "top_p", "min_p", "u", "tokens", "probs"])):
        for off in (1, 2, 3):
            for name in names:
                d = type(base).from_buffer_copy(base)
                setattr(d, name, FAKE + off)
                assert call(ctypes.byref(d), None) == -3, name
            if base is not sample:
                d = type(base).from_buffer_copy(base)
                d.cache = cache(page_table=FAKE + off)
                assert call(ctypes.byref(d), None) == -3


def test_no_rows_need_no_arrays(L):
    # (what a framework's empty tensor gives as its address)
    append = q4.q4_paged_append_desc(cache(), FAKE, FAKE, 0, None, None, None, 0, 0, None, None, 0, 0, 4, FAKE, 128, 0, 1.0)
    attend = q4.q4_tree_attention_desc(cache(), FAKE, FAKE, 0, None, 1, None, None, 0, 0, 4, 0.0, FAKE,
                                       L.q4_tree_attention_workspace_bytes(128))
    sample = q4.q4_sample_desc(None, 0, 0, 1000, 0, None, None, None, None, None, None, None)
    for call, d in ((L.q4_paged_append, append), (L.q4_tree_attention, attend), (L.q4_sample, sample)):
        assert call(ctypes.byref(d), None) in (0, -6), L.q4_last_error()
        d.rows = 1
        assert call(ctypes.byref(d), None) == -1
