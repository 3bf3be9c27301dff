"""Host-side checks of the 8-bit cache's calls and of the append with norms that
need no GPU: struct layouts, refusals (no pointer is dereferenced)."""
import ctypes
import os
import subprocess

import pytest

import bit_quantized_gemv_q4_gb300 as q4
from test_serving_abi import CACHE_BAD, FAKE, ROOT, cache

STRUCTS = ["q4_head_norm", "q4_paged_cache8", "q4_paged_append8_desc", "q4_paged_read8_desc", "q4_tree_attention8_desc",
           "q4_tree_accept8_desc"]


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return q4.lib()


def test_struct_layouts_match_c(tmp_path):
    lines = []
    for t in STRUCTS:
        lines.append(f'printf("{t} %zu\\n", sizeof({t}));')
        for f, *_ in getattr(q4, t)._fields_:
            lines.append(f'printf("{t}.{f} %zu\\n", offsetof({t}, {f}));')
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"q4.h\"\nint main(void) {\n" +
                   "\n".join(lines) + "\nreturn Q4_CACHE8_BLOCK != 16; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for ln in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        key, val = ln.rsplit(" ", 1)
        t, _, f = key.partition(".")
        got = getattr(getattr(q4, t), f).offset if f else ctypes.sizeof(getattr(q4, t))
        assert got == int(val), key


def test_packed_descriptors_are_the_structures():
    for packed, kind in ((q4._APPEND_NORM, q4.q4_paged_append_desc), (q4._APPEND8, q4.q4_paged_append8_desc),
                         (q4._NORM, q4.q4_head_norm), (q4._READ8, q4.q4_paged_read8_desc),
                         (q4._ATTENTION8, q4.q4_tree_attention8_desc), (q4._ACCEPT8, q4.q4_tree_accept8_desc)):
        values, n = [], 0

        def build(t):
            nonlocal n
            out = t()
            for f, ty in t._fields_:
                if issubclass(ty, ctypes.Structure):
                    setattr(out, f, build(ty))
                    continue
                n += 1
                v = 0.5 * n if ty is ctypes.c_float else 1000 * n + 1
                values.append(v)
                setattr(out, f, v)
            return out

        want = build(kind)
        assert packed.pack(*values) == bytes(want), kind


def cache8(**kw):
    c = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, page_table=FAKE, n_pages=8, page_size=16, n_kv_heads=2,
             head_dim=128, n_seqs=2, max_pages=4)
    c.update(kw)
    return q4.q4_paged_cache8(*[c[f] for f, _ in q4.q4_paged_cache8._fields_])


CACHE8_BAD = CACHE_BAD + [("k_scales", None, -1), ("v_scales", None, -1), ("k_scales", FAKE + 2, -3), ("v_scales", FAKE + 1, -3),
                          ("page_table", FAKE + 2, -3), ("n_kv_heads", (1 << 17) + 1, -2), ("n_seqs", (1 << 27) + 1, -2),
                          ("max_pages", 1 << 27, -2)]
NORM = q4.q4_head_norm(1, 1, FAKE, FAKE, 1e-6)


def append(c):
    kind = q4.q4_paged_append8_desc if isinstance(c, q4.q4_paged_cache8) else q4.q4_paged_append_desc
    return kind(c, FAKE, FAKE, 4, None, FAKE, FAKE, 0, 0, FAKE, FAKE, 0, 0, 4, FAKE, 128, 0, 1.0)


def refuse(call, base, bad, make=cache8, cache_bad=CACHE8_BAD, sizes=("ctx_len", "row_start")):
    for f, v, want in bad:
        d = type(base).from_buffer_copy(base)
        setattr(d, f, v)
        assert call(ctypes.byref(d)) == want, (f, v)
        assert q4.lib().q4_last_error() != b""
    for f, v, want in cache_bad:
        d = type(base).from_buffer_copy(base)
        d.cache = make(**{f: v})
        assert call(ctypes.byref(d)) == want, (f, v)
    for f in sizes:
        for v, want in ((None, -1), (FAKE + 2, -3)):
            d = type(base).from_buffer_copy(base)
            setattr(d, f, v)
            assert call(ctypes.byref(d)) == want, f
    d = type(base).from_buffer_copy(base)
    d.rows = -1
    assert call(ctypes.byref(d)) == -1
    assert call(None) == -1


ROWS_BAD = [
    ("k", None, -1), ("v", None, -1), ("q", None, -1), ("q_out", None, -1), ("n_q_heads", 0, -1), ("rot_dim", 130, -1),
    ("rot_dim", 63, -1), ("rot_dim", -2, -1), ("rot_dim", 0, -1), ("freqs", None, -1), ("layout", 2, -1),
    ("amplitude", -1.0, -1), ("amplitude", float("nan"), -1), ("freqs", FAKE + 4, -3), ("k", FAKE + 8, -3),
    ("v", FAKE + 8, -3), ("q", FAKE + 8, -3), ("q_out", FAKE + 8, -3), ("ldk", 255, -1), ("ldk", 260, -3), ("ldv", 8, -1),
    ("ldq", 511, -1), ("ldqo", 513, -3), ("ldq", 1024, -1), ("n_q_heads", 1 << 20, -2), ("positions", FAKE + 1, -3)]


@pytest.mark.parametrize("norm", [None, NORM])
def test_append_refusals(L, norm):
    n = None if norm is None else ctypes.byref(norm)
    refuse(lambda d: L.q4_paged_append8(d, n, None), append(cache8()), ROWS_BAD)
    refuse(lambda d: L.q4_paged_append_norm(d, n, None), append(cache()), ROWS_BAD, cache, CACHE_BAD)


def test_norm_refusals(L):
    for f, v, want in [("eps", -1e-6, -1), ("eps", float("nan"), -1), ("eps", float("inf"), -1), ("q_weight", FAKE + 1, -3),
                       ("k_weight", FAKE + 1, -3)]:
        n = q4.q4_head_norm.from_buffer_copy(NORM)
        setattr(n, f, v)
        assert L.q4_paged_append8(ctypes.byref(append(cache8())), ctypes.byref(n), None) == want, (f, v)
        assert L.q4_paged_append_norm(ctypes.byref(append(cache())), ctypes.byref(n), None) == want, (f, v)


def test_read_refusals(L):
    d = q4.q4_paged_read8_desc(cache8(), FAKE, FAKE, 4, FAKE, FAKE, 0, 0)
    refuse(lambda d: L.q4_paged_read8(d, None), d, [("k", FAKE + 8, -3), ("v", FAKE + 2, -3), ("ldk", 255, -1), ("ldv", 260, -3)],
           sizes=("first", "row_start"))


def attention(need, rows=4):
    return q4.q4_tree_attention8_desc(cache8(), FAKE, FAKE, rows, FAKE, 1, FAKE, FAKE, 0, 0, 4, 0.0, FAKE, need)


def test_attention_refusals(L):
    need = L.q4_tree_attention_workspace_bytes(128)
    refuse(lambda d: L.q4_tree_attention8(d, None), attention(need), [
        ("q", None, -1), ("out", None, -1), ("workspace", None, -1), ("workspace_bytes", need - 1, -1),
        ("workspace", FAKE + 16, -3), ("n_q_heads", 1, -1), ("n_q_heads", 5, -1), ("mask_words", 0, -1),
        ("mask", FAKE + 2, -3), ("scale", -1.0, -1), ("scale", float("inf"), -1), ("scale", float("nan"), -1),
        ("scale", 1e-38, -1), ("ldq", 500, -1), ("ldo", 516, -3), ("q", FAKE + 8, -3), ("out", FAKE + 4, -3),
        ("rows", 2**31 - 1, -2), ("n_q_heads", 1 << 20, -2)])


def accept(layers=2, stride=8 * 16 * 2 * 128, scales=8 * 2):
    return q4.q4_tree_accept8_desc(cache8(), FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, layers, stride, scales)


def test_accept_refusals(L):
    names = ("draft", "parents", "sampled", "accepted", "path", "next_token", "ctx_out")
    refuse(lambda d: L.q4_tree_accept8(d, None), accept(),
           [(f, None, -1) for f in names] + [(f, FAKE + 2, -3) for f in names] +
           [("n_layers", -1, -1), ("n_layers", (1 << 16) + 1, -1), ("layer_stride", 8 * 16 * 2 * 128 - 16, -1),
            ("layer_stride", 8 * 16 * 2 * 128 + 8, -3), ("scale_stride", 15, -1)])


def test_no_rows_need_no_arrays(L):
    # (what a framework's empty tensor gives as its address)
    for call, d in ((lambda d: L.q4_paged_append8(d, None, None), append(cache8())),
                    (lambda d: L.q4_paged_append_norm(d, None, None), append(cache())),
                    (lambda d: L.q4_tree_attention8(d, None), attention(L.q4_tree_attention_workspace_bytes(128))),
                    (lambda d: L.q4_paged_read8(d, None), q4.q4_paged_read8_desc(cache8(), FAKE, FAKE, 4, None, None, 0, 0)),
                    (lambda d: L.q4_tree_accept8(d, None), accept(0))):
        d.rows = 0
        for f in ("k", "v", "q", "q_out", "out", "draft", "parents", "sampled", "path"):
            if hasattr(d, f):
                setattr(d, f, None)
        if isinstance(d, q4.q4_tree_accept8_desc):
            continue  # (sequences without rows are accepted too: it would run where there is a device)
        assert call(ctypes.byref(d)) in (0, -6), L.q4_last_error()


def test_binding_checks_its_tensors(L):
    torch = pytest.importorskip("torch")
    host = torch.zeros(8 * 16 * 2 * 128, dtype=torch.uint8)
    c = q4.PagedCache8(host, FAKE, FAKE, FAKE, 8, 16, 2, 128, FAKE, 2, 4)
    with pytest.raises(ValueError, match="CUDA device memory"):
        q4.q4_paged_read8(c, FAKE, FAKE, 4, FAKE, FAKE)
    c = q4.PagedCache8(FAKE, FAKE, FAKE, FAKE, 8, 16, 2, 128, FAKE, 2, 4)
    with pytest.raises(ValueError, match="CUDA device memory"):
        q4.q4_paged_append8(c, FAKE, FAKE, 4, FAKE, FAKE, norm=q4.HeadNorm(torch.zeros(128, dtype=torch.float16)))
    if torch.cuda.is_available():
        return
    with pytest.raises(q4.Q4Error, match="NO_DEVICE"):
        q4.q4_paged_append8(c, FAKE, FAKE, 4, FAKE, FAKE, norm=q4.HeadNorm())
    with pytest.raises(q4.Q4Error, match="eps"):
        q4.q4_paged_append8(c, FAKE, FAKE, 4, FAKE, FAKE, norm=q4.HeadNorm(eps=-1.0))
    with pytest.raises(q4.Q4Error, match="NO_DEVICE"):
        q4.q4_tree_attention8(c, FAKE, FAKE, 4, FAKE, 4, FAKE, FAKE, 1 << 30)


@pytest.mark.parametrize("packed,kind", [("_APPEND", "q4_paged_append_desc"), ("_ATTENTION", "q4_tree_attention_desc"),
                                         ("_ACCEPT", "q4_tree_accept_desc")])
def test_packed_descriptors_of_the_fp16_cache_are_the_structures(packed, kind):
    values = []

    def build(t):
        out = t()
        for f, ty in t._fields_:
            if issubclass(ty, ctypes.Structure):
                setattr(out, f, build(ty))
                continue
            values.append(0.5 * len(values) + 0.5 if ty is ctypes.c_float else 1000 * len(values) + 7)
            setattr(out, f, values[-1])
        return out

    want = build(getattr(q4, kind))
    assert getattr(q4, packed).pack(*values) == bytes(want)


def test_binding_of_the_fp16_cache_passes_its_arguments_on(L):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        return  # (the addresses below are nobody's)
    c = q4.PagedCache(FAKE, FAKE, 8, 16, 2, 128, FAKE, 2, 4)
    append = lambda **kw: q4.q4_paged_append(c, FAKE, FAKE, 4, FAKE, FAKE, **kw)  # noqa: E731
    for match, call in (("NO_DEVICE", append), ("NULL", lambda: append(q=FAKE)), ("amplitude", lambda: append(amplitude=-1.0)),
                        ("layout", lambda: append(layout=5)),
                        ("NO_DEVICE", lambda: q4.q4_tree_attention(c, FAKE, FAKE, 4, FAKE, 4, FAKE, FAKE, 1 << 30)),
                        ("workspace", lambda: q4.q4_tree_attention(c, FAKE, FAKE, 4, FAKE, 4, FAKE, FAKE, 1 << 10)),
                        ("multiple", lambda: q4.q4_tree_attention(c, FAKE, FAKE, 4, FAKE, 3, FAKE, FAKE, 1 << 30)),
                        ("NO_DEVICE", lambda: q4.q4_tree_accept(c, FAKE, FAKE, 4, *[FAKE] * 7)),
                        ("layer_stride", lambda: q4.q4_tree_accept(c, FAKE, FAKE, 4, *[FAKE] * 7, n_layers=2, layer_stride=8)),
                        ("n_layers", lambda: q4.q4_tree_accept(c, FAKE, FAKE, 4, *[FAKE] * 7, n_layers=-1))):
        with pytest.raises(q4.Q4Error, match=match):
            call()
