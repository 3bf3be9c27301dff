"""Python binding of the Q4 group-64 decode-matmul library (``include/q4.h``).

Argument marshalling only: every function here forwards to the C ABI of
``libq4gb300.so``; each step of the computation runs in the library's CUDA
kernels.  torch tensors are accepted for device buffers (their data pointers
are passed) and the current torch stream is used unless one is given.  There
is no fallback: if the library is missing or a call fails, an exception is
raised.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "Q4Error", "lib", "q4_selftest_expired_wait", "q4_gemv", "q4_gemv8", "q4_gemv_ex", "Segment", "q4_device_status",
    "LayerTable", "q4_decode_step", "q4_decode_workspace_bytes", "q4_decode_buffers",
    "q4_layer_table_release", "q4_decode_path", "q4_moe_route", "q4_moe_route_workspace_bytes",
    "q4_moe_gather", "q4_moe_gemm", "q4_moe_combine",
    "PagedCache", "q4_rope_frequencies", "q4_paged_append", "q4_tree_attention", "q4_tree_attention_workspace_bytes",
    "q4_tree_accept", "q4_sample", "Q4_ROPE_HALF", "Q4_ROPE_INTERLEAVED",
    "Q4_F32", "Q4_F16", "Q4_GEMV_PLAIN", "Q4_GEMV_GLU", "Q4_DECODE_NO_GRAPH", "Q4_DECODE_NO_PDL",
    "Q4_DECODE_TAGGED",
    "Q4_DECODE_PERSISTENT", "Q4_DECODE_CLUSTERED", "Q4_GEMV_EARLY_WEIGHTS",
]

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libq4gb300.so")

Q4_F32, Q4_F16 = 0, 1
Q4_GEMV_PLAIN, Q4_GEMV_GLU = 0, 1
Q4_DECODE_NO_GRAPH, Q4_DECODE_NO_PDL, Q4_DECODE_TAGGED, Q4_DECODE_PERSISTENT = 1, 2, 4, 8
Q4_DECODE_ATTENTION = 16
Q4_DECODE_CLUSTERED = 32
Q4_GEMV_EARLY_WEIGHTS = 1
Q4_MAX_SEGMENTS = 4
Q4_ROPE_HALF, Q4_ROPE_INTERLEAVED = 0, 1

STATUS = {0: "Q4_OK", -1: "Q4_ERR_INVALID_ARG", -2: "Q4_ERR_UNSUPPORTED", -3: "Q4_ERR_MISALIGNED",
          -4: "Q4_ERR_CUDA", -5: "Q4_ERR_TIMEOUT", -6: "Q4_ERR_NO_DEVICE", -7: "Q4_ERR_DEVICE_CHECK"}

# Every symbol include/q4.h declares.
EXPORTS = ["q4_last_error", "q4_status_string", "q4_version", "q4_device_status",
           "q4_selftest_expired_wait", "q4_gemv", "q4_gemv8", "q4_gemv_bits",
           "q4_gemv_ex", "q4_decode_workspace_bytes", "q4_decode_buffers", "q4_decode_step",
           "q4_layer_table_release", "q4_decode_path", "q4_moe_route_workspace_bytes", "q4_moe_route",
           "q4_moe_route_noalloc",
           "q4_moe_gather", "q4_moe_gemm", "q4_moe_combine", "q4_gemm", "q4_prefill_workspace_bytes",
           "q4_prefill", "q4_attention_workspace_bytes", "q4_attention", "q4_gemm_workspace_bytes",
           "q4_prefill_buffers", "q4_rope_frequencies", "q4_paged_append", "q4_tree_attention_workspace_bytes",
           "q4_tree_attention", "q4_tree_accept", "q4_sample"]


class Q4Error(RuntimeError):
    def __init__(self, status: int, where: str, text: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{where}: {self.name}: {text}")


vp = ctypes.c_void_p
i32 = ctypes.c_int


class q4_segment(ctypes.Structure):
    _fields_ = [("Wq", vp), ("scales", vp), ("biases", vp), ("N", i32), ("ldy", i32), ("y", vp),
                ("residual", vp)]


class q4_gemv_desc(ctypes.Structure):
    _fields_ = [("M", i32), ("K", i32), ("x", vp), ("ldx", i32), ("n_segments", i32),
                ("seg", q4_segment * Q4_MAX_SEGMENTS), ("out_dtype", i32), ("mode", i32), ("x_rmsnorm", i32),
                ("norm_weight", vp), ("norm_eps", ctypes.c_float), ("flags", i32)]


class q4_linear(ctypes.Structure):
    _fields_ = [("Wq", vp), ("scales", vp), ("biases", vp), ("N", i32), ("K", i32)]


class q4_layer_weights(ctypes.Structure):
    _fields_ = [(n, q4_linear) for n in ("q", "k", "v", "o", "gate", "up", "down")] + [
        ("attn_norm", vp), ("ffn_norm", vp), ("k_cache", vp), ("v_cache", vp)]


class q4_layer_table(ctypes.Structure):
    _fields_ = [("n_layers", i32), ("hidden", i32), ("M", i32), ("layers", ctypes.POINTER(q4_layer_weights)),
                ("lm_head", q4_linear), ("final_norm", vp), ("norm_eps", ctypes.c_float),
                ("logits_dtype", i32), ("workspace", vp),
                ("workspace_bytes", ctypes.c_size_t), ("flags", i32), ("plan", vp),
                ("head_dim", i32), ("max_seq", i32), ("rope_theta", ctypes.c_float), ("pos", vp)]


class q4_decode_buffers_t(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("h", "h_mid", "q", "k", "v", "act", "a")]


class q4_moe_desc(ctypes.Structure):
    _fields_ = [("E", i32), ("N", i32), ("K", i32), ("R", i32), ("mode", i32), ("out_dtype", i32)]


class q4_attention_desc(ctypes.Structure):
    _fields_ = [("q", vp), ("k", vp), ("v", vp), ("k_cache", vp), ("v_cache", vp), ("pos", vp),
                ("n_q_heads", i32), ("n_kv_heads", i32), ("head_dim", i32), ("max_seq", i32),
                ("rope_theta", ctypes.c_float), ("a", vp), ("workspace", vp), ("workspace_bytes", ctypes.c_size_t)]


class q4_prefill_buffers_t(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("n", "q", "k", "v", "act", "a")]


class q4_gemm_desc(ctypes.Structure):
    _fields_ = [("M", i32), ("X", vp), ("w", q4_linear), ("up", q4_linear), ("mode", i32), ("out_dtype", i32),
                ("Y", vp), ("residual", vp), ("workspace", vp), ("workspace_bytes", ctypes.c_size_t)]


class q4_paged_cache(ctypes.Structure):
    _fields_ = [("k", vp), ("v", vp), ("page_table", vp), ("n_pages", i32), ("page_size", i32), ("n_kv_heads", i32),
                ("head_dim", i32), ("n_seqs", i32), ("max_pages", i32)]


class q4_rope_desc(ctypes.Structure):
    _fields_ = [("rot_dim", i32), ("orig_len", i32)] + [(n, ctypes.c_double)
                                                        for n in ("theta", "factor", "alpha", "beta")]


class q4_paged_append_desc(ctypes.Structure):
    _fields_ = [("cache", q4_paged_cache), ("ctx_len", vp), ("row_start", vp), ("rows", i32), ("positions", vp),
                ("k", vp), ("v", vp), ("ldk", i32), ("ldv", i32), ("q", vp), ("q_out", vp), ("ldq", i32),
                ("ldqo", i32), ("n_q_heads", i32), ("freqs", vp), ("rot_dim", i32), ("layout", i32),
                ("amplitude", ctypes.c_float)]


class q4_tree_attention_desc(ctypes.Structure):
    _fields_ = [("cache", q4_paged_cache), ("ctx_len", vp), ("row_start", vp), ("rows", i32), ("mask", vp),
                ("mask_words", i32), ("q", vp), ("out", vp), ("ldq", i32), ("ldo", i32), ("n_q_heads", i32),
                ("scale", ctypes.c_float), ("workspace", vp), ("workspace_bytes", ctypes.c_size_t)]


class q4_tree_accept_desc(ctypes.Structure):
    _fields_ = [("cache", q4_paged_cache), ("ctx_len", vp), ("row_start", vp), ("rows", i32), ("draft", vp),
                ("parents", vp), ("sampled", vp), ("accepted", vp), ("path", vp), ("next_token", vp),
                ("ctx_out", vp), ("n_layers", i32), ("layer_stride", ctypes.c_size_t)]


class q4_sample_desc(ctypes.Structure):
    _fields_ = [("logits", vp), ("dtype", i32), ("rows", i32), ("vocab", i32), ("ld", i32), ("temperature", vp),
                ("top_k", vp), ("top_p", vp), ("min_p", vp), ("u", vp), ("tokens", vp), ("probs", vp)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load ``libq4gb300.so`` (built by ``build.py``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run bit_quantized_gemv_q4_gb300/build.py "
                              "(or __graft_entry__.build()) first")
        L = ctypes.CDLL(LIB_PATH)
        st = ctypes.c_int
        L.q4_last_error.restype = ctypes.c_char_p
        L.q4_status_string.restype = ctypes.c_char_p
        L.q4_status_string.argtypes = [st]
        L.q4_version.restype = i32
        L.q4_device_status.restype = st
        L.q4_device_status.argtypes = [vp]
        L.q4_selftest_expired_wait.restype = st
        L.q4_selftest_expired_wait.argtypes = [vp]
        L.q4_gemv.restype = st
        L.q4_gemv.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp]
        L.q4_gemv8.restype = st
        L.q4_gemv8.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp]
        L.q4_gemv_bits.restype = st
        L.q4_gemv_bits.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp]
        L.q4_gemv_ex.restype = st
        L.q4_gemv_ex.argtypes = [ctypes.POINTER(q4_gemv_desc), vp]
        L.q4_decode_workspace_bytes.restype = ctypes.c_size_t
        L.q4_decode_workspace_bytes.argtypes = [ctypes.POINTER(q4_layer_table)]
        L.q4_decode_buffers.restype = st
        L.q4_decode_buffers.argtypes = [ctypes.POINTER(q4_layer_table), ctypes.POINTER(q4_decode_buffers_t)]
        L.q4_decode_step.restype = st
        L.q4_decode_step.argtypes = [ctypes.POINTER(q4_layer_table), vp, vp, vp]
        L.q4_layer_table_release.restype = st
        L.q4_layer_table_release.argtypes = [ctypes.POINTER(q4_layer_table)]
        L.q4_decode_path.restype = ctypes.c_int
        L.q4_decode_path.argtypes = [ctypes.POINTER(q4_layer_table)]
        L.q4_moe_route_workspace_bytes.restype = ctypes.c_size_t
        L.q4_moe_route_workspace_bytes.argtypes = [i32, i32, i32]
        L.q4_moe_route.restype = st
        L.q4_moe_route.argtypes = [vp, i32, i32, i32] + [vp] * 7 + [ctypes.c_size_t, vp]
        L.q4_moe_route_noalloc.restype = st
        L.q4_moe_route_noalloc.argtypes = [vp, i32, i32, i32] + [vp] * 6 + [vp]
        L.q4_moe_gather.restype = st
        L.q4_moe_gather.argtypes = [vp, i32, i32, vp, i32, vp, vp]
        L.q4_moe_gemm.restype = st
        L.q4_moe_gemm.argtypes = [vp] * 7 + [ctypes.POINTER(q4_moe_desc), vp]
        L.q4_moe_combine.restype = st
        L.q4_moe_combine.argtypes = [vp, i32, i32, vp, vp, i32, i32, vp, i32, vp]
        L.q4_gemm_workspace_bytes.restype = ctypes.c_size_t
        L.q4_gemm_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.q4_gemm.restype = st
        L.q4_gemm.argtypes = [ctypes.POINTER(q4_gemm_desc), vp]
        L.q4_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.q4_prefill_workspace_bytes.argtypes = [ctypes.POINTER(q4_layer_table), i32]
        L.q4_prefill.restype = st
        L.q4_prefill.argtypes = [ctypes.POINTER(q4_layer_table), vp, i32, i32, vp, vp, ctypes.c_size_t, vp]
        L.q4_prefill_buffers.restype = st
        L.q4_prefill_buffers.argtypes = [ctypes.POINTER(q4_layer_table), i32, vp, ctypes.POINTER(q4_prefill_buffers_t)]
        L.q4_attention_workspace_bytes.restype = ctypes.c_size_t
        L.q4_attention_workspace_bytes.argtypes = [i32, i32, i32]
        L.q4_attention.restype = st
        L.q4_attention.argtypes = [ctypes.POINTER(q4_attention_desc), vp]
        L.q4_rope_frequencies.restype = st
        L.q4_rope_frequencies.argtypes = [ctypes.POINTER(q4_rope_desc), vp, vp]
        L.q4_paged_append.restype = st
        L.q4_paged_append.argtypes = [ctypes.POINTER(q4_paged_append_desc), vp]
        L.q4_tree_attention_workspace_bytes.restype = ctypes.c_size_t
        L.q4_tree_attention_workspace_bytes.argtypes = [i32]
        L.q4_tree_attention.restype = st
        L.q4_tree_attention.argtypes = [ctypes.POINTER(q4_tree_attention_desc), vp]
        L.q4_tree_accept.restype = st
        L.q4_tree_accept.argtypes = [ctypes.POINTER(q4_tree_accept_desc), vp]
        L.q4_sample.restype = st
        L.q4_sample.argtypes = [ctypes.POINTER(q4_sample_desc), vp]
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise Q4Error(status, where, lib().q4_last_error().decode(errors="replace"))


def _ptr(t) -> int | None:
    """Device pointer of a torch tensor in CUDA memory, an int (a raw device
    pointer, passed as is), or None.  A tensor in host memory is refused here:
    the kernels would dereference its address on the device."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"expected a tensor in CUDA device memory, got one on {t.device}")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def q4_device_status(stream=None) -> int:
    """Synchronise and return (and clear) the device error status (0 = ok)."""
    return lib().q4_device_status(_stream(stream))


def q4_selftest_expired_wait(stream=None):
    """Enqueue the bounded-wait self-test (each wait expires after 2 s)."""
    _check(lib().q4_selftest_expired_wait(_stream(stream)), "q4_selftest_expired_wait")


# ------------------------------------------------------------------ GEMV ---

def q4_gemv(Wq, scales, biases, x, y, M: int, N: int, K: int, stream=None):
    _check(lib().q4_gemv(_ptr(Wq), _ptr(scales), _ptr(biases), _ptr(x), _ptr(y), M, N, K, _stream(stream)),
           "q4_gemv")


def q4_gemv8(Wq, scales, biases, x, y, M: int, N: int, K: int, stream=None):
    """q4_gemv for 8-bit codes: Wq uint32 [N, K/4], lowest byte first."""
    _check(lib().q4_gemv8(_ptr(Wq), _ptr(scales), _ptr(biases), _ptr(x), _ptr(y), M, N, K, _stream(stream)),
           "q4_gemv8")


def q4_gemv_bits(Wq, scales, biases, x, y, M: int, N: int, K: int, bits: int, stream=None):
    """q4_gemv for b-bit codes (b in 2, 3, 4, 5, 6, 8): Wq uint32 [N, K*b/32],
    a little-endian bit stream per row."""
    _check(lib().q4_gemv_bits(_ptr(Wq), _ptr(scales), _ptr(biases), _ptr(x), _ptr(y), M, N, K, bits,
                              _stream(stream)), "q4_gemv_bits")


class Segment:
    """One matrix of a fused launch: weights, output, optional fp16 residual."""

    def __init__(self, Wq, scales, biases, N: int, y=None, residual=None, ldy: int = 0):
        self.Wq, self.scales, self.biases, self.N, self.y, self.residual, self.ldy = (
            Wq, scales, biases, N, y, residual, ldy)


def q4_gemv_ex(segments, x, M: int, K: int, out_dtype=Q4_F32, mode=Q4_GEMV_PLAIN, ldx: int = 0,
               rmsnorm: bool = False, norm_weight=None, norm_eps: float = 1e-6, stream=None, flags: int = 0):
    d = q4_gemv_desc()
    d.flags = flags
    d.M, d.K, d.x, d.ldx = M, K, _ptr(x), ldx
    d.x_rmsnorm, d.norm_weight, d.norm_eps = int(rmsnorm), _ptr(norm_weight), norm_eps
    d.n_segments = len(segments)
    for i, s in enumerate(segments):
        d.seg[i] = q4_segment(_ptr(s.Wq), _ptr(s.scales), _ptr(s.biases), s.N, s.ldy, _ptr(s.y),
                              _ptr(s.residual))
    d.out_dtype, d.mode = out_dtype, mode
    _check(lib().q4_gemv_ex(ctypes.byref(d), _stream(stream)), "q4_gemv_ex")


# ---------------------------------------------------------------- decode ---

def _linear(Wq, scales, biases, N, K) -> q4_linear:
    return q4_linear(_ptr(Wq), _ptr(scales), _ptr(biases), N, K)


class LayerTable:
    """Owns a ``q4_layer_table`` and keeps the tensors it points to alive.

    ``layers``: list of dicts name -> (Wq, scales, biases, N, K) for q, k, v,
    o, gate, up, down, and optionally "attn_norm" / "ffn_norm" -> fp16 [hidden]
    device tensors; ``lm_head`` likewise; ``final_norm`` optional."""

    def __init__(self, layers, lm_head, hidden: int, M: int, workspace=None, workspace_bytes: int = 0,
                 logits_dtype=Q4_F32, flags: int = 0, final_norm=None, norm_eps: float = 0.0,
                 head_dim: int = 0, max_seq: int = 0, rope_theta: float = 1.0e6, pos=None):
        self._keep = (layers, lm_head, workspace, final_norm, pos)
        n = len(layers)
        self._arr = (q4_layer_weights * max(n, 1))()
        for i, d in enumerate(layers):
            for nm in ("q", "k", "v", "o", "gate", "up", "down"):
                setattr(self._arr[i], nm, _linear(*d[nm]))
            self._arr[i].attn_norm = _ptr(d.get("attn_norm"))
            self._arr[i].ffn_norm = _ptr(d.get("ffn_norm"))
            self._arr[i].k_cache = _ptr(d.get("k_cache"))
            self._arr[i].v_cache = _ptr(d.get("v_cache"))
        t = q4_layer_table()
        t.n_layers, t.hidden, t.M = n, hidden, M
        t.layers = ctypes.cast(self._arr, ctypes.POINTER(q4_layer_weights))
        t.lm_head = _linear(*lm_head)
        t.final_norm, t.norm_eps = _ptr(final_norm), norm_eps
        t.logits_dtype, t.flags = logits_dtype, flags
        t.workspace, t.workspace_bytes = _ptr(workspace), workspace_bytes
        t.plan = None
        t.head_dim, t.max_seq, t.rope_theta, t.pos = head_dim, max_seq, rope_theta, _ptr(pos)
        self.t = t

    def set_workspace(self, workspace, nbytes: int):
        self._keep = self._keep[:2] + (workspace,) + self._keep[3:]
        self.t.workspace, self.t.workspace_bytes = _ptr(workspace), nbytes

    def release(self):
        q4_layer_table_release(self)

    def __del__(self):
        try:
            if self.t.plan:
                lib().q4_layer_table_release(ctypes.byref(self.t))
        except Exception:
            pass


def q4_decode_workspace_bytes(table: LayerTable) -> int:
    n = lib().q4_decode_workspace_bytes(ctypes.byref(table.t))
    if n == 0:
        raise Q4Error(-1, "q4_decode_workspace_bytes", lib().q4_last_error().decode())
    return n


def q4_decode_buffers(table: LayerTable) -> dict:
    b = q4_decode_buffers_t()
    _check(lib().q4_decode_buffers(ctypes.byref(table.t), ctypes.byref(b)), "q4_decode_buffers")
    return {n: getattr(b, n) for n in ("h", "h_mid", "q", "k", "v", "act", "a")}


def q4_decode_step(table: LayerTable, x, logits, stream=None):
    _check(lib().q4_decode_step(ctypes.byref(table.t), _ptr(x), _ptr(logits), _stream(stream)), "q4_decode_step")


def q4_decode_path(table: LayerTable) -> int:
    """0 = not planned, 1 = per-stage launches, 2 = persistent launch, 3 = clustered step + lm_head."""
    return lib().q4_decode_path(ctypes.byref(table.t))


def q4_layer_table_release(table: LayerTable):
    _check(lib().q4_layer_table_release(ctypes.byref(table.t)), "q4_layer_table_release")


# ------------------------------------------------------------------- MoE ---

def q4_moe_route_workspace_bytes(T: int, E: int, topk: int) -> int:
    return lib().q4_moe_route_workspace_bytes(T, E, topk)


def q4_moe_route(logits, T, E, topk, topk_ids, topk_weights, offsets, token_of, expert_of, pos, workspace,
                 workspace_bytes, stream=None):
    _check(lib().q4_moe_route(_ptr(logits), T, E, topk, _ptr(topk_ids), _ptr(topk_weights), _ptr(offsets),
                              _ptr(token_of), _ptr(expert_of), _ptr(pos), _ptr(workspace), workspace_bytes,
                              _stream(stream)), "q4_moe_route")


def q4_moe_route_noalloc(logits, T, E, topk, topk_ids, topk_weights, offsets, token_of, expert_of, pos,
                         stream=None):
    """q4_moe_route with the library's static scratch instead of a workspace."""
    _check(lib().q4_moe_route_noalloc(_ptr(logits), T, E, topk, _ptr(topk_ids), _ptr(topk_weights), _ptr(offsets),
                                      _ptr(token_of), _ptr(expert_of), _ptr(pos), _stream(stream)),
           "q4_moe_route_noalloc")


def q4_moe_gather(X, T, K, token_of, R, X_sorted, stream=None):
    _check(lib().q4_moe_gather(_ptr(X), T, K, _ptr(token_of), R, _ptr(X_sorted), _stream(stream)),
           "q4_moe_gather")


def q4_moe_gemm(Wq, scales, biases, X, expert_ids, offsets, Y, E, N, K, R, mode=Q4_GEMV_PLAIN,
                out_dtype=Q4_F32, stream=None):
    d = q4_moe_desc(E, N, K, R, mode, out_dtype)
    _check(lib().q4_moe_gemm(_ptr(Wq), _ptr(scales), _ptr(biases), _ptr(X), _ptr(expert_ids), _ptr(offsets),
                             _ptr(Y), ctypes.byref(d), _stream(stream)), "q4_moe_gemm")


def q4_moe_combine(Y, y_dtype, N, pos, topk_weights, T, topk, out, out_dtype, stream=None):
    _check(lib().q4_moe_combine(_ptr(Y), y_dtype, N, _ptr(pos), _ptr(topk_weights), T, topk, _ptr(out),
                                out_dtype, _stream(stream)), "q4_moe_combine")


# --------------------------------------------------------------- prefill ---

def q4_gemm_workspace_bytes(M: int, N: int, K: int, mode=Q4_GEMV_PLAIN) -> int:
    return lib().q4_gemm_workspace_bytes(M, N, K, mode)


def q4_gemm(w, X, Y, M: int, mode=Q4_GEMV_PLAIN, out_dtype=Q4_F32, up=None, residual=None, workspace=None,
            workspace_bytes: int = 0, stream=None):
    """Dense Y[M, N] = X[M, K] W^T on the tensor cores.  ``w`` (and ``up`` in
    GLU mode) are (Wq, scales, biases, N, K); a workspace lets K split."""
    d = q4_gemm_desc()
    d.M, d.X, d.w = M, _ptr(X), _linear(*w)
    if up is not None:
        d.up = _linear(*up)
    d.mode, d.out_dtype, d.Y, d.residual = mode, out_dtype, _ptr(Y), _ptr(residual)
    d.workspace, d.workspace_bytes = _ptr(workspace), workspace_bytes
    _check(lib().q4_gemm(ctypes.byref(d), _stream(stream)), "q4_gemm")


def q4_prefill_workspace_bytes(table: LayerTable, chunk: int) -> int:
    n = lib().q4_prefill_workspace_bytes(ctypes.byref(table.t), chunk)
    if n == 0:
        raise Q4Error(-1, "q4_prefill_workspace_bytes", lib().q4_last_error().decode())
    return n


def q4_prefill(table: LayerTable, h, T: int, chunk: int, logits, workspace, workspace_bytes: int, stream=None):
    """Chunked prefill: h fp16 [T, hidden] in place; logits of the last token (or None)."""
    _check(lib().q4_prefill(ctypes.byref(table.t), _ptr(h), T, chunk, _ptr(logits), _ptr(workspace),
                            workspace_bytes, _stream(stream)), "q4_prefill")


# ------------------------------------------------------------- attention ---

def q4_attention_workspace_bytes(n_q_heads: int, head_dim: int, max_seq: int) -> int:
    return lib().q4_attention_workspace_bytes(n_q_heads, head_dim, max_seq)


def q4_attention(q, k, v, k_cache, v_cache, pos, n_q_heads: int, n_kv_heads: int, head_dim: int, max_seq: int,
                 a, workspace, workspace_bytes: int, rope_theta: float = 1.0e6, stream=None):
    """One token's cache append and decode attention (pos: device int32, not advanced)."""
    d = q4_attention_desc(_ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(pos), n_q_heads,
                          n_kv_heads, head_dim, max_seq, rope_theta, _ptr(a), _ptr(workspace), workspace_bytes)
    _check(lib().q4_attention(ctypes.byref(d), _stream(stream)), "q4_attention")


def q4_prefill_buffers(table: LayerTable, chunk: int, workspace) -> dict:
    b = q4_prefill_buffers_t()
    _check(lib().q4_prefill_buffers(ctypes.byref(table.t), chunk, _ptr(workspace), ctypes.byref(b)),
           "q4_prefill_buffers")
    return {n: getattr(b, n) for n in ("n", "q", "k", "v", "act", "a")}


# ----------------------------------------- paged cache, trees, sampling ---
#
# A call here takes a dozen tensors and its kernel a few microseconds, so the
# checks of a plain argument (element type, current device, contiguous, large
# enough) are four attribute reads in _arg / _rows; whatever does not pass them
# goes to the functions behind, which say what is wrong or find the stride.

_torch = None


def _get_torch():
    """torch, imported at the first call that needs it."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _stream_of(torch, dev: int, stream):
    """_stream without building a torch Stream object, which costs as much as a launch."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else None
    return _stream(stream)


def _arg_other(t, dtype, need: int, dev: int, name: str):
    """Pointer of an argument that is not a plain contiguous tensor of its type, or the error."""
    torch = _get_torch()
    p = _ptr(t)
    same = {torch.int32: (torch.int32, torch.uint32), torch.int64: (torch.int64, torch.uint64)}
    # words: the signed type of the same width holds the same bits
    kinds = same[dtype] if name in ("mask", "freqs") else (dtype,)
    if dtype is not None and t.dtype not in kinds:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < need:
        raise ValueError(f"{name}: holds {t.numel()} elements, the call needs {need}")
    return p


def _device(torch) -> int:
    """The current device; -2, which is no tensor's, where there is none."""
    cuda = torch.cuda
    return cuda.current_device() if cuda.is_initialized() or cuda.is_available() else -2


def _arg(t, dtype, need: int, dev: int, name: str):
    """Device pointer of a packed argument of at least `need` elements; ints and None pass as in _ptr."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is dtype and t.get_device() == dev and t.numel() >= need and t.is_contiguous():
        return t.data_ptr()
    return _arg_other(t, dtype, need, dev, name)


def _rows_other(t, dtype, rows: int, width: int, ld: int, dev: int, name: str):
    p = _ptr(t)
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if t.dim() == 2 and not ld:
        ld = t.stride(0) if t.size(0) > 1 else max(width, t.size(1))
    elif t.dim() != 2 and not t.is_contiguous():
        raise ValueError(f"{name}: give a [rows][width] view or a contiguous tensor")
    if t.numel() and t.size(-1) != 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    need = (rows - 1) * (ld or width) + width if rows > 0 else 0
    have = 1 + sum((n - 1) * st for n, st in zip(t.shape, t.stride())) if t.numel() else 0
    if have < need:
        raise ValueError(f"{name}: reaches over {have} elements, the call needs {need}")
    return p, ld


def _rows(t, dtype, rows: int, width: int, ld: int, dev: int, name: str):
    """(device pointer, row stride) of a matrix argument; a 2-D tensor's own stride unless one is given."""
    if t is None or t.__class__ is int:
        return t, ld
    if (not ld and t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.size(-1) == width
            and t.numel() >= rows * width):
        return t.data_ptr(), width
    return _rows_other(t, dtype, rows, width, ld, dev, name)


class PagedCache:
    """Key / value pools fp16 [n_pages][n_kv_heads][page_size][head_dim] (for
    q4_tree_accept one such pool per layer, layer_stride elements apart) and
    the sequences' page table int32 [n_seqs][max_pages]; keeps the tensors."""

    __slots__ = ("k", "v", "page_table", "sizes", "pool")

    def __init__(self, k, v, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, page_table, n_seqs: int,
                 max_pages: int):
        self.k, self.v, self.page_table = k, v, page_table
        self.sizes = (n_pages, page_size, n_kv_heads, head_dim, n_seqs, max_pages)
        self.pool = n_pages * page_size * n_kv_heads * head_dim  # elements of one layer's keys

    def _desc(self, torch, dev: int, elements: int) -> q4_paged_cache:
        s = self.sizes
        return q4_paged_cache(_arg(self.k, torch.float16, elements, dev, "cache.k"),
                              _arg(self.v, torch.float16, elements, dev, "cache.v"),
                              _arg(self.page_table, torch.int32, s[4] * s[5], dev, "cache.page_table"), *s)


def q4_rope_frequencies(freqs, rot_dim: int, theta: float = 1.0e6, factor: float = 1.0, orig_len: int = 0,
                        alpha: float = 1.0, beta: float = 32.0, stream=None):
    """freqs: int64 (or uint64) [rot_dim / 2] out, turns per position in units of 2^-64."""
    torch = _get_torch()
    d = q4_rope_desc(rot_dim, orig_len, theta, factor, alpha, beta)
    dev = _device(torch)
    p = _arg(freqs, torch.int64, rot_dim // 2, dev, "freqs")
    _check(lib().q4_rope_frequencies(ctypes.byref(d), p, _stream_of(torch, dev, stream)), "q4_rope_frequencies")


def q4_paged_append(cache: PagedCache, ctx_len, row_start, rows: int, k, v, q=None, q_out=None, n_q_heads: int = 0,
                    positions=None, freqs=None, rot_dim: int = 0, layout=Q4_ROPE_HALF, amplitude: float = 1.0,
                    ldq: int = 0, ldk: int = 0, ldv: int = 0, ldqo: int = 0, stream=None):
    """New rows' keys (rotated) and values into the paged cache, queries (rotated) into q_out."""
    torch = _get_torch()
    dev = _device(torch)
    f16, i32_ = torch.float16, torch.int32
    _, _, heads, hd, n_seqs, _ = cache.sizes
    pk, ldk = _rows(k, f16, rows, heads * hd, ldk, dev, "k")
    pv, ldv = _rows(v, f16, rows, heads * hd, ldv, dev, "v")
    pq, ldq = _rows(q, f16, rows, n_q_heads * hd, ldq, dev, "q")
    po, ldqo = _rows(q_out, f16, rows, n_q_heads * hd, ldqo, dev, "q_out")
    d = q4_paged_append_desc(
        cache._desc(torch, dev, cache.pool), _arg(ctx_len, i32_, n_seqs, dev, "ctx_len"),
        _arg(row_start, i32_, n_seqs + 1, dev, "row_start"), rows, _arg(positions, i32_, rows, dev, "positions"), pk, pv,
        ldk, ldv, pq, po, ldq, ldqo, n_q_heads, _arg(freqs, torch.int64, rot_dim // 2, dev, "freqs"), rot_dim, layout,
        amplitude)
    _check(lib().q4_paged_append(ctypes.byref(d), _stream_of(torch, dev, stream)), "q4_paged_append")


def q4_tree_attention_workspace_bytes(head_dim: int) -> int:
    return lib().q4_tree_attention_workspace_bytes(head_dim)


def q4_tree_attention(cache: PagedCache, ctx_len, row_start, rows: int, q, n_q_heads: int, out, workspace,
                      workspace_bytes: int, mask=None, mask_words: int = 0, scale: float = 0.0, ldq: int = 0,
                      ldo: int = 0, stream=None):
    """Attention of the new rows over the cached positions and, by the mask (None: causal), their own."""
    torch = _get_torch()
    dev = _device(torch)
    f16, i32_ = torch.float16, torch.int32
    w, n_seqs = n_q_heads * cache.sizes[3], cache.sizes[4]
    pq, ldq = _rows(q, f16, rows, w, ldq, dev, "q")
    po, ldo = _rows(out, f16, rows, w, ldo, dev, "out")
    if workspace is not None and workspace.__class__ is not int:
        if workspace.numel() * workspace.element_size() < workspace_bytes:
            raise ValueError(f"workspace: smaller than {workspace_bytes} bytes")
        workspace = _arg(workspace, workspace.dtype, 0, dev, "workspace")
    d = q4_tree_attention_desc(
        cache._desc(torch, dev, cache.pool), _arg(ctx_len, i32_, n_seqs, dev, "ctx_len"),
        _arg(row_start, i32_, n_seqs + 1, dev, "row_start"), rows, _arg(mask, i32_, rows * mask_words, dev, "mask"),
        mask_words, pq, po, ldq, ldo, n_q_heads, scale, workspace, workspace_bytes)
    _check(lib().q4_tree_attention(ctypes.byref(d), _stream_of(torch, dev, stream)), "q4_tree_attention")


def q4_tree_accept(cache: PagedCache, ctx_len, row_start, rows: int, draft, parents, sampled, accepted, path,
                   next_token, ctx_out, n_layers: int = 1, layer_stride: int = 0, stream=None):
    """Walks each sequence's drafted tree along the sampled tokens and moves the path's cache rows into place."""
    torch = _get_torch()
    dev = _device(torch)
    i32_, n_seqs = torch.int32, cache.sizes[4]
    elements = (n_layers - 1) * layer_stride + cache.pool if n_layers > 0 else 0
    d = q4_tree_accept_desc(
        cache._desc(torch, dev, elements), _arg(ctx_len, i32_, n_seqs, dev, "ctx_len"),
        _arg(row_start, i32_, n_seqs + 1, dev, "row_start"), rows, _arg(draft, i32_, rows, dev, "draft"),
        _arg(parents, i32_, rows, dev, "parents"), _arg(sampled, i32_, rows, dev, "sampled"),
        _arg(accepted, i32_, n_seqs, dev, "accepted"), _arg(path, i32_, rows, dev, "path"),
        _arg(next_token, i32_, n_seqs, dev, "next_token"), _arg(ctx_out, i32_, n_seqs, dev, "ctx_out"), n_layers,
        layer_stride)
    _check(lib().q4_tree_accept(ctypes.byref(d), _stream_of(torch, dev, stream)), "q4_tree_accept")


def q4_sample(logits, dtype, rows: int, vocab: int, tokens, temperature=None, top_k=None, top_p=None, min_p=None,
              u=None, probs=None, ld: int = 0, stream=None):
    """One token per row of logits (q4.h section 8); u: fp32 random numbers of [0, 1), None = the greatest logit."""
    torch = _get_torch()
    dev = _device(torch)
    f32, i32_ = torch.float32, torch.int32
    p, ld = _rows(logits, torch.float16 if dtype == Q4_F16 else f32, rows, vocab, ld, dev, "logits")
    d = q4_sample_desc(p, dtype, rows, vocab, ld, _arg(temperature, f32, rows, dev, "temperature"),
                       _arg(top_k, i32_, rows, dev, "top_k"), _arg(top_p, f32, rows, dev, "top_p"),
                       _arg(min_p, f32, rows, dev, "min_p"), _arg(u, f32, rows, dev, "u"),
                       _arg(tokens, i32_, rows, dev, "tokens"), _arg(probs, f32, rows, dev, "probs"))
    _check(lib().q4_sample(ctypes.byref(d), _stream_of(torch, dev, stream)), "q4_sample")
