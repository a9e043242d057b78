"""Python binding of libfusedlin, the fused transformer dense layer for GB300.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libfusedlin.so (built in-tree by gemm_epilogue_tma_gb300._build).
PyTorch supplies device memory and the current stream. If the library is
missing, every call raises; there is no fallback path.

Entry points mirror the C ABI declared in include/fusedlin.h:
    gemm_epilogue(A, W, bias, residual, out, pattern)   seven GEMM-first patterns
    norm_gemm(x, gamma, W, beta, bias, out, eps, norm, act)
    norm_gemm_multi(x, gamma, Ws, beta, biases, outs, acts, eps, norm)   one norm, several weights
    input_bias_gemm(A, bias_in, W, bias, residual, out, act)             (A + bias_in) W^T epilogue
    rms_norm(x, gamma, out, eps)                                          standalone RMSNorm
    swiglu_ffn(x, gamma, Wg, Wu, Wd, bias_down, out, eps, workspace)
    w4_quantize(W, group)                                                 16-bit weight -> 4-bit codes, group scales
    w4_gemm(x, q, scales, zeros, gamma, bias, residual, out, eps, act)    dense layer on a 4-bit weight
    w4_swiglu_ffn(x, gamma, Wg, Wu, Wd, bias_down, out, eps, workspace)   the SwiGLU block on 4-bit weights
    rope(q, k, positions, inv_freq, sections)                             rotary positions, one to four axes
    kv_write / kv_read                                                    paged 8-bit key/value cache
"""
from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfusedlin.so")

PATTERNS = (
    "gemm_bias_gelu", "gemm_bias_silu", "gemm_bias_relu", "gemm_bias", "gemm_bias_residual",
    "gemm_gelu", "gemm_silu", "layernorm_gemm", "rmsnorm_gemm",
)
NORMS = {"rms": 0, "layer": 1}
ACTS = {"none": 0, "gelu": 1, "silu": 2, "relu": 3}
DTYPE_CODES = {"f16": 0, "bf16": 1}
STATUS_NAMES = {0: "FL_OK", 1: "FL_ERR_INVALID_ARG", 2: "FL_ERR_UNSUPPORTED", 3: "FL_ERR_ALIGNMENT",
                4: "FL_ERR_WORKSPACE", 5: "FL_ERR_CUDA", 6: "FL_ERR_TIMEOUT", 7: "FL_ERR_RANGE"}
OPTIONS = {"tile_n": 0, "variant": 1, "timeout_ms": 2, "split_k": 3, "pdl": 4, "weight_preload": 5,
           "launch_cache": 6}

class LayerDesc(ctypes.Structure):
    """fl_layer_desc: sizes, dtype, eps and the device pointers of one decoder layer's dense part."""
    _fields_ = [("dtype", ctypes.c_int), ("M", ctypes.c_int), ("D", ctypes.c_int), ("Dkv", ctypes.c_int),
                ("F", ctypes.c_int), ("eps", ctypes.c_float)] + [
        (name, ctypes.c_void_p) for name in ("x", "gamma_attn", "Wq", "Wk", "Wv", "q", "k", "v", "attn", "Wo",
                                             "bias_o", "h", "gamma_ffn", "Wg", "Wu", "Wd", "out")]


class W4Weight(ctypes.Structure):
    """fl_w4_weight: the device pointers of one 4-bit weight."""
    _fields_ = [("q", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("group", ctypes.c_int)]


class RopeDesc(ctypes.Structure):
    """fl_rope_desc."""
    _fields_ = ([(n, ctypes.c_int) for n in ("dtype", "rows", "heads_q", "heads_k", "head_dim", "rotary_dim", "n_axes",
                                             "interleaved", "inverse")]
                + [("axis_of", ctypes.c_char_p), ("positions", ctypes.c_void_p), ("positions_stride", ctypes.c_longlong),
                   ("inv_freq", ctypes.c_void_p)]
                + [(n, ctypes.c_void_p) for n in ("q", "k", "q_out", "k_out")]
                + [(n, ctypes.c_longlong) for n in ("q_row", "q_head", "k_row", "k_head", "q_out_row", "q_out_head",
                                                    "k_out_row", "k_out_head")])


class KvDesc(ctypes.Structure):
    """fl_kv_desc."""
    _fields_ = ([(n, ctypes.c_int) for n in ("dtype", "format", "rows", "heads", "head_dim", "page_size", "n_pages",
                                             "n_seqs", "table_pages")]
                + [("table_stride", ctypes.c_longlong)]
                + [(n, ctypes.c_void_p) for n in ("page_table", "cu_rows", "start", "k", "v")]
                + [(n, ctypes.c_longlong) for n in ("k_row", "k_head", "v_row", "v_head")]
                + [(n, ctypes.c_void_p) for n in ("k_cache", "v_cache", "k_scale", "v_scale")])


class LayerCacheDesc(ctypes.Structure):
    """fl_layer_cache_desc."""
    _fields_ = ([(n, ctypes.c_int) for n in ("head_dim", "rotary_dim", "n_axes", "interleaved")]
                + [("axis_of", ctypes.c_char_p), ("positions", ctypes.c_void_p), ("positions_stride", ctypes.c_longlong),
                   ("inv_freq", ctypes.c_void_p)]
                + [(n, ctypes.c_int) for n in ("format", "page_size", "n_pages", "n_seqs", "table_pages")]
                + [("table_stride", ctypes.c_longlong)]
                + [(n, ctypes.c_void_p) for n in ("page_table", "cu_rows", "start", "k_cache", "v_cache", "k_scale",
                                                  "v_scale")])


# C ABI: name -> (restype, argtypes)
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_w4 = ctypes.POINTER(W4Weight)
SIGNATURES = {
    "fl_gemm_epilogue": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "fl_norm_gemm": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _f, _i, _i, _i, _vp]),
    "fl_swiglu_ffn_workspace_size": (_sz, [_i, _i, _i]),
    "fl_swiglu_ffn": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _f, _vp, _sz, _i, _vp]),
    "fl_swiglu_ffn_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _f, _i, _vp]),
    "fl_norm_gemm_multi": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _f, _i, _i, _vp]),
    "fl_input_bias_gemm": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "fl_rms_norm": (_i, [_vp, _vp, _vp, _i, _i, _f, _i, _vp]),
    "fl_w4_quantize": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "fl_w4_gemm_workspace_size": (_sz, [_i, _i, _i]),
    "fl_w4_gemm": (_i, [_vp, _vp, _w4, _vp, _vp, _vp, _i, _i, _i, _f, _i, _vp, _sz, _i, _vp]),
    "fl_w4_swiglu_ffn_workspace_size": (_sz, [_i, _i, _i]),
    "fl_w4_swiglu_ffn": (_i, [_vp, _vp, _w4, _w4, _w4, _vp, _vp, _i, _i, _i, _f, _vp, _sz, _i, _vp]),
    "fl_rope": (_i, [ctypes.POINTER(RopeDesc), _vp]),
    "fl_kv_write": (_i, [ctypes.POINTER(KvDesc), _vp]),
    "fl_kv_read": (_i, [ctypes.POINTER(KvDesc), _vp]),
    "fl_layer_create": (_i, [ctypes.POINTER(LayerDesc), ctypes.POINTER(_vp)]),
    "fl_layer_attach_cache": (_i, [_vp, ctypes.POINTER(LayerCacheDesc)]),
    "fl_layer_issue": (_i, [_vp, _i, _vp]),
    "fl_layer_destroy": (None, [_vp]),
    "fl_capture_begin": (_i, [_vp]),
    "fl_capture_end": (_i, [_vp, ctypes.POINTER(_vp)]),
    "fl_graph_launch": (_i, [_vp, _vp]),
    "fl_graph_destroy": (None, [_vp]),
    "fl_launch_cache_stats": (_i, [ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(ctypes.c_longlong)]),
    "fl_launch_cache_clear": (None, []),
    "fl_kernel_launches": (_i, [ctypes.POINTER(ctypes.c_longlong)]),
    "fl_last_error": (ctypes.c_char_p, []),
    "fl_device_status": (_i, [_vp]),
    "fl_set_option": (_i, [_i, _i]),
    "fl_debug_wait_timeout": (_i, [_i, _vp]),
    "fl_version": (ctypes.c_char_p, []),
}


class FusedLinError(RuntimeError):
    """A libfusedlin call returned a non-OK status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m gemm_epilogue_tma_gb300._build` (needs nvcc)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype, fn.argtypes = res, args
        _lib = handle
    return _lib


def last_error() -> str:
    return lib().fl_last_error().decode()


def version() -> str:
    return lib().fl_version().decode()


def _check(status: int) -> None:
    if status != 0:
        raise FusedLinError(status, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    """The raw handle of `stream`, or of the current stream of the current device. (Read directly: building the
    Stream object that torch.cuda.current_stream() returns takes as long as a launch.)"""
    if stream is None:
        from torch import _C
        return _C._cuda_getCurrentRawStream(_C._cuda_getDevice())
    return stream.cuda_stream


_captures = []  # of each Graph.capture at work: what the calls made for themselves, which every replay uses


def _made(t):
    """t (a tensor, several, or what holds them), which a call made for itself. A graph under capture keeps it: replays
    write and read that memory, and torch's allocator, which does not know of the capture, would hand it to others."""
    for kept in _captures:
        kept.append(t)
    return t


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return 0
    if t.dtype == torch.bfloat16:
        return 1
    raise TypeError(f"libfusedlin computes on fp16 or bf16 tensors, got {t.dtype}")


def _check_tensors(dt_ref, **tensors):
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous (row-major)")
        if t.dtype != dt_ref:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dt_ref}")


def gemm_epilogue(A, W, bias=None, residual=None, out=None, pattern="gemm_bias_gelu", stream=None):
    """out[M,N] = epilogue(A[M,K] W[N,K]^T) for a GEMM-first pattern name or enum value."""
    import torch
    p = PATTERNS.index(pattern) if isinstance(pattern, str) else int(pattern)
    M, K = A.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W has shape {tuple(W.shape)}, expected [N, {K}]")
    if out is None:
        out = _made(torch.empty((M, N), dtype=A.dtype, device=A.device))
    _check_tensors(A.dtype, A=A, W=W, bias=bias, residual=residual, out=out)
    _check(lib().fl_gemm_epilogue(_ptr(A), _ptr(W), _ptr(bias), _ptr(residual), _ptr(out), M, N, K, p,
                                  _dtype_code(A), _stream(stream)))
    return out


def norm_gemm(x, gamma, W, beta=None, bias=None, out=None, eps=1e-6, norm="rms", act="none", stream=None):
    """out[M,N] = act(norm(x)[M,K] W[N,K]^T + bias); norm "rms" or "layer"."""
    import torch
    M, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W has shape {tuple(W.shape)}, expected [N, {K}]")
    if out is None:
        out = _made(torch.empty((M, N), dtype=x.dtype, device=x.device))
    _check_tensors(x.dtype, x=x, gamma=gamma, W=W, beta=beta, bias=bias, out=out)
    _check(lib().fl_norm_gemm(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(W), _ptr(bias), _ptr(out), M, N, K,
                              float(eps), NORMS[norm], ACTS[act], _dtype_code(x), _stream(stream)))
    return out


MAX_OUTPUTS = 4


def norm_gemm_multi(x, gamma, Ws, beta=None, biases=None, outs=None, acts=None, eps=1e-6, norm="rms", stream=None):
    """outs[i][M,N_i] = act_i(norm(x) Ws[i]^T + biases[i]) for every weight in one launch."""
    import torch
    n = len(Ws)
    if not 1 <= n <= MAX_OUTPUTS:
        raise ValueError(f"1..{MAX_OUTPUTS} weights, got {n}")
    M, K = x.shape
    for i, W in enumerate(Ws):
        if W.shape[1] != K:
            raise ValueError(f"Ws[{i}] has shape {tuple(W.shape)}, expected [N, {K}]")
    if outs is None:
        outs = _made([torch.empty((M, W.shape[0]), dtype=x.dtype, device=x.device) for W in Ws])
    biases = list(biases) if biases is not None else [None] * n
    acts = list(acts) if acts is not None else ["none"] * n
    if len(outs) != n or len(biases) != n or len(acts) != n:
        raise ValueError("Ws, outs, biases and acts must have the same length")
    _check_tensors(x.dtype, x=x, gamma=gamma, beta=beta,
                   **{f"W{i}": W for i, W in enumerate(Ws)}, **{f"out{i}": o for i, o in enumerate(outs)},
                   **{f"bias{i}": b for i, b in enumerate(biases)})
    arr = ctypes.c_void_p * n
    W_arr = arr(*[W.data_ptr() for W in Ws])
    b_arr = arr(*[(b.data_ptr() if b is not None else None) for b in biases])
    o_arr = arr(*[o.data_ptr() for o in outs])
    N_arr = (ctypes.c_int * n)(*[W.shape[0] for W in Ws])
    a_arr = (ctypes.c_int * n)(*[ACTS[a] for a in acts])
    _check(lib().fl_norm_gemm_multi(_ptr(x), _ptr(gamma), _ptr(beta), n, W_arr, b_arr, o_arr, N_arr, a_arr, M, K,
                                    float(eps), NORMS[norm], _dtype_code(x), _stream(stream)))
    return outs


def input_bias_gemm(A, bias_in, W, bias=None, residual=None, out=None, act="none", stream=None):
    """out[M,N] = act((A + bias_in) W^T + bias) (+ residual); bias_in runs along K."""
    import torch
    M, K = A.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W has shape {tuple(W.shape)}, expected [N, {K}]")
    if out is None:
        out = _made(torch.empty((M, N), dtype=A.dtype, device=A.device))
    _check_tensors(A.dtype, A=A, bias_in=bias_in, W=W, bias=bias, residual=residual, out=out)
    _check(lib().fl_input_bias_gemm(_ptr(A), _ptr(bias_in), _ptr(W), _ptr(bias), _ptr(residual), _ptr(out), M, N,
                                    K, ACTS[act], _dtype_code(A), _stream(stream)))
    return out


def rms_norm(x, gamma, out=None, eps=1e-6, stream=None):
    """out[M,K] = x * gamma / sqrt(mean(x^2) + eps), rounded once (out may be x)."""
    import torch
    M, K = x.shape
    if out is None:
        out = _made(torch.empty_like(x))
    _check_tensors(x.dtype, x=x, gamma=gamma, out=out)
    _check(lib().fl_rms_norm(_ptr(x), _ptr(gamma), _ptr(out), M, K, float(eps), _dtype_code(x), _stream(stream)))
    return out


class DecoderLayer:
    """The dense part of a decoder layer as a prepared call sequence (fl_layer_*).

    half 0: q, k, v = RMSNorm(x) [Wq; Wk; Wv]^T; the caller's attention then
    writes attn; half 1: h = attn Wo^T (+ bias_o) + x, out = SwiGLU_FFN(h) + h.
    Every tensor is fixed for the life of the layer: write new inputs into x
    and attn in place. Capture whole steps with Graph.capture().
    """

    NAMES = ("x", "gamma_attn", "Wq", "Wk", "Wv", "q", "k", "v", "attn", "Wo", "bias_o", "h", "gamma_ffn", "Wg",
             "Wu", "Wd", "out")

    def __init__(self, eps=1e-6, **tensors):
        x = tensors["x"]
        M, D = x.shape
        F = tensors["Wg"].shape[0]
        Dkv = tensors["Wk"].shape[0]
        _check_tensors(x.dtype, **tensors)
        self.tensors = tensors  # keep every buffer alive while the graphs exist
        desc = LayerDesc(dtype=_dtype_code(x), M=M, D=D, Dkv=Dkv, F=F, eps=float(eps),
                         **{n: (tensors[n].data_ptr() if tensors.get(n) is not None else None) for n in self.NAMES})
        h = ctypes.c_void_p()
        _check(lib().fl_layer_create(ctypes.byref(desc), ctypes.byref(h)))
        self._h = h
        self.attached = ()

    def attach_cache(self, head_dim, positions=None, inv_freq=None, sections=None, interleaved=False, k_cache=None,
                     v_cache=None, k_scale=None, v_scale=None, page_table=None, start=None, cu_rows=None) -> None:
        """Half 0 then also rotates q and k in place (rope's positions, inv_freq, sections, interleaved) and writes k
        and v into the paged cache (kv_write's tensors; cu_rows None: one row per sequence). Either part may be left
        out; with neither, a part attached before is taken off. The tensors stay fixed: write new positions, pages and
        starts into them in place."""
        import torch
        T = self.tensors
        here = T["x"].device
        if inv_freq is None and k_cache is None:
            _check(lib().fl_layer_attach_cache(self._h, None))
            self.attached = ()
            return
        if int(head_dim) < 1 or T["q"].shape[1] % head_dim or T["k"].shape[1] % head_dim:
            raise ValueError(f"head_dim {head_dim} must divide the widths of q and k")
        d = LayerCacheDesc(head_dim=head_dim)
        kept = []

        def use(name, t, dtype, shape=None, contiguous=True):
            if t.device != here or t.dtype != dtype:
                raise ValueError(f"{name} must be a {dtype} tensor on {here}, got {t.dtype} on {t.device}")
            if contiguous and not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if shape is not None and tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
            kept.append(t)
            return t.data_ptr()

        M = T["x"].shape[0]
        if inv_freq is not None:
            if positions is None or positions.dim() not in (1, 2) or inv_freq.dim() != 1:
                raise ValueError("positions [rows] or [axes, rows] and inv_freq [pairs] must be given")
            pairs, axes = inv_freq.shape[0], positions.shape[0] if positions.dim() == 2 else 1
            sections = (pairs,) if sections is None and axes == 1 else sections
            if sections is None or len(sections) != axes or sum(sections) != pairs or min(sections) < 0 or axes > 4:
                raise ValueError(f"sections must give the {pairs} pairs to the {axes} axes (1..4)")
            d.rotary_dim, d.n_axes, d.interleaved = 2 * pairs, axes, int(bool(interleaved))
            d.axis_of = b"".join(bytes((a,)) * n for a, n in enumerate(sections))
            if M > 1 and positions.stride(-1) != 1:
                raise ValueError("positions must be contiguous along the rows")
            d.positions = use("positions", positions, torch.int32, (axes, M) if positions.dim() == 2 else (M,), contiguous=False)
            d.positions_stride = positions.stride(0) if positions.dim() == 2 else M
            d.inv_freq = use("inv_freq", inv_freq, torch.float32, (pairs,))
        if k_cache is not None:
            formats = {torch.int8: 0, torch.float8_e4m3fn: 1}
            if k_cache.dtype not in formats:
                raise ValueError(f"k_cache has dtype {k_cache.dtype}, expected int8 or float8_e4m3fn")
            if start is None or page_table is None or v_cache is None or k_scale is None or v_scale is None:
                raise ValueError("v_cache, k_scale, v_scale, page_table and start must be given")
            if k_cache.dim() != 4 or page_table.dim() != 2:
                raise ValueError("k_cache must have four axes and page_table two")
            pages, size = k_cache.shape[:2]
            seqs, per = page_table.shape
            shape = (pages, size, T["k"].shape[1] // head_dim, head_dim)
            d.format, d.page_size, d.n_pages, d.n_seqs, d.table_pages = formats[k_cache.dtype], size, pages, seqs, per
            d.table_stride = per
            d.page_table = use("page_table", page_table, torch.int32)
            d.start = use("start", start, torch.int32, (seqs,))
            d.cu_rows = None if cu_rows is None else use("cu_rows", cu_rows, torch.int32, (seqs + 1,))
            d.k_cache, d.v_cache = (use(n, t, k_cache.dtype, shape) for n, t in (("k_cache", k_cache), ("v_cache", v_cache)))
            d.k_scale, d.v_scale = (use(n, t, torch.float32, shape[:3]) for n, t in (("k_scale", k_scale),
                                                                                     ("v_scale", v_scale)))
        _check(lib().fl_layer_attach_cache(self._h, ctypes.byref(d)))
        self.attached = tuple(kept)  # kept alive as long as the layer uses them

    def issue(self, half: int, stream=None) -> None:
        """Issue half 0 or 1 on the stream (capturable; the graph keeps the layer and what is attached to it now)."""
        _made((self, self.attached))
        _check(lib().fl_layer_issue(self._h, int(half), _stream(stream)))

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().fl_layer_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Graph:
    """A CUDA graph of library calls (fl_capture_begin / fl_capture_end / fl_graph_launch)."""

    def __init__(self, handle):
        self._h = handle

    @classmethod
    def capture(cls, fn, stream=None):
        """Run fn() (which issues library calls on `stream`) under capture; returns the graph.
        The stream must not be the legacy default stream (CUDA cannot capture it). The graph keeps what the calls make for
        themselves (outputs and workspaces not given) and the layers issued, with what is attached to them, until it is
        closed; tensors that fn is given or makes by other means are the caller's to keep."""
        s = _stream(stream)
        _check(lib().fl_capture_begin(s))
        kept = []
        _captures.append(kept)
        try:
            fn()
        finally:
            _captures[:] = [c for c in _captures if c is not kept]
            h = ctypes.c_void_p()
            st = lib().fl_capture_end(s, ctypes.byref(h))
        _check(st)
        graph = cls(h)
        graph._kept = kept
        return graph

    def launch(self, stream=None) -> None:
        _check(lib().fl_graph_launch(self._h, _stream(stream)))

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().fl_graph_destroy(self._h)
            self._h = None
            self._kept = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def swiglu_ffn_workspace_size(M: int, F: int, dtype) -> int:
    import torch
    code = {torch.float16: 0, torch.bfloat16: 1}.get(dtype, DTYPE_CODES.get(dtype))
    return int(lib().fl_swiglu_ffn_workspace_size(M, F, code))


def swiglu_ffn(x, gamma, Wg, Wu, Wd, bias_down=None, out=None, eps=1e-6, workspace=None, stream=None):
    """Llama-style SwiGLU FFN block: out = (silu(xh Wg^T) * (xh Wu^T)) Wd^T (+ bias_down) + x."""
    import torch
    M, D = x.shape
    F = Wg.shape[0]
    if out is None:
        out = _made(torch.empty_like(x))
    need = swiglu_ffn_workspace_size(M, F, x.dtype)
    if workspace is None:
        workspace = _made(torch.empty(need, dtype=torch.uint8, device=x.device))
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _check_tensors(x.dtype, x=x, gamma=gamma, Wg=Wg, Wu=Wu, Wd=Wd, bias_down=bias_down, out=out)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().fl_swiglu_ffn(_ptr(x), _ptr(gamma), _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(bias_down), _ptr(out),
                               M, D, F, float(eps), _ptr(workspace), ws_bytes, _dtype_code(x), _stream(stream)))
    return out


def swiglu_ffn_noalloc(x, gamma, Wg, Wu, Wd, bias_down=None, out=None, eps=1e-6, stream=None):
    """swiglu_ffn for callers that may not allocate device memory: h lives in the
    library's fixed 8 MiB device array (M * F * 2 bytes at most). Calls whose
    kernels overlap on the GPU race on that array."""
    import torch
    M, D = x.shape
    F = Wg.shape[0]
    if out is None:
        out = _made(torch.empty_like(x))
    _check_tensors(x.dtype, x=x, gamma=gamma, Wg=Wg, Wu=Wu, Wd=Wd, bias_down=bias_down, out=out)
    _check(lib().fl_swiglu_ffn_noalloc(_ptr(x), _ptr(gamma), _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(bias_down),
                                       _ptr(out), M, D, F, float(eps), _dtype_code(x), _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# serving operators: 4-bit weights, rotary positions, the quantised cache
# ---------------------------------------------------------------------------
_ops = None


def ops():
    """The extension module that passes torch tensors to the operators below (raises if it has not been built)."""
    global _ops
    if _ops is None:
        import torch  # noqa: F401  (its libraries are loaded first)
        lib()
        try:
            from . import _torch_binding
        except ImportError as e:
            raise ImportError(f"gemm_epilogue_tma_gb300/_torch_binding.so cannot be loaded ({e}): build it with "
                              "`python -m gemm_epilogue_tma_gb300._build`") from e
        _torch_binding.set_error(FusedLinError)
        _ops = _torch_binding
    return _ops


def _on(stream, name, args, makes=True):
    """ops().name(*args) on `stream`. Tensors that the call makes for itself (makes: it may) are `stream`'s, as those of
    any torch call under torch.cuda.stream(stream). (Calls on the current stream take no detour through here: it would
    add a tenth to the host time of the shortest ones.)"""
    f = getattr(ops(), name)
    if not makes:
        return f(*args, stream.cuda_stream)
    import torch
    with torch.cuda.stream(stream):
        return f(*args, None)


def _output(r):
    """The output of a call that returns it with the workspace it made, or None."""
    if _captures:
        _made(r)
    return r[0]


def w4_quantize(W, group=128, q=None, scales=None, stream=None):
    """Symmetric round-to-nearest 4-bit quantisation of W [N, K]: returns (q, scales), codes [N, K / 2] uint8 (two
    along K to a byte, the even k in the low half, 8 standing for zero) and one scale of W's dtype per `group` k."""
    if stream is None:
        r = (_ops or ops()).w4_quantize(W, group, q, scales, None)
    else:
        r = _on(stream, "w4_quantize", (W, group, q, scales), q is None or scales is None)
    return _made(r) if _captures else r


def w4_gemm_workspace_size(M: int, K: int, norm: bool) -> int:
    return int(lib().fl_w4_gemm_workspace_size(M, K, int(norm)))


def w4_gemm(x, q, scales, zeros=None, gamma=None, bias=None, residual=None, out=None, eps=1e-6, act="none",
            workspace=None, stream=None):
    """out[M,N] = act(norm(x) W^T + bias) (+ residual) with W[n, k] = scales[n, k / group] * (code[n, k] -
    zeros[n, k / group]); norm is RMSNorm with `gamma`, or none. q, scales: as w4_quantize returns them; zeros
    [N, K / group] uint8 (8 everywhere if None). The workspace (w4_gemm_workspace_size bytes) must not be
    shared by calls or captured graphs that may overlap on the GPU."""
    if stream is None:
        return _output((_ops or ops()).w4_gemm(x, q, scales, zeros, gamma, bias, residual, out, eps, ACTS[act], workspace,
                                               None))
    return _output(_on(stream, "w4_gemm", (x, q, scales, zeros, gamma, bias, residual, out, eps, ACTS[act], workspace),
                       out is None or workspace is None))


def w4_swiglu_ffn_workspace_size(M: int, D: int, F: int) -> int:
    return int(lib().fl_w4_swiglu_ffn_workspace_size(M, D, F))


def w4_swiglu_ffn(x, gamma, Wg, Wu, Wd, bias_down=None, out=None, eps=1e-6, workspace=None, stream=None):
    """swiglu_ffn on 4-bit weights, each a tuple (q, scales) or (q, scales, zeros)."""
    if stream is None:
        return _output((_ops or ops()).w4_swiglu_ffn(x, gamma, Wg, Wu, Wd, bias_down, out, eps, workspace, None))
    return _output(_on(stream, "w4_swiglu_ffn", (x, gamma, Wg, Wu, Wd, bias_down, out, eps, workspace),
                       out is None or workspace is None))


def rope(q, k, positions, inv_freq, sections=None, interleaved=False, inverse=False, out_q=None, out_k=None,
         stream=None):
    """Rotary positions of q [rows, heads_q, D] and k [rows, heads_k, D] (k may be None): returns (out_q, out_k).

    The pairs (i, i + R/2) of the first R = 2 * len(inv_freq) channels, or (2i, 2i + 1) if interleaved, are turned
    by positions * inv_freq[i]; the other channels are copied. positions: int32 [rows], or [axes, rows] with
    `sections` saying how many consecutive pairs follow each axis (rows contiguous; one row expanded to the axes will
    do). inverse turns back: the gradient with respect to the input. q, k and the outputs may be strided views with
    contiguous channels (column ranges of a stacked projection's output); an output may be its input itself."""
    if stream is None:
        r = (_ops or ops()).rope(q, k, positions, inv_freq, sections, interleaved, inverse, out_q, out_k, None)
    else:
        r = _on(stream, "rope", (q, k, positions, inv_freq, sections, interleaved, inverse, out_q, out_k),
                out_q is None or (out_k is None and k is not None))
    return _made(r) if _captures else r


def kv_write(k, v, k_cache, v_cache, k_scale, v_scale, page_table, start, cu_rows=None, stream=None):
    """Quantises rows of k and v [rows, heads, head_dim] into the paged cache.

    k_cache, v_cache: int8 or float8_e4m3fn [pages, page_size, heads, head_dim]; k_scale, v_scale: fp32
    [pages, page_size, heads]. Row i of sequence b (cu_rows[b] <= i < cu_rows[b + 1]; without cu_rows, row b) is
    position start[b] + i - cu_rows[b] of it, in page page_table[b][position / page_size]. Rows behind the
    last sequence are left out; one whose position has no page is skipped and device_status() raises FL_ERR_RANGE.
    No two rows of a call may have the same place in the cache."""
    if start is None:
        raise ValueError("start must be given")
    (_ops or ops()).kv_write(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_rows, start,
                             None if stream is None else stream.cuda_stream)


def kv_read(k_cache, v_cache, k_scale, v_scale, page_table, cu_rows, start=None, out_k=None, out_v=None, stream=None):
    """Reads rows of the cache back (scale * code) into out_k, out_v [rows, heads, head_dim]: row i of the outputs is
    the position start[b] + i - cu_rows[b] (start: 0 if None) of the sequence b that cu_rows gives it to; with
    cu_rows None it is position start[i] of sequence i. Rows that belong to no sequence are left as they were.
    Returns (out_k, out_v)."""
    if out_k is None or out_v is None:
        raise ValueError("out_k and out_v must be given: the row count is not known on the host")
    (_ops or ops()).kv_read(out_k, out_v, k_cache, v_cache, k_scale, v_scale, page_table, cu_rows, start,
                            None if stream is None else stream.cuda_stream)
    return out_k, out_v


def launch_cache_stats():
    """(hits, misses) of the host-side launch cache since the library was loaded."""
    h, m = ctypes.c_longlong(), ctypes.c_longlong()
    _check(lib().fl_launch_cache_stats(ctypes.byref(h), ctypes.byref(m)))
    return h.value, m.value


def launch_cache_clear() -> None:
    lib().fl_launch_cache_clear()


def kernel_launches() -> int:
    """Kernels the library has launched (or recorded into a capture) since it was loaded."""
    n = ctypes.c_longlong()
    _check(lib().fl_kernel_launches(ctypes.byref(n)))
    return n.value


def device_status(stream=None) -> None:
    """Synchronise the stream and raise FusedLinError: FL_ERR_TIMEOUT if a kernel's wait ran out, FL_ERR_RANGE if a
    row of the paged cache had no page."""
    _check(lib().fl_device_status(_stream(stream)))


def set_option(key: str, value: int) -> None:
    _check(lib().fl_set_option(OPTIONS[key], int(value)))


def debug_wait_timeout(limit_us: int, stream=None) -> None:
    """Launch the bounded-wait probe (a wait nothing completes); read the result with device_status()."""
    _check(lib().fl_debug_wait_timeout(int(limit_us), _stream(stream)))
