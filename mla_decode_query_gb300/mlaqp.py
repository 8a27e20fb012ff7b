"""ctypes binding of ``libmlaqp.so`` (declared in ``include/mlaqp.h`` and ``include/mlaqp_kv4.h``).

Argument marshalling only: every function here forwards to the C entry point
of the same name and returns its status code unchanged; all of the operation
runs in the library's CUDA kernels.  Tensor arguments may be ``torch.Tensor``
objects on the GPU (their ``data_ptr()`` is passed) or raw integer device
addresses; ``None`` passes NULL.  ``stream=None`` means PyTorch's current
CUDA stream.

If the library has not been built the first call raises ``RuntimeError``:
there is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import re
import threading
from pathlib import Path

from .build import INCLUDE, LIB_PATH

MLAQP_WEIGHT_BF16 = 0
MLAQP_WEIGHT_MXFP8 = 1
MLAQP_OUT_BF16 = 0
MLAQP_OUT_E4M3 = 1

MLAQP_OK = 0
MLAQP_ERR_UNSUPPORTED = 1
MLAQP_ERR_INVALID_ARG = 2
MLAQP_ERR_CUDA = 3

MLAQP_DEVSTATUS_WAIT_TIMEOUT = 1
MLAQP_DEVSTATUS_BAD_INDEX = 2
MLAQP_DEVSTATUS_OUT_OF_PAGES = 4

NOPE_DIM = 128
LATENT_DIM = 512
ROPE_DIM = 64
OUT_DIM = 576
MAX_M = 256
MAX_M_DECODE = 32
V_HEAD_DIM = 128

WEIGHT_FORMATS = {"bf16": MLAQP_WEIGHT_BF16, "mxfp8": MLAQP_WEIGHT_MXFP8}
OUT_DTYPES = {"bf16": MLAQP_OUT_BF16, "e4m3": MLAQP_OUT_E4M3}

_lock = threading.Lock()
_lib = None

_c_void_p = ctypes.c_void_p
_c_int = ctypes.c_int
_c_int64 = ctypes.c_int64
# block_table, its stride, num_seqs, seq_lens, ref_count, num_pages, page_size
_KV4_TABLES = [_c_void_p, _c_int64, _c_int, _c_void_p, _c_void_p, _c_int, _c_int]
# cache, page_stride, layer_stride, layers
_KV4_POOL = [_c_void_p, _c_int64, _c_int64, _c_int]
# q, its stride, q_dtype, q_scale; one layer's cache; tables; sizes; x, lse, workspace
_KV4_ATTEND = [_c_void_p, _c_int64, _c_int, _c_void_p, _c_void_p, _c_int64, _c_int, _c_int, _c_void_p, _c_int64, _c_int,
               _c_void_p, _c_void_p, _c_int, _c_int, _c_int, ctypes.c_float, _c_void_p, _c_int64, _c_void_p, _c_void_p,
               _c_int64]
_SIGNATURES = {
    "mlaqp_can_implement": (_c_int, [_c_int] * 8),
    "mlaqp_prewarm": (_c_int, [_c_int] * 5),
    "mlaqp_run": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.c_int64,
                           _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    "mlaqp_run_pdl": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.c_int64,
                               _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    "mlaqp_run_strided": (_c_int, [_c_void_p, ctypes.c_int64, ctypes.c_int64, _c_void_p, ctypes.c_int64,
                                   ctypes.c_int64, _c_void_p, _c_void_p, _c_void_p, ctypes.c_int64, _c_void_p,
                                   _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    "mlaqp_debug_run_arm": (_c_int, [_c_void_p, ctypes.c_int64, ctypes.c_int64, _c_void_p, ctypes.c_int64,
                                     ctypes.c_int64, _c_void_p, _c_void_p, _c_void_p, ctypes.c_int64, _c_void_p,
                                     _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    "mlaqp_debug_set_policy": (_c_int, [_c_int, _c_int]),
    "mlaqp_prefetch_weights": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    "mlaqp_launch_shape": (_c_int, [_c_int, _c_int, _c_int, _c_int, ctypes.POINTER(_c_int),
                                    ctypes.POINTER(_c_int)]),
    "mlaqp_debug_plan": (_c_int, [_c_int] * 8 + [ctypes.POINTER(_c_int)] * 6),
    "mlaqp_debug_v_plan": (_c_int, [_c_int] * 5 + [ctypes.POINTER(_c_int)] * 7),
    "mlaqp_device_status": (_c_int, [ctypes.POINTER(ctypes.c_uint), _c_int]),
    "mlaqp_debug_run_bounded_wait": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                              ctypes.c_int64, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                              ctypes.c_ulonglong, ctypes.c_uint, _c_void_p]),
    "mlaqp_debug_launch_null": (_c_int, [_c_int, _c_int, _c_int, _c_void_p]),
    "mlaqp_v_up_run": (_c_int, [_c_void_p, ctypes.c_int64, ctypes.c_int64, _c_void_p, _c_void_p, _c_void_p,
                                ctypes.c_int64, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    "mlaqp_v_up_can_implement": (_c_int, [_c_int] * 4),
    "mlaqp_v_up_prewarm": (_c_int, [_c_int] * 4),
    "mlaqp_debug_v_up_bounded_wait": (_c_int, [_c_void_p, ctypes.c_int64, ctypes.c_int64, _c_void_p, _c_void_p,
                                               _c_void_p, ctypes.c_int64, _c_int, _c_int, _c_int,
                                               ctypes.c_ulonglong, ctypes.c_uint, _c_void_p]),
    "mlaqp_kv4_page_bytes": (_c_int64, [_c_int]),
    "mlaqp_kv4_append": (_c_int, [_c_void_p, _c_int64, _c_void_p, _c_int64, _c_void_p, _c_int64, _c_int, _c_int,
                                  _c_void_p, _c_int, _c_void_p]),
    "mlaqp_kv4_gather": (_c_int, [_c_void_p, _c_int64, _c_int, _c_int, _c_void_p, _c_int, _c_void_p, _c_int64,
                                  _c_void_p]),
    "mlaqp_kv4_attend": (_c_int, _KV4_ATTEND + [_c_void_p]),
    "mlaqp_debug_kv4_attend_bounded_wait": (_c_int, _KV4_ATTEND + [ctypes.c_uint, _c_int, _c_void_p]),
    "mlaqp_kv4_attend_workspace": (_c_int64, [_c_int] * 4),
    "mlaqp_kv4_extend": (_c_int, _KV4_TABLES + [_c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p]),
    "mlaqp_kv4_fork": (_c_int, _KV4_TABLES + [_c_void_p, _c_void_p, _c_int] + _KV4_POOL
                       + [_c_void_p, _c_int64, _c_void_p]),
    "mlaqp_kv4_release": (_c_int, _KV4_TABLES + [_c_void_p, _c_int, _c_void_p]),
    "mlaqp_kv4_compact": (_c_int, _KV4_TABLES + _KV4_POOL + [_c_void_p, _c_void_p, _c_int64, _c_void_p]),
    "mlaqp_kv4_copy_pages": (_c_int, _KV4_POOL + [_c_int, _c_int, _c_void_p, _c_void_p, _c_int, _c_void_p]),
    "mlaqp_kv4_pages_workspace": (_c_int64, [_c_int, _c_int]),
    "mlaqp_kv4_prewarm": (_c_int, [_c_int]),
    "mlaqp_last_error": (ctypes.c_char_p, []),
    "mlaqp_version": (_c_int, []),
}


def header_functions(header: Path | None = None) -> list[str]:
    """Names of the functions ``include/*.h`` declares (parsed from text)."""
    names = []
    for h in ([header] if header else sorted(INCLUDE.glob("*.h"))):
        text = re.sub(r"/\*.*?\*/", "", Path(h).read_text(), flags=re.S)
        names += re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(mlaqp_\w+)\s*\(", text, flags=re.M)
    return names


def load_library(path: Path | str | None = None) -> ctypes.CDLL:
    """Load ``libmlaqp.so`` once and attach the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = Path(path) if path else LIB_PATH
        if not p.exists():
            raise RuntimeError(
                f"{p} is missing: build the CUDA library first "
                "(python -m mla_decode_query_gb300.build, or __graft_entry__.build())")
        lib = ctypes.CDLL(str(p))
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _ptr(x) -> int | None:
    if x is None or type(x) is int:
        return x
    try:
        return x.data_ptr()
    except AttributeError:
        pass
    if isinstance(x, int):
        return x
    raise TypeError(f"expected a tensor, an int address or None, got {type(x)!r}")


_current_stream = None


def _find_current_stream():
    """The handle of PyTorch's current stream.  Building the Stream object that
    torch.cuda.current_stream() returns takes 2.8 us (on the Arm host of a
    GB300), longer than a launch; the raw handle takes 0.2 us."""
    global _current_stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = torch.cuda.current_device
    if raw is None:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    else:
        _current_stream = lambda: raw(device())  # noqa: E731
    return _current_stream


def _stream(stream) -> int | None:
    if stream is None:
        return (_current_stream or _find_current_stream())()
    if isinstance(stream, int):
        return stream
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    raise TypeError(f"expected a torch.cuda.Stream, an int handle or None, got {type(stream)!r}")


def _fmt(v, table) -> int:
    return table[v] if isinstance(v, str) else int(v)


def mlaqp_can_implement(num_heads, max_m, nope_dim=NOPE_DIM, latent_dim=LATENT_DIM, rope_dim=ROPE_DIM,
                        weight_format="bf16", out_dtype="bf16", device=-1) -> int:
    return load_library().mlaqp_can_implement(num_heads, max_m, nope_dim, latent_dim, rope_dim,
                                              _fmt(weight_format, WEIGHT_FORMATS),
                                              _fmt(out_dtype, OUT_DTYPES), device)


def mlaqp_prewarm(num_heads, max_m, weight_format="bf16", out_dtype="bf16", device=-1) -> int:
    return load_library().mlaqp_prewarm(num_heads, max_m, _fmt(weight_format, WEIGHT_FORMATS),
                                        _fmt(out_dtype, OUT_DTYPES), device)


def _run_args(q_nope, q_pe, weight, weight_scale, out, out_row_stride, q_scale, M, H, weight_format,
              out_dtype):
    return (_ptr(q_nope), _ptr(q_pe), _ptr(weight), _ptr(weight_scale), _ptr(out), int(out_row_stride),
            _ptr(q_scale), int(M), int(H), _fmt(weight_format, WEIGHT_FORMATS), _fmt(out_dtype, OUT_DTYPES))


def mlaqp_run(q_nope, q_pe, weight, weight_scale, out, out_row_stride, q_scale, M, H, weight_format,
              out_dtype, stream=None) -> int:
    a = _run_args(q_nope, q_pe, weight, weight_scale, out, out_row_stride, q_scale, M, H, weight_format,
                  out_dtype)
    return load_library().mlaqp_run(*a, _stream(stream))


def mlaqp_run_pdl(q_nope, q_pe, weight, weight_scale, out, out_row_stride, q_scale, M, H, weight_format,
                  out_dtype, stream=None) -> int:
    a = _run_args(q_nope, q_pe, weight, weight_scale, out, out_row_stride, q_scale, M, H, weight_format,
                  out_dtype)
    return load_library().mlaqp_run_pdl(*a, _stream(stream))


def mlaqp_run_strided(q_nope, q_nope_token_stride, q_nope_head_stride, q_pe, q_pe_token_stride, q_pe_head_stride,
                      weight, weight_scale, out, out_row_stride, q_scale, M, H, nope_dim, weight_format, out_dtype,
                      pdl=False, stream=None) -> int:
    return load_library().mlaqp_run_strided(
        _ptr(q_nope), int(q_nope_token_stride), int(q_nope_head_stride), _ptr(q_pe), int(q_pe_token_stride),
        int(q_pe_head_stride), _ptr(weight), _ptr(weight_scale), _ptr(out), int(out_row_stride), _ptr(q_scale),
        int(M), int(H), int(nope_dim), _fmt(weight_format, WEIGHT_FORMATS), _fmt(out_dtype, OUT_DTYPES),
        int(pdl), _stream(stream))


def mlaqp_prefetch_weights(weight, weight_scale, H, nope_dim, weight_format, pdl=False, stream=None) -> int:
    return load_library().mlaqp_prefetch_weights(_ptr(weight), _ptr(weight_scale), int(H), int(nope_dim),
                                                 _fmt(weight_format, WEIGHT_FORMATS), int(pdl),
                                                 _stream(stream))


ARMS = {"auto": 0, "warp_mma": 1, "warp_fma": 2, "cta_mma": 3, "tcgen05": 4}


def mlaqp_debug_run_arm(q_nope, q_nope_token_stride, q_nope_head_stride, q_pe, q_pe_token_stride, q_pe_head_stride,
                        weight, weight_scale, out, out_row_stride, q_scale, M, H, nope_dim, weight_format, out_dtype,
                        pdl=False, arm="auto", stream=None) -> int:
    return load_library().mlaqp_debug_run_arm(
        _ptr(q_nope), int(q_nope_token_stride), int(q_nope_head_stride), _ptr(q_pe), int(q_pe_token_stride),
        int(q_pe_head_stride), _ptr(weight), _ptr(weight_scale), _ptr(out), int(out_row_stride), _ptr(q_scale),
        int(M), int(H), int(nope_dim), _fmt(weight_format, WEIGHT_FORMATS), _fmt(out_dtype, OUT_DTYPES),
        int(pdl), _fmt(arm, ARMS), _stream(stream))


def mlaqp_debug_set_policy(trig, cta_cap) -> int:
    return load_library().mlaqp_debug_set_policy(int(trig), int(cta_cap))


def mlaqp_debug_run_bounded_wait(q_nope, q_pe, weight, weight_scale, out, out_row_stride, q_scale, M, H,
                                 weight_format, out_dtype, wait_limit_ns, extra_tx_bytes, stream=None) -> int:
    a = _run_args(q_nope, q_pe, weight, weight_scale, out, out_row_stride, q_scale, M, H, weight_format,
                  out_dtype)
    return load_library().mlaqp_debug_run_bounded_wait(*a, int(wait_limit_ns), int(extra_tx_bytes),
                                                       _stream(stream))


def mlaqp_debug_launch_null(ctas, threads, pdl, stream=None) -> int:
    return load_library().mlaqp_debug_launch_null(int(ctas), int(threads), int(pdl), _stream(stream))


def mlaqp_v_up_run(x, x_token_stride, x_head_stride, weight, weight_scale, out, out_row_stride, M, H,
                   weight_format, pdl=False, stream=None) -> int:
    return load_library().mlaqp_v_up_run(_ptr(x), int(x_token_stride), int(x_head_stride), _ptr(weight),
                                         _ptr(weight_scale), _ptr(out), int(out_row_stride), int(M), int(H),
                                         _fmt(weight_format, WEIGHT_FORMATS), int(pdl), _stream(stream))


def mlaqp_v_up_can_implement(num_heads, max_m, weight_format="bf16", device=-1) -> int:
    return load_library().mlaqp_v_up_can_implement(num_heads, max_m, _fmt(weight_format, WEIGHT_FORMATS), device)


def mlaqp_v_up_prewarm(num_heads, max_m, weight_format="bf16", device=-1) -> int:
    return load_library().mlaqp_v_up_prewarm(num_heads, max_m, _fmt(weight_format, WEIGHT_FORMATS), device)


def mlaqp_debug_v_up_bounded_wait(x, x_token_stride, x_head_stride, weight, weight_scale, out, out_row_stride, M,
                                  H, weight_format, wait_limit_ns, extra_tx_bytes, stream=None) -> int:
    return load_library().mlaqp_debug_v_up_bounded_wait(
        _ptr(x), int(x_token_stride), int(x_head_stride), _ptr(weight), _ptr(weight_scale), _ptr(out),
        int(out_row_stride), int(M), int(H), _fmt(weight_format, WEIGHT_FORMATS), int(wait_limit_ns),
        int(extra_tx_bytes), _stream(stream))


def mlaqp_launch_shape(M, H, weight_format="bf16", out_dtype="bf16"):
    """Returns ``(status, grid_ctas, threads_per_cta)``."""
    g, t = _c_int(0), _c_int(0)
    st = load_library().mlaqp_launch_shape(int(M), int(H), _fmt(weight_format, WEIGHT_FORMATS),
                                           _fmt(out_dtype, OUT_DTYPES), ctypes.byref(g), ctypes.byref(t))
    return st, g.value, t.value


ARM_NAMES = {v: k for k, v in ARMS.items()}


def mlaqp_debug_plan(M, H, weight_format="bf16", out_dtype="bf16", nope_dim=128, pdl=1, arm="auto", sm_count=152):
    """The launch a query call would make on a device with ``sm_count`` SMs
    (host-side, no device).  Returns ``(status, plan)`` with plan a dict:
    arm (name), chunk_tokens, trig, cta_cap, grid_ctas, threads_per_cta."""
    out = [_c_int(0) for _ in range(6)]
    st = load_library().mlaqp_debug_plan(int(M), int(H), int(nope_dim), _fmt(weight_format, WEIGHT_FORMATS),
                                         _fmt(out_dtype, OUT_DTYPES), int(pdl), _fmt(arm, ARMS), int(sm_count),
                                         *[ctypes.byref(o) for o in out])
    keys = ("arm", "chunk_tokens", "trig", "cta_cap", "grid_ctas", "threads_per_cta")
    plan = {k: o.value for k, o in zip(keys, out)}
    plan["arm"] = ARM_NAMES.get(plan["arm"], plan["arm"])
    return st, plan


V_FORMS = {0: "plain", 1: "multicast", 2: "cluster"}


def mlaqp_debug_v_plan(M, H, weight_format="bf16", pdl=1, sm_count=152):
    """As mlaqp_debug_plan for a V call with contiguous x.  Returns
    ``(status, plan)``: form (plain / multicast / cluster), chunk_tokens,
    trig, cta_cap, grid_ctas, threads_per_cta, cluster."""
    out = [_c_int(0) for _ in range(7)]
    st = load_library().mlaqp_debug_v_plan(int(M), int(H), _fmt(weight_format, WEIGHT_FORMATS), int(pdl),
                                           int(sm_count), *[ctypes.byref(o) for o in out])
    keys = ("form", "chunk_tokens", "trig", "cta_cap", "grid_ctas", "threads_per_cta", "cluster")
    plan = {k: o.value for k, o in zip(keys, out)}
    plan["form"] = V_FORMS.get(plan["form"], plan["form"])
    return st, plan


def mlaqp_kv4_page_bytes(page_size) -> int:
    return load_library().mlaqp_kv4_page_bytes(int(page_size))


def mlaqp_kv4_append(latent, latent_token_stride, k_pe, k_pe_token_stride, cache, page_stride, num_pages, page_size,
                     slots, T, stream=None) -> int:
    return load_library().mlaqp_kv4_append(
        _ptr(latent), int(latent_token_stride), _ptr(k_pe), int(k_pe_token_stride), _ptr(cache), int(page_stride),
        int(num_pages), int(page_size), _ptr(slots), int(T), _stream(stream))


def mlaqp_kv4_gather(cache, page_stride, num_pages, page_size, slots, T, out, out_token_stride, stream=None) -> int:
    return load_library().mlaqp_kv4_gather(_ptr(cache), int(page_stride), int(num_pages), int(page_size), _ptr(slots),
                                           int(T), _ptr(out), int(out_token_stride), _stream(stream))


def mlaqp_kv4_attend(q, q_token_stride, q_dtype, q_scale, cache, page_stride, num_pages, page_size, block_table,
                     block_table_stride, num_seqs, seq_lens, seqs, B, q_len, H, softmax_scale, x, x_token_stride, lse,
                     workspace, workspace_bytes, stream=None) -> int:
    return load_library().mlaqp_kv4_attend(
        _ptr(q), int(q_token_stride), _fmt(q_dtype, OUT_DTYPES), _ptr(q_scale), _ptr(cache), int(page_stride),
        int(num_pages), int(page_size), _ptr(block_table), int(block_table_stride), int(num_seqs), _ptr(seq_lens),
        _ptr(seqs), int(B), int(q_len), int(H), float(softmax_scale), _ptr(x), int(x_token_stride), _ptr(lse),
        _ptr(workspace), int(workspace_bytes), _stream(stream))


def mlaqp_debug_kv4_attend_bounded_wait(q, q_token_stride, q_dtype, q_scale, cache, page_stride, num_pages, page_size,
                                        block_table, block_table_stride, num_seqs, seq_lens, seqs, B, q_len, H,
                                        softmax_scale, x, x_token_stride, lse, workspace, workspace_bytes,
                                        wait_limit_ns, held, stream=None) -> int:
    return load_library().mlaqp_debug_kv4_attend_bounded_wait(
        _ptr(q), int(q_token_stride), _fmt(q_dtype, OUT_DTYPES), _ptr(q_scale), _ptr(cache), int(page_stride),
        int(num_pages), int(page_size), _ptr(block_table), int(block_table_stride), int(num_seqs), _ptr(seq_lens),
        _ptr(seqs), int(B), int(q_len), int(H), float(softmax_scale), _ptr(x), int(x_token_stride), _ptr(lse),
        _ptr(workspace), int(workspace_bytes), int(wait_limit_ns), int(held), _stream(stream))


def mlaqp_kv4_attend_workspace(B, q_len, H, device=-1) -> int:
    """Bytes of workspace, or -1 (see ``mlaqp_last_error``)."""
    return load_library().mlaqp_kv4_attend_workspace(int(B), int(q_len), int(H), int(device))


def _kv4_tables(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size):
    return (_ptr(block_table), int(block_table_stride), int(num_seqs), _ptr(seq_lens), _ptr(ref_count), int(num_pages),
            int(page_size))


def mlaqp_kv4_extend(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size, seqs,
                     new_tokens, n, slots, max_new, stream=None) -> int:
    t = _kv4_tables(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size)
    return load_library().mlaqp_kv4_extend(*t, _ptr(seqs), _ptr(new_tokens), int(n), _ptr(slots), int(max_new),
                                           _stream(stream))


def mlaqp_kv4_fork(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size, parents,
                   children, n, cache, page_stride, layer_stride, layers, workspace, workspace_bytes,
                   stream=None) -> int:
    t = _kv4_tables(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size)
    return load_library().mlaqp_kv4_fork(*t, _ptr(parents), _ptr(children), int(n), _ptr(cache), int(page_stride),
                                         int(layer_stride), int(layers), _ptr(workspace), int(workspace_bytes),
                                         _stream(stream))


def mlaqp_kv4_release(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size, seqs, n,
                      stream=None) -> int:
    t = _kv4_tables(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size)
    return load_library().mlaqp_kv4_release(*t, _ptr(seqs), int(n), _stream(stream))


def mlaqp_kv4_compact(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size, cache,
                      page_stride, layer_stride, layers, n_live, workspace, workspace_bytes, stream=None) -> int:
    t = _kv4_tables(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size)
    return load_library().mlaqp_kv4_compact(*t, _ptr(cache), int(page_stride), int(layer_stride), int(layers),
                                            _ptr(n_live), _ptr(workspace), int(workspace_bytes), _stream(stream))


def mlaqp_kv4_copy_pages(cache, page_stride, layer_stride, layers, num_pages, page_size, src, dst, n,
                         stream=None) -> int:
    return load_library().mlaqp_kv4_copy_pages(_ptr(cache), int(page_stride), int(layer_stride), int(layers),
                                               int(num_pages), int(page_size), _ptr(src), _ptr(dst), int(n),
                                               _stream(stream))


def mlaqp_kv4_pages_workspace(num_pages, n) -> int:
    """Bytes of workspace, or -1 (see ``mlaqp_last_error``)."""
    return load_library().mlaqp_kv4_pages_workspace(int(num_pages), int(n))


def mlaqp_kv4_prewarm(device=-1) -> int:
    return load_library().mlaqp_kv4_prewarm(int(device))


def mlaqp_device_status(reset=False):
    """Returns ``(status, word)``."""
    v = ctypes.c_uint(0)
    st = load_library().mlaqp_device_status(ctypes.byref(v), 1 if reset else 0)
    return st, v.value


def mlaqp_last_error() -> str:
    return load_library().mlaqp_last_error().decode()


def mlaqp_version() -> int:
    return load_library().mlaqp_version()


class MlaqpError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"mlaqp status {status}: {message}")
        self.status = status


def check(status: int) -> None:
    """Raise ``MlaqpError`` with the library's message for a non-OK status."""
    if status != MLAQP_OK:
        raise MlaqpError(status, mlaqp_last_error())
