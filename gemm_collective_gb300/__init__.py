"""Python binding of libfcc (fused GEMM + collective on one GB300).

A thin ctypes layer over the C ABI declared in ``include/fcc.h``: every
function has the C name and argument order, and only marshals arguments
(lists of device pointers or CUDA tensors, a stream, an options struct).
All computation runs in the library's CUDA kernels.  Importing this module
loads ``libfcc.so``; if the library has not been built the import fails
loudly -- there is no fallback path.

Pointer-array arguments accept a sequence of ``int`` device addresses or of
objects with ``data_ptr()`` (torch tensors), or an array made once by
``ptr_array()``.  ``stream`` accepts ``None``
(the legacy default stream), an ``int`` handle or an object with a
``cuda_stream`` attribute (``torch.cuda.Stream``).
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfcc.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libfcc.so is not built ({LIB_PATH}); run gemm_collective_gb300/build.py "
        "or __graft_entry__.build() first")

_lib = ctypes.CDLL(LIB_PATH)

# ----------------------------------------------------------------- constants
FCC_BF16, FCC_F16, FCC_F32, FCC_E4M3 = range(4)
(FCC_OK, FCC_ERR_INVALID, FCC_ERR_UNSUPPORTED, FCC_ERR_CUDA, FCC_ERR_CAPACITY,
 FCC_ERR_TIMEOUT, FCC_ERR_WORKSPACE) = range(7)
(FCC_ALGO_AUTO, FCC_ALGO_FUSED, FCC_ALGO_UNFUSED, FCC_ALGO_INTERDECOM,
 FCC_ALGO_CE) = range(5)
FCC_OP_GEMM_RS, FCC_OP_GEMM_AR, FCC_OP_GEMV_AR, FCC_OP_AG_GEMM, FCC_OP_EMBEDDING_A2A = range(5)
FCC_MAX_RANKS = 8
FCC_MAX_EXPERTS = 64
FCC_MAX_TEACHER = 256


class fcc_opts(ctypes.Structure):
    _fields_ = [
        ("algo", ctypes.c_int),
        ("deterministic", ctypes.c_int),
        ("chunks", ctypes.c_int),
        ("max_ctas", ctypes.c_int),
        ("timeout_ns", ctypes.c_int64),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("cta_pair", ctypes.c_int),
        ("phase_ns", ctypes.c_void_p),
    ]


def make_opts(algo=FCC_ALGO_AUTO, deterministic=1, chunks=0, max_ctas=0, timeout_ns=0,
              workspace=None, workspace_bytes=0, cta_pair=0, phase_ns=None) -> fcc_opts:
    ws = workspace.data_ptr() if hasattr(workspace, "data_ptr") else workspace
    ph = phase_ns.data_ptr() if hasattr(phase_ns, "data_ptr") else phase_ns
    return fcc_opts(algo, deterministic, chunks, max_ctas, timeout_ns, ws, workspace_bytes,
                    cta_pair, ph)


class fcc_cache(ctypes.Structure):
    _fields_ = [
        ("K", ctypes.c_void_p),
        ("V", ctypes.c_void_p),
        ("K_exp", ctypes.c_void_p),
        ("V_exp", ctypes.c_void_p),
        ("pages", ctypes.c_int64),
        ("page_size", ctypes.c_int),
        ("H", ctypes.c_int),
        ("d", ctypes.c_int),
        ("dtype", ctypes.c_int),
    ]


class fcc_batch(ctypes.Structure):
    _fields_ = [
        ("start", ctypes.c_void_p),
        ("len", ctypes.c_void_p),
        ("table", ctypes.c_void_p),
        ("max_pages", ctypes.c_int64),
        ("T", ctypes.c_int64),
        ("B", ctypes.c_int),
    ]


def make_cache(K, V, pages, page_size, H, d, dtype=FCC_BF16, K_exp=None, V_exp=None) -> fcc_cache:
    """The description of a paged cache: one pool of keys and one of values for each rank.

    Made once and passed to every call; like ptr_array() it holds addresses only,
    and the tensors must stay alive while it is in use."""
    arrays = [None if x is None else ptr_array(x) for x in (K, V, K_exp, V_exp)]
    c = fcc_cache(*(None if a is None else ctypes.addressof(a) for a in arrays), pages, page_size,
                  H, d, dtype)
    c.arrays = arrays  # (the structure holds their addresses)
    used = arrays if dtype == FCC_E4M3 else arrays[:2]  # (the powers' arrays are ignored otherwise)
    c.ranks = min((len(a) for a in used if a is not None), default=0)
    return c


def _int32s(x, rows, width, what):
    # a tensor of another type, or with fewer or other places than the kernels read, would be misread without a word
    if hasattr(x, "data_ptr"):
        if str(x.dtype) != "torch.int32":
            raise FccError(FCC_ERR_INVALID, f"{what} holds {x.dtype}, not int32")
        dims = x.dim()
        if not (dims == 1 or dims == 2 and x.size(1) == width) or x.numel() < rows * width or not (
                x.is_contiguous() or dims == 2 and rows == 1 and x.stride(1) == 1):
            raise FccError(FCC_ERR_INVALID, f"{what} is not {rows} x {width} int32 values one after another")


def make_batch(start, len, table, T, B, max_pages) -> fcc_batch:
    """The description of a step's sequences (int32 arrays on the device): see fcc_batch in fcc.h.

    Tensors are checked for their type and size; addresses are taken as they are."""
    _int32s(start, 1, B + 1, "start")
    _int32s(len, 1, B, "len")
    _int32s(table, B, max_pages, "table")
    return fcc_batch(_addr(start), _addr(len), _addr(table), max_pages, T, B)


class FccError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fcc_status_string(status)} ({status})")


_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_OPTS = ctypes.POINTER(fcc_opts)


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_gemm_rs = _sig("fcc_gemm_rs", _I, [_I, _P, _P, _P, _I64, _I64, _I64, _I, _I, _OPTS, _P])
_gemm_ar = _sig("fcc_gemm_ar", _I, [_I, _P, _P, _P, _I64, _I64, _I64, _I, _I, _OPTS, _P])
_gemv_ar = _sig("fcc_gemv_ar", _I, [_I, _P, _P, _P, _I64, _I64, _I64, _I, _I, _OPTS, _P])
_gemv_ar_static = _sig("fcc_gemv_ar_static", _I,
                       [_I, _P, _P, _P, _I64, _I64, _I64, _I, _I, _OPTS, _P])
_ag_gemm = _sig("fcc_ag_gemm", _I, [_I, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _OPTS, _P])
_moe = _sig("fcc_moe_dispatch_gemm", _I,
            [_I, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P, _P, _I64, _P, _P, _P, _P, _P, _I, _I,
             _OPTS, _P])
_combine = _sig("fcc_moe_combine", _I,
                [_I, _P, _I64, _I64, _I64, _I, _I, _P, _P, _P, _P, _P, _I, _I, _OPTS, _P])
_combine_ws = _sig("fcc_moe_combine_workspace_size", ctypes.c_size_t, [_I, _I64, _I])
_emb = _sig("fcc_embedding_a2a", _I,
            [_I, _I, _P, _I64, _I64, _I64, _P, _P, _P, _I, _I, _OPTS, _P])
_emb_ws = _sig("fcc_embedding_workspace_size", ctypes.c_size_t,
               [_I, _I, _I64, _I64, _I, _OPTS])
_ws = _sig("fcc_workspace_size", ctypes.c_size_t, [_I, _I, _I64, _I64, _I64, _OPTS])
_moe_ws = _sig("fcc_moe_workspace_size", ctypes.c_size_t,
               [_I, _I64, _I64, _I64, _I, _I, _I64, _OPTS])
_stream_status = _sig("fcc_stream_status", _I, [_P])
_status_string = _sig("fcc_status_string", ctypes.c_char_p, [_I])
_chunks = _sig("fcc_interdecom_chunks", _I, [ctypes.c_double, ctypes.c_double,
                                              ctypes.c_double, _I])
_itime = _sig("fcc_interdecom_time", ctypes.c_double, [ctypes.c_double, ctypes.c_double,
                                                       ctypes.c_double, _I])
_choose = _sig("fcc_choose_algo", _I, [_I, _I, _I64, _I64, _I64, _I, _I])
_attn = _sig("fcc_ring_attention", _I,
             [_I, _P, _P, _P, _P, _I64, _I, _I64, _I, _I, _I, _OPTS, _P])
_F = ctypes.c_float
_xent = _sig("fcc_linear_xent", _I,
             [_I, _P, _P, _P, _I64, _I64, _I64, _P, _P, ctypes.c_int32, _F, _F, _F, _I, _OPTS, _P])
_xent_grad = _sig("fcc_linear_xent_grad", _I,
                  [_I, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P, ctypes.c_int32, _F, _F, _F,
                   _I, _I, _OPTS, _P])
_distill = _sig("fcc_linear_distill", _I,
                [_I, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _F, _F, _I, _OPTS, _P])
_distill_grad = _sig("fcc_linear_distill_grad", _I,
                     [_I, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _F, _F, _I, _I,
                      _OPTS, _P])
_loss_ws = _sig("fcc_linear_loss_workspace_size", ctypes.c_size_t,
                [_I, _I64, _I64, _I64, _I, _I, _OPTS])
_CACHE, _BATCH = ctypes.POINTER(fcc_cache), ctypes.POINTER(fcc_batch)
_append = _sig("fcc_cache_append", _I, [_I, _P, _P, _I64, _CACHE, _BATCH, _I, _OPTS, _P])
_gather = _sig("fcc_cache_gather", _I, [_I, _CACHE, _BATCH, _P, _P, _I64, _I, _OPTS, _P])
_paged = _sig("fcc_paged_attention", _I,
              [_I, _P, _I64, _CACHE, _BATCH, _I, _P, _I64, _P, _F, _I64, _I, _I, _OPTS, _P])
_paged_ws = _sig("fcc_paged_attention_workspace_size", ctypes.c_size_t,
                 [_I, _I64, _I, _I, _I, _I64, _OPTS])
_launches = _sig("fcc_launch_count", ctypes.c_uint64, [])
_version = _sig("fcc_version", ctypes.c_char_p, [])
_wait_timeout = _sig("fcc_test_wait_timeout", _I, [_I64, _P])
_suspended_wait_timeout = _sig("fcc_test_suspended_wait_timeout", _I, [_I64, _P])
_grouped_wait_timeout = _sig("fcc_test_grouped_wait_timeout", _I, [_I64, _P])
_ksplit_wait_timeout = _sig("fcc_test_ksplit_wait_timeout", _I, [_I64, _P])


# ---------------------------------------------------------------- marshalling
def _addr(x) -> int:
    if x is None:
        return 0
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    return int(x)


_PACK = [struct.Struct(f"{n}P").pack for n in range(FCC_MAX_EXPERTS + 1)]  # by length


def _ptrs(seq):
    if seq is None:
        return None
    if isinstance(seq, ctypes.Array):  # built once by ptr_array()
        return seq
    if not isinstance(seq, (list, tuple)):
        seq = list(seq)  # (an iterator can be walked only once)
    try:
        vals = [x.data_ptr() for x in seq]
    except AttributeError:
        vals = [_addr(x) for x in seq]
    n = len(vals)
    # (a bytes object passes as the address of its contents, at half the cost of
    # building a ctypes array)
    return _PACK[n](*vals) if n < len(_PACK) else struct.pack(f"{n}P", *vals)


def ptr_array(seq):
    """The C array of device pointers for a sequence of tensors (or addresses).

    Every call accepts it wherever it takes a pointer array; a loop that calls
    an operator on the same buffers again and again can build its arrays once
    instead of marshalling the tensors on every call.  It holds addresses
    only: the tensors must stay alive (and in place) while it is in use."""
    vals = [_addr(x) for x in seq]
    return (ctypes.c_void_p * len(vals))(*vals)


def _stream(s) -> int:
    if s is None:
        return 0
    try:
        return s.cuda_stream
    except AttributeError:
        return int(s)


def _opts(o):
    return ctypes.byref(o) if o is not None else None


def _check(st: int, where: str):
    if st != FCC_OK:
        raise FccError(st, where)


# ------------------------------------------------------------------ the calls
def fcc_gemm_rs(R, A, B, out_shard, M, N, K, in_dtype=FCC_BF16, out_dtype=FCC_BF16, opts=None,
                stream=None):
    _check(_gemm_rs(R, _ptrs(A), _ptrs(B), _ptrs(out_shard), M, N, K, in_dtype, out_dtype,
                    _opts(opts), _stream(stream)), "fcc_gemm_rs")


def fcc_gemm_ar(R, A, B, out, M, N, K, in_dtype=FCC_BF16, out_dtype=FCC_BF16, opts=None,
                stream=None):
    _check(_gemm_ar(R, _ptrs(A), _ptrs(B), _ptrs(out), M, N, K, in_dtype, out_dtype,
                    _opts(opts), _stream(stream)), "fcc_gemm_ar")


def fcc_gemv_ar(R, A, B, out, M, N, K, in_dtype=FCC_BF16, out_dtype=FCC_F32, opts=None,
                stream=None):
    _check(_gemv_ar(R, _ptrs(A), _ptrs(B), _ptrs(out), M, N, K, in_dtype, out_dtype,
                    _opts(opts), _stream(stream)), "fcc_gemv_ar")


def fcc_gemv_ar_static(R, A, B, out, M, N, K, in_dtype=FCC_BF16, out_dtype=FCC_F32, opts=None,
                       stream=None):
    """fcc_gemv_ar with its scratch in the library's static device array (no allocation)."""
    _check(_gemv_ar_static(R, _ptrs(A), _ptrs(B), _ptrs(out), M, N, K, in_dtype, out_dtype,
                           _opts(opts), _stream(stream)), "fcc_gemv_ar_static")


def fcc_ag_gemm(R, X_shard, B, out, gathered, M, N, K, in_dtype=FCC_BF16, out_dtype=FCC_BF16,
                opts=None, stream=None):
    _check(_ag_gemm(R, _ptrs(X_shard), _ptrs(B), _ptrs(out), _ptrs(gathered), M, N, K,
                    in_dtype, out_dtype, _opts(opts), _stream(stream)), "fcc_ag_gemm")


def fcc_moe_dispatch_gemm(R, X, logits, W, T, H, F, E, topk, recv_x, recv_y, cap, topk_idx,
                          topk_gate, expert_counts, send_counts, recv_src, in_dtype=FCC_BF16,
                          out_dtype=FCC_BF16, opts=None, stream=None):
    _check(_moe(R, _ptrs(X), _ptrs(logits), _ptrs(W), T, H, F, E, topk, _ptrs(recv_x),
                _ptrs(recv_y), cap, _ptrs(topk_idx), _ptrs(topk_gate), _addr(expert_counts),
                _addr(send_counts), _ptrs(recv_src), in_dtype, out_dtype, _opts(opts),
                _stream(stream)), "fcc_moe_dispatch_gemm")


def fcc_moe_combine(R, recv_y, cap, T, F, E, topk, topk_idx, topk_gate, recv_src,
                    expert_counts, y, in_dtype=FCC_BF16, out_dtype=FCC_BF16, opts=None,
                    stream=None):
    _check(_combine(R, _ptrs(recv_y), cap, T, F, E, topk, _ptrs(topk_idx), _ptrs(topk_gate),
                    _ptrs(recv_src), _addr(expert_counts), _ptrs(y), in_dtype, out_dtype,
                    _opts(opts), _stream(stream)), "fcc_moe_combine")


def fcc_moe_combine_workspace_size(R, T, topk) -> int:
    return int(_combine_ws(R, T, topk))


def fcc_embedding_a2a(R, ntables, tables, V, D, Bl, offsets, indices, out,
                      in_dtype=FCC_BF16, out_dtype=FCC_BF16, opts=None, stream=None):
    _check(_emb(R, ntables, _ptrs(tables), V, D, Bl, _ptrs(offsets), _ptrs(indices),
                _ptrs(out), in_dtype, out_dtype, _opts(opts), _stream(stream)),
           "fcc_embedding_a2a")


def fcc_embedding_workspace_size(R, ntables, D, Bl, out_dtype=FCC_BF16, opts=None) -> int:
    return int(_emb_ws(R, ntables, D, Bl, out_dtype, _opts(opts)))


def fcc_ring_attention(R, Q, K, V, O, S, H, d, causal=False, in_dtype=FCC_BF16,
                       out_dtype=FCC_BF16, opts=None, stream=None):
    _check(_attn(R, _ptrs(Q), _ptrs(K), _ptrs(V), _ptrs(O), S, H, d, 1 if causal else 0,
                 in_dtype, out_dtype, _opts(opts), _stream(stream)), "fcc_ring_attention")


def fcc_linear_xent(R, X, W, labels, T, V, D, loss, lse, ignore_index=-100, smoothing=0.0,
                    z_weight=0.0, softcap=0.0, in_dtype=FCC_BF16, opts=None, stream=None):
    """Cross entropy of a head split by vocabulary over R ranks; labels: [T] int32 on the device."""
    _check(_xent(R, _ptrs(X), _ptrs(W), _addr(labels), T, V, D, _ptrs(loss), _ptrs(lse),
                 ignore_index, smoothing, z_weight, softcap, in_dtype, _opts(opts),
                 _stream(stream)), "fcc_linear_xent")


def fcc_linear_xent_grad(R, X, W, labels, lse, dloss, T, V, D, dX, dW, ignore_index=-100,
                         smoothing=0.0, z_weight=0.0, softcap=0.0, in_dtype=FCC_BF16,
                         out_dtype=FCC_BF16, opts=None, stream=None):
    """Its gradient with respect to X and W (dX or dW None: not wanted); lse from the forward."""
    _check(_xent_grad(R, _ptrs(X), _ptrs(W), _addr(labels), _ptrs(lse), _addr(dloss), T, V, D,
                      _ptrs(dX), _ptrs(dW), ignore_index, smoothing, z_weight, softcap, in_dtype,
                      out_dtype, _opts(opts), _stream(stream)), "fcc_linear_xent_grad")


def fcc_linear_distill(R, X, W, teacher_idx, teacher_logits, T, V, D, topk, loss, lse,
                       temperature=1.0, softcap=0.0, in_dtype=FCC_BF16, opts=None, stream=None):
    """Distillation from a teacher's top logits ([T, topk] int32 and f32 on the device)."""
    _check(_distill(R, _ptrs(X), _ptrs(W), _addr(teacher_idx), _addr(teacher_logits), T, V, D,
                    topk, _ptrs(loss), _ptrs(lse), temperature, softcap, in_dtype, _opts(opts),
                    _stream(stream)), "fcc_linear_distill")


def fcc_linear_distill_grad(R, X, W, teacher_idx, teacher_logits, lse, dloss, T, V, D, topk, dX,
                            dW, temperature=1.0, softcap=0.0, in_dtype=FCC_BF16,
                            out_dtype=FCC_BF16, opts=None, stream=None):
    """Its gradient with respect to X and W (dX or dW None: not wanted); lse from the forward."""
    _check(_distill_grad(R, _ptrs(X), _ptrs(W), _addr(teacher_idx), _addr(teacher_logits),
                         _ptrs(lse), _addr(dloss), T, V, D, topk, _ptrs(dX), _ptrs(dW),
                         temperature, softcap, in_dtype, out_dtype, _opts(opts),
                         _stream(stream)), "fcc_linear_distill_grad")


def fcc_linear_loss_workspace_size(R, T, V, D, topk=0, grad=False, opts=None) -> int:
    return int(_loss_ws(R, T, V, D, topk, 1 if grad else 0, _opts(opts)))


def _cache(c, R):
    # a cache described for fewer ranks would be read past its arrays' end
    if c is not None and hasattr(c, "ranks") and c.ranks < R:
        raise FccError(FCC_ERR_INVALID, f"a cache of {c.ranks} ranks in a call for {R}")
    return c


def fcc_cache_append(R, K, V, cache, batch, ld=0, in_dtype=FCC_BF16, opts=None, stream=None):
    """Writes a step's keys and values ([T, H, d] per rank) into the paged cache."""
    _check(_append(R, _ptrs(K), _ptrs(V), ld, _cache(cache, R), batch, in_dtype, _opts(opts),
                   _stream(stream)), "fcc_cache_append")


def fcc_cache_gather(R, cache, batch, K, V, ld=0, out_dtype=FCC_BF16, opts=None, stream=None):
    """Reads a step's positions back out of the cache into K, V ([T, H, d] per rank)."""
    _check(_gather(R, _cache(cache, R), batch, _ptrs(K), _ptrs(V), ld, out_dtype, _opts(opts),
                   _stream(stream)), "fcc_cache_gather")


def fcc_paged_attention(R, Q, cache, batch, Hq, O, lse=None, scale=0.0, window=0, ldq=0, ldo=0,
                        in_dtype=FCC_BF16, out_dtype=FCC_BF16, opts=None, stream=None):
    """Attention of a step's rows (Q: [T, Hq, d] per rank) over the cache's pages."""
    _check(_paged(R, _ptrs(Q), ldq, _cache(cache, R), batch, Hq, _ptrs(O), ldo, _ptrs(lse), scale,
                  window, in_dtype, out_dtype, _opts(opts), _stream(stream)),
           "fcc_paged_attention")


def fcc_paged_attention_workspace_size(R, T, B, Hq, H, d, opts=None) -> int:
    return int(_paged_ws(R, T, B, Hq, H, d, _opts(opts)))


def fcc_choose_algo(op, R, M, N, K, sms=0, max_ctas=0) -> int:
    """The algorithm FCC_ALGO_AUTO runs for this operator and shape."""
    return int(_choose(op, R, M, N, K, sms, max_ctas))


def fcc_workspace_size(op, R, M, N, K, opts=None) -> int:
    return int(_ws(op, R, M, N, K, _opts(opts)))


def fcc_moe_workspace_size(R, T, H, F, E, topk, cap, opts=None) -> int:
    return int(_moe_ws(R, T, H, F, E, topk, cap, _opts(opts)))


def fcc_stream_status(stream=None) -> int:
    """Synchronise the stream; return (and clear) the device status word."""
    return int(_stream_status(_stream(stream)))


def fcc_status_string(status: int) -> str:
    return _status_string(status).decode()


def fcc_interdecom_chunks(G: float, X: float, alpha: float, max_chunks: int) -> int:
    return int(_chunks(G, X, alpha, max_chunks))


def fcc_interdecom_time(G: float, X: float, alpha: float, chunks: int) -> float:
    return float(_itime(G, X, alpha, chunks))


def fcc_launch_count() -> int:
    return int(_launches())


def fcc_version() -> str:
    return _version().decode()


def fcc_test_wait_timeout(timeout_ns: int, stream=None):
    _check(_wait_timeout(timeout_ns, _stream(stream)), "fcc_test_wait_timeout")


def fcc_test_suspended_wait_timeout(timeout_ns: int, stream=None):
    _check(_suspended_wait_timeout(timeout_ns, _stream(stream)), "fcc_test_suspended_wait_timeout")


def fcc_test_grouped_wait_timeout(timeout_ns: int, stream=None):
    _check(_grouped_wait_timeout(timeout_ns, _stream(stream)), "fcc_test_grouped_wait_timeout")


def fcc_test_ksplit_wait_timeout(timeout_ns: int, stream=None):
    _check(_ksplit_wait_timeout(timeout_ns, _stream(stream)), "fcc_test_ksplit_wait_timeout")


def raw_status(fn_name: str, *args) -> int:
    """Call a C entry point with already-marshalled ctypes arguments; return its status."""
    return int(getattr(_lib, fn_name)(*args))
