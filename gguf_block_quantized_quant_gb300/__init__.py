"""Python binding of libqg: decode GEMV on raw GGUF blocks for GB300 (sm_103a).

Thin marshalling layer over the C ABI declared in ``include/qg.h``: every function here
has the name of the C entry point it calls, takes torch CUDA tensors, passes their device
pointers and the current CUDA stream, and raises ``QGError`` on a non-zero status.  All
arithmetic runs in the library's CUDA kernels; PyTorch only provides device memory and
streams.  If ``libqg.so`` has not been built, every call raises: there is no fallback.

Block formats (GGUF type ids): Q4_0=2, Q4_1=3, Q5_0=6, Q5_1=7, Q8_0=8, Q2_K=10, Q3_K=11,
Q4_K=12, Q5_K=13, Q6_K=14, IQ4_NL=20, IQ4_XS=23.
A weight matrix of N rows and K columns is passed as a uint8 CUDA tensor holding the N
rows of raw blocks back to back (``row_bytes(fmt, K)`` bytes per row).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import build as _build

Q4_0, Q4_1, Q5_0, Q5_1, Q8_0, Q4_K, Q5_K, Q6_K, IQ4_NL, IQ4_XS = 2, 3, 6, 7, 8, 12, 13, 14, 20, 23
Q2_K, Q3_K = 10, 11
FORMATS = {"Q4_0": Q4_0, "Q4_1": Q4_1, "Q5_0": Q5_0, "Q5_1": Q5_1, "Q8_0": Q8_0, "Q2_K": Q2_K, "Q3_K": Q3_K,
           "Q4_K": Q4_K, "Q5_K": Q5_K, "Q6_K": Q6_K, "IQ4_NL": IQ4_NL, "IQ4_XS": IQ4_XS}
BLOCK_ELEMS = {Q4_0: 32, Q4_1: 32, Q5_0: 32, Q5_1: 32, Q8_0: 32, Q2_K: 256, Q3_K: 256, Q4_K: 256, Q5_K: 256,
               Q6_K: 256, IQ4_NL: 32, IQ4_XS: 256}
BLOCK_BYTES = {Q4_0: 18, Q4_1: 20, Q5_0: 22, Q5_1: 24, Q8_0: 34, Q2_K: 84, Q3_K: 110, Q4_K: 144, Q5_K: 176,
               Q6_K: 210, IQ4_NL: 18, IQ4_XS: 136}

# element types (GGUF type ids) and frequency scalings of the decoder-layer operators
F32, F16, BF16 = 0, 1, 30
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = 0, 1, 2, 3

QG_OP_GEMV, QG_OP_GEMV_Q, QG_OP_MOE_FFN, QG_OP_FFN_SUBLAYER, QG_OP_MOE_FFN_S16, QG_OP_PREFILL = 1, 2, 3, 4, 5, 6
QG_OK, QG_EINVAL, QG_EWORKSPACE, QG_EALIGN, QG_ECUDA, QG_EDEVICE = 0, -1, -2, -3, -4, -5
WS_INVALID = ctypes.c_size_t(-1).value

LIB_PATH = _build.LIB

# every symbol declared in include/qg.h
EXPORTS = ("qg_quantize_act", "qg_gemv", "qg_gemv_q", "qg_moe_ffn", "qg_ffn_sublayer", "qg_workspace_size",
           "qg_moe_ws_layout", "qg_ffn_ws_layout", "qg_block_dots", "qg_device_error", "qg_strerror",
           "qg_version", "qg_gemv_static_ws", "qg_quantize_act_s16", "qg_moe_ffn_s16", "qg_moe_s16_ws_layout",
           "qg_prefill_gemm", "qg_dequant_f16", "qg_test_wait_expiry", "qg_norm_residual", "qg_rope_turns",
           "qg_rope_append", "qg_attn_paged", "qg_attn_workspace_size", "qg_rope_append_at", "qg_attn_shaped", "qg_attn_tree",
           "qg_tree_masks", "qg_cache_keep", "qg_logits_adjust")
QG_STATIC_WS_BYTES = 2097152  # include/qg.h


class QGError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what} failed: status {status} ({strerror(status)})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if libqg.so is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libqg.so not found at {LIB_PATH}; build it first "
                "(python -c 'import __graft_entry__ as g; g.build()'). There is no CPU fallback.")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.qg_quantize_act.argtypes = [P, I, I, P, P, P, P]
        L.qg_gemv.argtypes = [I, P, P, P, I, I, I, P, S, P]
        L.qg_gemv_q.argtypes = [I, P, P, P, P, P, I, I, I, P, S, P]
        L.qg_gemv_static_ws.argtypes = [I, P, P, P, I, I, I, P]
        L.qg_moe_ffn.argtypes = [I, P, I, I, P, I, I, P, P, P, P, P, P, I, P, P, P, P, S, P]
        L.qg_moe_ffn_s16.argtypes = [I, P, I, I, P, I, I, P, P, P, P, P, P, I, P, P, P, P, S, P]
        L.qg_quantize_act_s16.argtypes = [P, I, I, P, P, P, P]
        L.qg_moe_s16_ws_layout.argtypes = [I, I, I, I, I, ctypes.POINTER(S)]
        L.qg_ffn_sublayer.argtypes = [I, P, P, P, P, P, I, I, I, P, S, P]
        L.qg_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
        L.qg_workspace_size.restype = S
        L.qg_moe_ws_layout.argtypes = [I, I, I, I, I, ctypes.POINTER(S)]
        L.qg_ffn_ws_layout.argtypes = [I, I, I, I, ctypes.POINTER(S)]
        L.qg_block_dots.argtypes = [I, P, P, P, I, I, I, P, P, P]
        L.qg_prefill_gemm.argtypes = [I, P, P, P, I, I, I, P, S, P]
        L.qg_dequant_f16.argtypes = [I, P, I, I, P, P]
        L.qg_test_wait_expiry.argtypes = [ctypes.c_ulonglong, P]
        Q, F = ctypes.c_int64, ctypes.c_float
        L.qg_norm_residual.argtypes = [P, I, Q, P, I, Q, P, P, Q, P, F, F, F, P, P, I, I, I, P]
        L.qg_rope_turns.argtypes = [I] + [ctypes.c_double, I] + [ctypes.c_double] * 4 + [P, ctypes.POINTER(F)]
        L.qg_rope_append.argtypes = [P, Q, Q, P, Q, Q, P, Q, Q, I, I, I, P, I, I, F, P, P, F, P, ctypes.c_char_p, P]
        L.qg_attn_paged.argtypes = [P, Q, Q, I, I, I, I, F, I, P, I, P, ctypes.c_char_p, P, S, P]
        L.qg_rope_append_at.argtypes = [P, Q, Q, P, Q, Q, P, Q, Q, I, I, I, P, I, I, F, P, P, F, P, P, ctypes.c_char_p, P]
        L.qg_attn_shaped.argtypes = [P, Q, Q, I, I, I, I, F, I, F, P, P, P, P, I, P, ctypes.c_char_p, P, S, P]
        L.qg_attn_tree.argtypes = [P, Q, Q, I, I, I, I, F, I, F, P, P, I, P, P, I, P, ctypes.c_char_p, P, S, P]
        L.qg_tree_masks.argtypes = [P, P, P, I, I, P, I, P, P]
        L.qg_cache_keep.argtypes = [P, Q, P, I, I, Q, Q, P, ctypes.c_char_p, P]
        L.qg_logits_adjust.argtypes = [P, I, Q, P, I, Q, I, I, ctypes.c_char_p, P]
        L.qg_attn_workspace_size.argtypes = [I, I, I, I, I]
        L.qg_attn_workspace_size.restype = S
        L.qg_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        L.qg_strerror.argtypes = [I]
        L.qg_strerror.restype = ctypes.c_char_p
        L.qg_version.restype = I
        for name in EXPORTS:
            getattr(L, name)
        _lib = L
    return _lib


def strerror(status: int) -> str:
    try:
        return lib().qg_strerror(int(status)).decode()
    except RuntimeError:
        return "libqg not loaded"


def row_bytes(fmt: int, K: int) -> int:
    return (K // BLOCK_ELEMS[fmt]) * BLOCK_BYTES[fmt]


def _ptr(t, host_ok=True):
    """Device address of a tensor: a CUDA tensor, or (where the C API allows host memory:
    activations and outputs) a page-locked host tensor, which the kernels address directly."""
    if t is None:
        return None
    if not (t.is_cuda or (host_ok and t.is_pinned())):
        raise ValueError("libqg takes CUDA tensors" + (" or page-locked (pinned) host tensors" if host_ok else ""))
    if not t.is_contiguous():
        raise ValueError("libqg takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


def _dev(t):
    """The CUDA device of a call whose activations are t (the current device for host t)."""
    return t.device if t.is_cuda else torch.device("cuda", torch.cuda.current_device())


def _empty(shape, dtype, device, stream, seen):
    """Device memory of a call on `stream`, from that stream's pool: memory of the current stream's could
    be handed out again while the call still runs, or have readers there that are not done.  seen:
    an output, which the caller reads on the current stream."""
    if stream is None or stream == torch.cuda.current_stream(device):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if seen:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _out(shape, dtype, like, stream):
    """An output next to the activations: on their device, or page-locked host memory."""
    if like.is_cuda:
        return _empty(shape, dtype, like.device, stream, True)
    return torch.empty(shape, dtype=dtype, pin_memory=True)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, what: str):
    if rc != 0:
        raise QGError(rc, what)


def _ws(ws, size_query, like, stream):
    """The workspace and its byte count: the caller's (the C call checks its size), or a new
    one of qg_workspace_size bytes on the device of the activations `like` (size_query()
    and the device lookup run only then)."""
    if ws is not None:
        return ws, ws.numel()
    nbytes = size_query()
    if nbytes == WS_INVALID:
        raise QGError(QG_EINVAL, "qg_workspace_size")
    if nbytes > 0:
        ws = _empty(nbytes, torch.uint8, _dev(like), stream, False)
    return ws, (0 if ws is None else ws.numel())


# ----------------------------------------------------------------------------- entry points
def qg_workspace_size(op: int, fmt: int, M: int, N: int, K: int, E: int = 0, topk: int = 0, I: int = 0) -> int:
    return int(lib().qg_workspace_size(op, fmt, M, N, K, E, topk, I))


def qg_quantize_act(x, xq=None, xd=None, xs=None, stream=None):
    M, K = x.shape
    xq = _out((M, K), torch.int8, x, stream) if xq is None else xq
    xd = _out((M, K // 32), torch.float32, x, stream) if xd is None else xd
    xs = _out((M, K // 32), torch.int32, x, stream) if xs is None else xs
    _check(lib().qg_quantize_act(_ptr(x), M, K, _ptr(xq), _ptr(xd), _ptr(xs), _stream(stream)),
           "qg_quantize_act")
    return xq, xd, xs


def qg_quantize_act_s16(x, xq=None, xd=None, xs=None, stream=None):
    M, K = x.shape
    xq = _out((M, K), torch.int16, x, stream) if xq is None else xq
    xd = _out((M, K // 32), torch.float32, x, stream) if xd is None else xd
    xs = _out((M, K // 32), torch.int32, x, stream) if xs is None else xs
    _check(lib().qg_quantize_act_s16(_ptr(x), M, K, _ptr(xq), _ptr(xd), _ptr(xs), _stream(stream)),
           "qg_quantize_act_s16")
    return xq, xd, xs


def qg_gemv(fmt: int, W, x, N: int, y=None, ws=None, stream=None):
    M, K = x.shape
    y = _out((M, N), torch.float32, x, stream) if y is None else y
    ws, nws = _ws(ws, lambda: qg_workspace_size(QG_OP_GEMV, fmt, M, N, K), x, stream)
    _check(lib().qg_gemv(fmt, _ptr(W, False), _ptr(x), _ptr(y), N, K, M, _ptr(ws, False), nws, _stream(stream)), "qg_gemv")
    return y


def qg_gemv_static_ws(fmt: int, W, x, N: int, y=None, stream=None):
    """qg_gemv on the library's fixed device scratch, for callers that cannot allocate
    device memory where they call (a plugin inside a framework whose allocator owns the
    device memory, or a path that cannot afford cudaMalloc's synchronization).  Nothing is
    allocated inside the call when y is given.  Every call on a device shares the scratch:
    calls that may overlap on the GPU must be ordered on one stream.  The first call on a
    device looks up the scratch address and should come before any stream capture."""
    M, K = x.shape
    y = _out((M, N), torch.float32, x, stream) if y is None else y
    _check(lib().qg_gemv_static_ws(fmt, _ptr(W, False), _ptr(x), _ptr(y), N, K, M, _stream(stream)), "qg_gemv_static_ws")
    return y


def qg_gemv_q(fmt: int, W, xq, xd, xs, N: int, y=None, ws=None, stream=None):
    M, K = xq.shape
    y = _out((M, N), torch.float32, xq, stream) if y is None else y
    ws, nws = _ws(ws, lambda: qg_workspace_size(QG_OP_GEMV_Q, fmt, M, N, K), xq, stream)
    _check(lib().qg_gemv_q(fmt, _ptr(W, False), _ptr(xq), _ptr(xd), _ptr(xs), _ptr(y), N, K, M, _ptr(ws, False), nws,
                           _stream(stream)), "qg_gemv_q")
    return y


def qg_moe_ffn(fmt: int, x, Wr, topk: int, Wg_exps, Wu_exps, Wd_exps, Wg_sh, Wu_sh, Wd_sh, I: int,
               y=None, topk_ids=None, topk_w=None, ws=None, stream=None):
    M, H = x.shape
    E = Wr.shape[0]
    y = _out((M, H), torch.float32, x, stream) if y is None else y
    ws, nws = _ws(ws, lambda: qg_workspace_size(QG_OP_MOE_FFN, fmt, M, H, H, E, topk, I), x, stream)
    _check(lib().qg_moe_ffn(fmt, _ptr(x), M, H, _ptr(Wr, False), E, topk, _ptr(Wg_exps, False), _ptr(Wu_exps, False), _ptr(Wd_exps, False),
                            _ptr(Wg_sh, False), _ptr(Wu_sh, False), _ptr(Wd_sh, False), I, _ptr(y), _ptr(topk_ids), _ptr(topk_w),
                            _ptr(ws, False), nws, _stream(stream)), "qg_moe_ffn")
    return y


def qg_moe_ffn_s16(fmt: int, x, Wr, topk: int, Wg_exps, Wu_exps, Wd_exps, Wg_sh, Wu_sh, Wd_sh, I: int,
                   y=None, topk_ids=None, topk_w=None, ws=None, stream=None):
    M, H = x.shape
    E = Wr.shape[0]
    y = _out((M, H), torch.float32, x, stream) if y is None else y
    ws, nws = _ws(ws, lambda: qg_workspace_size(QG_OP_MOE_FFN_S16, fmt, M, H, H, E, topk, I), x, stream)
    _check(lib().qg_moe_ffn_s16(fmt, _ptr(x), M, H, _ptr(Wr, False), E, topk, _ptr(Wg_exps, False), _ptr(Wu_exps, False),
                                _ptr(Wd_exps, False), _ptr(Wg_sh, False), _ptr(Wu_sh, False), _ptr(Wd_sh, False), I, _ptr(y), _ptr(topk_ids),
                                _ptr(topk_w), _ptr(ws, False), nws, _stream(stream)), "qg_moe_ffn_s16")
    return y


def qg_ffn_sublayer(fmt: int, Wg, Wu, Wd, x, I: int, y=None, ws=None, stream=None):
    M, H = x.shape
    y = _out((M, H), torch.float32, x, stream) if y is None else y
    ws, nws = _ws(ws, lambda: qg_workspace_size(QG_OP_FFN_SUBLAYER, fmt, M, H, H, 0, 0, I), x, stream)
    _check(lib().qg_ffn_sublayer(fmt, _ptr(Wg, False), _ptr(Wu, False), _ptr(Wd, False), _ptr(x), _ptr(y), M, H, I, _ptr(ws, False), nws,
                                 _stream(stream)), "qg_ffn_sublayer")
    return y


def qg_moe_ws_layout(M: int, H: int, E: int, topk: int, I: int):
    off = (ctypes.c_size_t * 7)()
    _check(lib().qg_moe_ws_layout(M, H, E, topk, I, off), "qg_moe_ws_layout")
    return list(off)


def qg_moe_s16_ws_layout(M: int, H: int, E: int, topk: int, I: int):
    off = (ctypes.c_size_t * 7)()
    _check(lib().qg_moe_s16_ws_layout(M, H, E, topk, I, off), "qg_moe_s16_ws_layout")
    return list(off)


def qg_ffn_ws_layout(fmt: int, M: int, H: int, I: int):
    off = (ctypes.c_size_t * 3)()
    _check(lib().qg_ffn_ws_layout(fmt, M, H, I, off), "qg_ffn_ws_layout")
    return list(off)


def qg_block_dots(fmt: int, W, xq, xs, N: int, stream=None):
    M, K = xq.shape
    dots = _out((M, N, K // 32), torch.int32, xq, stream)
    aux = _out((M, N, K // 32), torch.int32, xq, stream)
    _check(lib().qg_block_dots(fmt, _ptr(W, False), _ptr(xq), _ptr(xs), N, K, M, _ptr(dots), _ptr(aux), _stream(stream)),
           "qg_block_dots")
    return dots, aux


def qg_prefill_gemm(fmt: int, W, x, N: int, y=None, ws=None, stream=None):
    """Prefill GEMM on the tensor cores: y = fp16(W) fp16(x)^T in fp32, for M >> 16 tokens."""
    M, K = x.shape
    y = _out((M, N), torch.float32, x, stream) if y is None else y
    ws, nws = _ws(ws, lambda: qg_workspace_size(QG_OP_PREFILL, fmt, M, N, K), x, stream)
    _check(lib().qg_prefill_gemm(fmt, _ptr(W, False), _ptr(x), _ptr(y), N, K, M, _ptr(ws, False), nws,
                                 _stream(stream)), "qg_prefill_gemm")
    return y


def qg_dequant_f16(fmt: int, W, N: int, K: int, stream=None):
    """Test hook: the fp16 weights (uint16 bit patterns, N x K) the prefill GEMM multiplies."""
    out = _empty((N, K), torch.int16, W.device, stream, True)
    _check(lib().qg_dequant_f16(fmt, _ptr(W, False), N, K, _ptr(out), _stream(stream)), "qg_dequant_f16")
    return out


# ------------------------------------------------------------- the rest of a decoder layer
# These calls are marshalled in C++ (csrc/qg_torch.cpp): through ctypes the host would take many
# times as long as the kernels of a single token.
_module = None


def _torch_module():
    global _module
    if _module is None:
        lib()
        built_for = _build.module_is_for()
        if built_for != _build._torch_id():
            raise RuntimeError(f"the module of the decoder-layer calls ({_build.TORCH_MODULE}) is " +
                               ("missing" if built_for is None else f"built for {built_for}, this is {_build._torch_id()}") +
                               "; build it (python -c 'import __graft_entry__ as g; g.build()'). There is no CPU fallback.")
        loader = importlib.machinery.ExtensionFileLoader("qg_torch", _build.TORCH_MODULE)
        spec = importlib.util.spec_from_file_location("qg_torch", _build.TORCH_MODULE, loader=loader)
        _module = importlib.util.module_from_spec(spec)
        loader.exec_module(_module)
    return _module


def _done(r, what):
    if type(r) is int:
        raise QGError(r, what)
    return r


def qg_norm_residual(y, res, w_pre, w_post=None, gate=None, alpha: float = 1.0, eps: float = 1e-6, w_offset: float = 0.0,
                     x_dtype=None, res_out=None, x_out=None, stream=None):
    """r = res + alpha * [gate *] [norm(y) * w_post] and x = norm(r) * w_pre, one pass.

    y: (rows, width), fp32, fp16 or bf16; res: the same shape, fp32 or y's type, or None;
    gate: y's type, (rows, width) or (width,); w_pre, w_post: fp32 (width,), w_pre None skips x.
    Returns (r, x); r has res's type (y's without res), x x_dtype (default y's)."""
    return _done((_module or _torch_module()).norm_residual(
        y, res, w_pre, w_post, gate, alpha, eps, w_offset, x_dtype, res_out, x_out, None if stream is None else stream.cuda_stream), "qg_norm_residual")


def qg_rope_turns(rot: int, base: float = 10000.0, scaling: int = ROPE_PLAIN, factor: float = 1.0, original: float = 4096.0,
                  beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(turns, amp): the phase increments (host int64 tensor of rot / 2; upload it once) and the
    factor that qg_rope_append takes."""
    turns = torch.empty(max(rot // 2, 1), dtype=torch.int64)
    amp = ctypes.c_float(1.0)
    _check(lib().qg_rope_turns(rot, base, scaling, factor, original, beta_fast, beta_slow, turns.data_ptr(), ctypes.byref(amp)),
           "qg_rope_turns")
    return turns, amp.value


def qg_rope_append(q, nk, nv, turns, k, v, q_start, kv_len, pages, kd=None, vd=None, pairs: bool = False, amp: float = 1.0,
                   wq=None, wk=None, eps: float = 1e-6, q_dtype=None, q_out=None, stream=None, positions=None):
    """Rotates the new tokens' q (tokens, heads, dim) and nk (tokens, kv_heads, dim) by their
    positions and appends nk and nv to the pools k, v (pages, kv_heads, page, dim); the steps of
    an int8 cache go to kd, vd.  turns: int64 CUDA tensor of rot / 2.  positions: int32 (tokens,), the
    rotary positions where they are not the slots (drafts of a tree).  Returns the rotated q,
    fp16 (bf16 beside a bf16 cache; q_dtype, if given, has to be that)."""
    return _done((_module or _torch_module()).rope_append(
        q, nk, nv, turns, k, v, q_start, kv_len, pages, kd, vd, pairs, amp, wq, wk, eps, q_dtype, q_out,
        None if stream is None else stream.cuda_stream, positions), "qg_rope_append")


def qg_attn_workspace_size(dim: int, q_heads: int, kv_heads: int, tokens: int, batch: int) -> int:
    return int(lib().qg_attn_workspace_size(dim, q_heads, kv_heads, tokens, batch))


def qg_attn_paged(q, k, v, q_start, kv_len, pages, kd=None, vd=None, max_new: int | None = None, scale: float | None = None,
                  window: int = 0, out_dtype=None, out=None, lse=None, ws=None, stream=None):
    """Causal attention of new tokens q (tokens, heads, dim) over the paged pools k, v
    (pages, kv_heads, page, dim).  max_new: the longest chunk, where the caller knows it (it
    only chooses the kernel; by default tokens that divide evenly over the sequences count as chunks of
    one length, else as one chunk among single tokens); scale: default dim ** -0.5; out_dtype:
    q's type or fp32; lse: optional fp32 (tokens, heads) output.  Returns out (tokens, heads, dim)."""
    return _done((_module or _torch_module()).attn_paged(
        q, k, v, q_start, kv_len, pages, kd, vd, max_new, scale, window, out_dtype, out, lse, ws,
        None if stream is None else stream.cuda_stream), "qg_attn_paged")


def qg_attn_shaped(q, k, v, q_start, kv_len, pages, kd=None, vd=None, cap: float = 0.0, slopes=None, prefix=None, first=None,
                   max_new: int | None = None, scale: float | None = None, window: int = 0, out_dtype=None, out=None, lse=None, ws=None,
                   stream=None):
    """qg_attn_paged with other scores and masks: scores capped at +-cap by cap * tanh(z / cap) (0: not),
    less slopes[head] * distance (fp32 (heads,)); the first prefix[b] slots (int32 (batch,)) seen by every
    token of sequence b, and no token seeing slots before its first[t] (int32 (tokens,)), the start of
    its document.  Returns out (tokens, heads, dim)."""
    return _done((_module or _torch_module()).attn_shaped(
        q, k, v, q_start, kv_len, pages, kd, vd, max_new, scale, window, out_dtype, out, lse, ws,
        None if stream is None else stream.cuda_stream, cap, slopes, prefix, first), "qg_attn_shaped")


def qg_attn_tree(q, k, v, q_start, kv_len, pages, tree, positions=None, kd=None, vd=None, cap: float = 0.0, slopes=None,
                 max_new: int | None = None, scale: float | None = None, window: int = 0, out_dtype=None, out=None, lse=None, ws=None,
                 stream=None):
    """Attention of trees of drafted tokens, which are the new tokens of their sequences: each sees the
    slots before the drafts and the drafts whose bits are set in its row of tree (int32 (tokens, words),
    bit i % 32 of word i // 32 for draft i of its sequence).  positions: int32 (tokens,), where they
    are not the slots (for window and slopes).  qg_tree_masks makes both.  Others as qg_attn_shaped."""
    return _done((_module or _torch_module()).attn_tree(
        q, k, v, q_start, kv_len, pages, kd, vd, max_new, scale, window, out_dtype, out, lse, ws,
        None if stream is None else stream.cuda_stream, tree, positions, cap, slopes), "qg_attn_tree")


def qg_tree_masks(parents, q_start, kv_len, words: int, tree=None, positions=None, stream=None):
    """(tree, positions) of drafted trees from parents (int32 (tokens,): the index among its sequence's
    drafts of the one that a draft follows, -1 for a root).  words: 32-bit words of a mask, for up to
    32 * words drafts of a sequence."""
    return _done((_module or _torch_module()).tree_masks(
        parents, q_start, kv_len, words, tree, positions, None if stream is None else stream.cuda_stream), "qg_tree_masks")


def qg_cache_keep(k, v, q_start, kv_len, pages, keep, keep_len, kd=None, vd=None, kv_out=None, stream=None):
    """Keeps the drafts keep[b, :keep_len[b]] (int32, rising indices among the sequence's drafts) of every
    sequence: their keys and values move together behind the slots before the drafts.  Pools may have a
    dimension of layers in front.  Returns the new lengths (kv_out, which may be kv_len itself)."""
    return _done((_module or _torch_module()).cache_keep(
        k, v, q_start, kv_len, pages, keep, keep_len, kd, vd, kv_out, None if stream is None else stream.cuda_stream), "qg_cache_keep")


def qg_logits_adjust(logits, out=None, out_dtype=None, seq=None, history=None, history_len=None, prompt_len=None, repetition=None,
                     frequency=None, presence=None, bias_start=None, bias_ids=None, bias=None, allow=None, drafts=None, tree=None,
                     q_start=None, stream=None):
    """Logits (rows, ids) with biases, penalties for ids said before and a grammar mask, before sampling.

    seq: int32 (rows,), the sequence of each row (default: row i is sequence i).  history: int32
    (sequences, longest), what each has said, history_len ids, the first prompt_len of them its prompt.
    repetition, frequency, presence: fp32 (sequences,).  bias_start (int32, sequences + 1) delimits each
    sequence's part of bias_ids and bias (of several entries for one id the last counts).  allow: int32
    (rows, words), bit v % 32 of word v // 32 set where id v is allowed; others become -inf.  drafts,
    tree, q_start: the row's own draft and those that it follows count as said (as in qg_attn_tree).
    Returns out (default fp32); out may be logits itself."""
    return _done((_module or _torch_module()).logits_adjust(
        logits, out, out_dtype, seq, history, history_len, prompt_len, repetition, frequency, presence, bias_start, bias_ids, bias, allow,
        drafts, tree, q_start, None if stream is None else stream.cuda_stream), "qg_logits_adjust")


def qg_test_wait_expiry(limit_ns: int, stream=None):
    """Test hook: a bounded wait that nothing satisfies gives up after limit_ns and sets the
    device error word (read it with qg_device_error)."""
    _check(lib().qg_test_wait_expiry(int(limit_ns), _stream(stream)), "qg_test_wait_expiry")


def qg_device_error() -> int:
    v = ctypes.c_uint(0)
    _check(lib().qg_device_error(ctypes.byref(v)), "qg_device_error")
    return int(v.value)


def qg_version() -> int:
    return int(lib().qg_version())
