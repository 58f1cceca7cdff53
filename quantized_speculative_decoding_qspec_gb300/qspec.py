"""Thin ctypes binding of libqspec.so: same names as the C ABI in include/qspec.h.

Every function only marshals arguments (torch tensors -> device pointers and sizes, the current
CUDA stream) and raises ``QSpecError`` on a non-OK status.  All computation happens in the CUDA
library; there is no fallback of any kind -- if the library is missing, loading fails loudly.
The sizes passed to the library come from the leading input's shape; every other tensor must hold
at least the elements the call reads or writes (ValueError otherwise, before any launch), since
the C ABI sees plain pointers and cannot check them itself.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqspec.so")

STATUS = {
    0: "QSPEC_OK",
    1: "QSPEC_ERR_INVALID_ARG",
    2: "QSPEC_ERR_UNSUPPORTED_SHAPE",
    3: "QSPEC_ERR_MISALIGNED",
    4: "QSPEC_ERR_WORKSPACE",
    5: "QSPEC_ERR_CUDA",
    6: "QSPEC_ERR_TIMEOUT",
}

# exported symbol -> (restype, argtypes)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_F64 = ctypes.c_double
_bf16, _int32, _f32 = torch.bfloat16, torch.int32, torch.float32
SIGNATURES = {
    "qspec_pack_weights": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P]),
    "qspec_linear_workspace_size": (ctypes.c_size_t, [_I64, _I64, _I64]),
    "qspec_linear_w4a16": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _P, _P, ctypes.c_size_t, _P]),
    "qspec_linear_w4a4": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "qspec_linear_w4a8": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "qspec_verify_workspace_size": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "qspec_verify_greedy": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "qspec_verify_sample": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P,
                                           ctypes.c_size_t, _P]),
    "qspec_verify_top1": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _P, _P, _P, ctypes.c_float, _P, _P,
                                         ctypes.c_size_t, _P]),
    "qspec_verify_greedy_noalloc": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _P, _P, _P]),
    "qspec_verify_tree_workspace_size": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "qspec_verify_tree_greedy": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "qspec_gather_rows": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _P, _P]),
    "qspec_select_tokens": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P]),
    "qspec_linear_group_workspace_size": (ctypes.c_size_t, [_I64, _P, _I32, _I64]),
    "qspec_linear_group": (ctypes.c_int, [_I32, _P, _I64, _I64, _P, _I32, _P, ctypes.c_size_t, _P]),
    "qspec_linear_pass_workspace_size": (ctypes.c_size_t, []),
    "qspec_linear_pass": (ctypes.c_int, [_I32, _I64, _P, _I32, _P, ctypes.c_size_t, _P]),
    "qspec_rotary_turns": (ctypes.c_int, [_I32, _F64, _I32, _F64, _F64, _F64, _F64, _P, _P]),
    "qspec_rotary": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _I32, _I32, _P, _I32, _P, _I64, _I64, _P]),
    "qspec_kv_append": (ctypes.c_int, [_P, _P, _P, _I64, _P, _I64, _P, _P, _P, _I64, _I32, _P, _I64, _P]),
    "qspec_kv_attention_workspace_size": (ctypes.c_size_t, []),
    "qspec_kv_attention": (ctypes.c_int, [_P, _P, _P, _I64, _I32, ctypes.c_float, _I32, _P, _P, _I64, _P, _P,
                                          ctypes.c_size_t, _P]),
    "qspec_logits_adjust": (ctypes.c_int, [_P, _I32, _I32, _I32, _P, _P, _I64, _P, _P, _P, _P, _P, _I32, _P, _P, _P]),
    "qspec_kv_attention_shared": (ctypes.c_int, [_P, _P, _P, _P, _I64, _I32, ctypes.c_float, _I32, _P, _P, _I64, _P, _P,
                                                 ctypes.c_size_t, _P]),
    "qspec_beam_workspace_size": (ctypes.c_size_t, [_I32, _I32, _I32, _I32]),
    "qspec_beam_select": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "qspec_kv_pages": (ctypes.c_int, [_P, _P, _I32, _I32, _P, _P, _P, _I32, _I32, _P, _I64, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "qspec_kv_copy_pages": (ctypes.c_int, [_P, _I32, _P, _P, _P, _I32, _P]),
    "qspec_kv_compact": (ctypes.c_int, [_P, _I32, _P, _P, _P, _I32, _I32, _P]),
    "qspec_check_status": (ctypes.c_int, [_P, _P]),
    "qspec_copy": (ctypes.c_int, [_P, _P, ctypes.c_size_t, _P]),
    "qspec_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}


class QSpecError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}")
        self.code = code


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libqspec.so (built by build.py / __graft_entry__.build()) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libqspec.so not found at {p}: build it first (python -m "
                           "quantized_speculative_decoding_qspec_gb300.build)")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:  # (the handle itself: a Stream object would cost more than the rest of a small call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(fn: str, code: int):
    if code != 0:
        raise QSpecError(fn, code)


def _dt(t, dtype, name):
    if t is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _need(t, n, name):
    """The library writes or reads n elements of t: refuse a smaller tensor before any launch."""
    if t is not None and t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs {n}")


def _arg32(x, name):
    """x as the 32-bit argument that it becomes (ctypes would cut it down silently)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} does not fit 32 bits: {x}")
    return x


def qspec_pack_weights(W, Wp, S, stream=None):
    """W bf16 [N, K] -> Wp uint8 [N, K/2], S fp16 [N, K/128] (outputs written in place)."""
    _dt(W, torch.bfloat16, "W"); _dt(Wp, torch.uint8, "Wp"); _dt(S, torch.float16, "S")
    N, K = W.shape
    _need(Wp, N * (K // 2), "Wp"); _need(S, N * (K // 128), "S")
    _check("qspec_pack_weights", load().qspec_pack_weights(_ptr(W), N, K, _ptr(Wp), _ptr(S), _stream(stream)))


def qspec_linear_workspace_size(M, N, K):
    """Workspace bytes for an [M, K] x [N, K] product on the current device."""
    return int(load().qspec_linear_workspace_size(M, N, K))


def new_linear_workspace(M, N, K, device="cuda"):
    """A zero-filled linear workspace (zero once; calls of this (M, N, K) keep it ready, other shapes
    need their own)."""
    n = qspec_linear_workspace_size(M, N, K)
    if n == 0:
        raise ValueError("invalid linear shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _need_linear(M, N, K, Wp, S, y, xq_out=None, xs_out=None, acc_out=None):
    _need(Wp, N * (K // 2), "Wp"); _need(S, N * (K // 128), "S"); _need(y, M * N, "y")
    _need(xq_out, M * K, "xq_out"); _need(xs_out, M, "xs_out"); _need(acc_out, M * N * (K // 128), "acc_out")


def qspec_linear_w4a16(x, Wp, S, y, ws, stream=None):
    """y bf16 [M, N] = x bf16 [M, K] . dequant(Wp, S)^T."""
    _dt(x, torch.bfloat16, "x"); _dt(Wp, torch.uint8, "Wp"); _dt(S, torch.float16, "S"); _dt(y, torch.bfloat16, "y")
    _dt(ws, torch.uint8, "ws")
    M, K = x.shape
    N = Wp.shape[0]
    _need_linear(M, N, K, Wp, S, y)
    _check("qspec_linear_w4a16",
           load().qspec_linear_w4a16(_ptr(x), _ptr(Wp), _ptr(S), M, N, K, _ptr(y), _ptr(ws), ws.numel(),
                                     _stream(stream)))


def qspec_linear_w4a4(x, Wp, S, y, ws, xq_out=None, xs_out=None, acc_out=None, stream=None):
    """Draft-mode linear with the per-token INT4 activation quantiser fused."""
    _dt(x, torch.bfloat16, "x"); _dt(Wp, torch.uint8, "Wp"); _dt(S, torch.float16, "S"); _dt(y, torch.bfloat16, "y")
    _dt(xq_out, torch.int8, "xq_out"); _dt(xs_out, torch.float32, "xs_out"); _dt(acc_out, torch.int32, "acc_out")
    _dt(ws, torch.uint8, "ws")
    M, K = x.shape
    N = Wp.shape[0]
    _need_linear(M, N, K, Wp, S, y, xq_out, xs_out, acc_out)
    _check("qspec_linear_w4a4",
           load().qspec_linear_w4a4(_ptr(x), _ptr(Wp), _ptr(S), M, N, K, _ptr(y), _ptr(xq_out), _ptr(xs_out),
                                    _ptr(acc_out), _ptr(ws), ws.numel(), _stream(stream)))


def qspec_linear_w4a8(x, Wp, S, y, ws, xq_out=None, xs_out=None, acc_out=None, stream=None):
    """The W4A8 configuration: qspec_linear_w4a4 with per-token INT8 activation codes."""
    _dt(x, torch.bfloat16, "x"); _dt(Wp, torch.uint8, "Wp"); _dt(S, torch.float16, "S"); _dt(y, torch.bfloat16, "y")
    _dt(xq_out, torch.int8, "xq_out"); _dt(xs_out, torch.float32, "xs_out"); _dt(acc_out, torch.int32, "acc_out")
    _dt(ws, torch.uint8, "ws")
    M, K = x.shape
    N = Wp.shape[0]
    _need_linear(M, N, K, Wp, S, y, xq_out, xs_out, acc_out)
    _check("qspec_linear_w4a8",
           load().qspec_linear_w4a8(_ptr(x), _ptr(Wp), _ptr(S), M, N, K, _ptr(y), _ptr(xq_out), _ptr(xs_out),
                                    _ptr(acc_out), _ptr(ws), ws.numel(), _stream(stream)))


class LinearPart(ctypes.Structure):
    """One part of qspec_linear_group (the C struct qspec_linear_part)."""
    _fields_ = [("Wp", ctypes.c_void_p), ("S", ctypes.c_void_p), ("y", ctypes.c_void_p), ("N", ctypes.c_int64)]


class LinearGroup:
    """Several linears that read the same activations, in one launch (qspec_linear_group).

    x: bf16 [M, K]; parts: list of (Wp, S, y) -- Wp uint8 [N, K/2], S fp16 [N, K/128], y bf16 [M, N].
    abits: 16 (W4A16), 4 (W4A4) or 8 (W4A8).  The tensors must stay alive while the group is used.
    """

    def __init__(self, abits, x, parts, ws):
        _dt(x, torch.bfloat16, "x"); _dt(ws, torch.uint8, "ws")
        if not parts:
            raise ValueError("a group needs at least one part")
        self.M, self.K = x.shape
        self.abits, self.x, self.ws = int(abits), x, ws
        self.arr = (LinearPart * len(parts))()
        self._keep = [x]
        for i, (Wp, S, y) in enumerate(parts):
            _dt(Wp, torch.uint8, "Wp"); _dt(S, torch.float16, "S"); _dt(y, torch.bfloat16, "y")
            N = Wp.shape[0]
            _need_linear(self.M, N, self.K, Wp, S, y)
            self.arr[i] = LinearPart(_ptr(Wp), _ptr(S), _ptr(y), N)
            self._keep += [Wp, S, y]

    def run(self, stream=None):
        _check("qspec_linear_group", load().qspec_linear_group(self.abits, _ptr(self.x), self.M, self.K, self.arr,
                                                               len(self.arr), _ptr(self.ws), self.ws.numel(),
                                                               _stream(stream)))


def qspec_linear_group_workspace_size(M, Ns, K):
    """Bytes of the workspace for a group of parts with N in Ns (0 if the arguments are invalid)."""
    arr = (LinearPart * len(Ns))()
    for i, N in enumerate(Ns):
        arr[i] = LinearPart(16, 16, 16, int(N))  # (only N is read; non-null, aligned placeholders)
    return int(load().qspec_linear_group_workspace_size(M, arr, len(Ns), K))


def new_linear_group_workspace(M, Ns, K, device="cuda"):
    """A zero-filled workspace for qspec_linear_group over parts with N in Ns."""
    n = qspec_linear_group_workspace_size(M, Ns, K)
    if n == 0:
        raise ValueError("invalid group shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def qspec_linear_group(abits, x, parts, ws, stream=None):
    """One launch over (Wp, S, y) parts that read the same x (see LinearGroup)."""
    LinearGroup(abits, x, parts, ws).run(stream)


class PassLayer(ctypes.Structure):
    """One layer of qspec_linear_pass (the C struct qspec_pass_layer)."""
    _fields_ = [("x", ctypes.c_void_p), ("Wp", ctypes.c_void_p), ("S", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("after", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def qspec_linear_pass_workspace_size():
    return int(load().qspec_linear_pass_workspace_size())


def new_pass_workspace(device="cuda"):
    """A zero-filled linear-pass workspace (zero once; passes keep it ready)."""
    return torch.zeros(qspec_linear_pass_workspace_size(), dtype=torch.uint8, device=device)


class LinearPass:
    """A pass of decode-size linears in one mode, described once and launched with run().

    layers: list of (x, Wp, S, y, after) -- x bf16 [M, K] (the same M for all), Wp uint8 [N, K/2],
    S fp16 [N, K/128], y bf16 [M, N], after: the layer reads outputs of earlier layers of the pass.
    abits: 16 (W4A16), 4 (W4A4) or 8 (W4A8).  The tensors must stay alive while the pass is used.
    """

    def __init__(self, abits, layers, ws):
        _dt(ws, torch.uint8, "ws")
        if not layers:
            raise ValueError("a pass needs at least one layer")
        self.M = layers[0][0].shape[0]
        self.abits = int(abits)
        self.ws = ws
        self.arr = (PassLayer * len(layers))()
        self._keep = []
        for i, (x, Wp, S, y, after) in enumerate(layers):
            _dt(x, torch.bfloat16, "x"); _dt(Wp, torch.uint8, "Wp"); _dt(S, torch.float16, "S")
            _dt(y, torch.bfloat16, "y")
            M, K = x.shape
            if M != self.M:
                raise ValueError("every layer of a pass has the same number of tokens")
            N = Wp.shape[0]
            _need_linear(M, N, K, Wp, S, y)
            self.arr[i] = PassLayer(_ptr(x), _ptr(Wp), _ptr(S), _ptr(y), N, K, 1 if after else 0, 0)
            self._keep += [x, Wp, S, y]

    def run(self, stream=None):
        _check("qspec_linear_pass", load().qspec_linear_pass(self.abits, self.M, self.arr, len(self.arr),
                                                             _ptr(self.ws), self.ws.numel(), _stream(stream)))


def qspec_linear_pass(abits, layers, ws, stream=None):
    """One launch over a list of (x, Wp, S, y, after) linears in one mode (see LinearPass)."""
    LinearPass(abits, layers, ws).run(stream)


def qspec_verify_workspace_size(B, gamma, V):
    return int(load().qspec_verify_workspace_size(B, gamma, V))


def _need_greedy(B, G1, draft_tok, accept_len, out_tok, tgt_argmax):
    _need(draft_tok, B * (G1 - 1), "draft_tok"); _need(accept_len, B, "accept_len")
    _need(out_tok, B * G1, "out_tok"); _need(tgt_argmax, B * G1, "tgt_argmax")


def qspec_verify_greedy(tgt_logits, draft_tok, accept_len, out_tok, ws, tgt_argmax=None, stream=None):
    """Greedy verify: tgt_logits bf16 [B, gamma+1, V], draft_tok int32 [B, gamma]."""
    _dt(tgt_logits, torch.bfloat16, "tgt_logits"); _dt(draft_tok, torch.int32, "draft_tok")
    _dt(accept_len, torch.int32, "accept_len"); _dt(out_tok, torch.int32, "out_tok")
    _dt(tgt_argmax, torch.int32, "tgt_argmax"); _dt(ws, torch.uint8, "ws")
    B, G1, V = tgt_logits.shape
    _need_greedy(B, G1, draft_tok, accept_len, out_tok, tgt_argmax)
    _check("qspec_verify_greedy",
           load().qspec_verify_greedy(_ptr(tgt_logits), _ptr(draft_tok), B, G1 - 1, V, _ptr(accept_len),
                                      _ptr(out_tok), _ptr(tgt_argmax), _ptr(ws), ws.numel(), _stream(stream)))


def qspec_verify_greedy_noalloc(tgt_logits, draft_tok, accept_len, out_tok, tgt_argmax=None, stream=None):
    """Greedy verify without a workspace (scratch inside the library; for callers that cannot allocate)."""
    _dt(tgt_logits, torch.bfloat16, "tgt_logits"); _dt(draft_tok, torch.int32, "draft_tok")
    _dt(accept_len, torch.int32, "accept_len"); _dt(out_tok, torch.int32, "out_tok")
    _dt(tgt_argmax, torch.int32, "tgt_argmax")
    B, G1, V = tgt_logits.shape
    _need_greedy(B, G1, draft_tok, accept_len, out_tok, tgt_argmax)
    _check("qspec_verify_greedy_noalloc",
           load().qspec_verify_greedy_noalloc(_ptr(tgt_logits), _ptr(draft_tok), B, G1 - 1, V, _ptr(accept_len),
                                              _ptr(out_tok), _ptr(tgt_argmax), _stream(stream)))


def qspec_verify_sample(tgt_logits, draft_logits, draft_tok, u_accept, u_resample, accept_len, out_tok, ws,
                        accept_prob=None, p_tok=None, q_tok=None, stream=None):
    """Sampling verify (min(1, p/q) test, residual / bonus resampling from the given uniforms)."""
    _dt(tgt_logits, torch.bfloat16, "tgt_logits"); _dt(draft_logits, torch.bfloat16, "draft_logits")
    _dt(draft_tok, torch.int32, "draft_tok"); _dt(u_accept, torch.float32, "u_accept")
    _dt(u_resample, torch.float32, "u_resample"); _dt(accept_len, torch.int32, "accept_len")
    _dt(out_tok, torch.int32, "out_tok"); _dt(ws, torch.uint8, "ws")
    for name, t in (("accept_prob", accept_prob), ("p_tok", p_tok), ("q_tok", q_tok)):
        _dt(t, torch.float32, name)
    B, G1, V = tgt_logits.shape
    g = G1 - 1
    _need(draft_logits, B * g * V, "draft_logits"); _need(draft_tok, B * g, "draft_tok")
    _need(u_accept, B * g, "u_accept"); _need(u_resample, B * G1, "u_resample")
    _need(accept_len, B, "accept_len"); _need(out_tok, B * G1, "out_tok")
    _need(accept_prob, B * g, "accept_prob"); _need(p_tok, B * g, "p_tok"); _need(q_tok, B * g, "q_tok")
    _check("qspec_verify_sample",
           load().qspec_verify_sample(_ptr(tgt_logits), _ptr(draft_logits), _ptr(draft_tok), _ptr(u_accept),
                                      _ptr(u_resample), B, G1 - 1, V, _ptr(accept_len), _ptr(out_tok),
                                      _ptr(accept_prob), _ptr(p_tok), _ptr(q_tok), _ptr(ws), ws.numel(),
                                      _stream(stream)))


def qspec_verify_top1(tgt_logits, draft_logits, tgt_top1, draft_top1, ws, tgt_p1=None, draft_p1=None,
                      high=0.8, tally=None, stream=None):
    """Each mode's top-1 token and top-1 probability at every draft position; optional running tally
    (fp64 [8], accumulated: positions, agree, both>high, agree there, both<=high, agree there, sums of p1)."""
    _dt(tgt_logits, torch.bfloat16, "tgt_logits"); _dt(draft_logits, torch.bfloat16, "draft_logits")
    _dt(tgt_top1, torch.int32, "tgt_top1"); _dt(draft_top1, torch.int32, "draft_top1")
    _dt(tgt_p1, torch.float32, "tgt_p1"); _dt(draft_p1, torch.float32, "draft_p1")
    _dt(tally, torch.float64, "tally"); _dt(ws, torch.uint8, "ws")
    if tally is not None and tally.numel() < 8:
        raise ValueError("tally needs 8 fp64 entries")
    B, G1, V = tgt_logits.shape
    g = G1 - 1
    _need(draft_logits, B * g * V, "draft_logits")
    _need(tgt_top1, B * g, "tgt_top1"); _need(draft_top1, B * g, "draft_top1")
    _need(tgt_p1, B * g, "tgt_p1"); _need(draft_p1, B * g, "draft_p1")
    _check("qspec_verify_top1",
           load().qspec_verify_top1(_ptr(tgt_logits), _ptr(draft_logits), B, G1 - 1, V, _ptr(tgt_top1),
                                    _ptr(draft_top1), _ptr(tgt_p1), _ptr(draft_p1), float(high), _ptr(tally),
                                    _ptr(ws), ws.numel(), _stream(stream)))


def qspec_gather_rows(src, idx, dst, stream=None):
    """dst[m] = src[idx[m]] over the leading dimension (rows of src.numel() / src.shape[0] elements)."""
    _dt(idx, torch.int32, "idx")
    if src.dtype != dst.dtype:
        raise TypeError("src and dst must have the same dtype")
    n_src, n = src.shape[0], idx.numel()
    row_bytes = src[0].numel() * src.element_size()
    if dst.shape[0] != n or dst[0].numel() * dst.element_size() != row_bytes:
        raise ValueError("dst must be [len(idx), row of src]")
    _check("qspec_gather_rows", load().qspec_gather_rows(_ptr(src), n_src, row_bytes, _ptr(idx), n, _ptr(dst),
                                                         _stream(stream)))


def qspec_select_tokens(logits, tok, u=None, stream=None):
    """Next token per row of bf16 logits [R, V]: argmax when u is None, else an inverse-CDF draw with u [R]."""
    _dt(logits, torch.bfloat16, "logits"); _dt(tok, torch.int32, "tok"); _dt(u, torch.float32, "u")
    R, V = logits.shape
    _need(tok, R, "tok"); _need(u, R, "u")
    _check("qspec_select_tokens", load().qspec_select_tokens(_ptr(logits), R, V, _ptr(u), _ptr(tok), _stream(stream)))


def qspec_verify_tree_workspace_size(B, T, V):
    return int(load().qspec_verify_tree_workspace_size(B, T, V))


def new_tree_workspace(B, T, V, device="cuda"):
    """A zero-filled tree-verify workspace (zero once; calls keep it ready)."""
    n = qspec_verify_tree_workspace_size(B, T, V)
    if n == 0:
        raise ValueError("invalid tree shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def qspec_verify_tree_greedy(tgt_logits, tree_tok, tree_parent, accept_len, out_tok, ws, accept_nodes=None,
                             stream=None):
    """Greedy verify of a candidate tree: tgt_logits bf16 [B, T+1, V], tree_tok / tree_parent int32 [B, T]."""
    _dt(tgt_logits, torch.bfloat16, "tgt_logits"); _dt(tree_tok, torch.int32, "tree_tok")
    _dt(tree_parent, torch.int32, "tree_parent"); _dt(accept_len, torch.int32, "accept_len")
    _dt(out_tok, torch.int32, "out_tok"); _dt(accept_nodes, torch.int32, "accept_nodes"); _dt(ws, torch.uint8, "ws")
    B, R, V = tgt_logits.shape
    T = R - 1
    _need(tree_tok, B * T, "tree_tok"); _need(tree_parent, B * T, "tree_parent")
    _need(accept_len, B, "accept_len"); _need(out_tok, B * R, "out_tok"); _need(accept_nodes, B * T, "accept_nodes")
    _check("qspec_verify_tree_greedy",
           load().qspec_verify_tree_greedy(_ptr(tgt_logits), _ptr(tree_tok), _ptr(tree_parent), B, R - 1, V,
                                           _ptr(accept_len), _ptr(out_tok), _ptr(accept_nodes), _ptr(ws),
                                           ws.numel(), _stream(stream)))


def _rows(t, heads, dim, name):
    """Pointer and token stride of a [T, heads, dim] GPU tensor whose tokens are contiguous rows."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [T, {heads}, {dim}], got {list(shape)}")
    strides = t.stride()
    if (dim > 1 and strides[2] != 1) or (heads > 1 and strides[1] != dim):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    return t.data_ptr(), strides[0] if shape[0] > 1 else heads * dim


class RotaryPlan(ctypes.Structure):
    """A rotary embedding on the device (the C struct qspec_rotary_plan)."""
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("mult", ctypes.c_float), ("reserved", ctypes.c_int32)]


ROTARY_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "yarn": 4}


def qspec_rotary_turns(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=4.0):
    """Frequencies of a rotary embedding: (int64 CPU tensor [rot/2] of 64-bit turn fractions, mult)."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALINGS)}")
    rot = _arg32(rot, "rot")
    turns = torch.empty(max(min(rot, 1024) // 2, 1), dtype=torch.int64)
    mult = ctypes.c_float()
    _check("qspec_rotary_turns", load().qspec_rotary_turns(rot, base, ROTARY_SCALINGS[scaling], factor, original, low,
                                                           high, turns.data_ptr(), ctypes.addressof(mult)))
    return turns, mult.value


class Rotary:
    """A rotary embedding, made once: frequencies on the device and the pair layout.

    rot: rotated values per head; interleaved: pairs (2i, 2i+1) instead of (i, i + rot/2); scaling:
    "none", "linear", "base", "bands" (original, low, high) or "yarn" (original, slow, fast).
    """

    def __init__(self, rot, base=10000.0, interleaved=False, scaling="none", factor=1.0, original=0.0, low=1.0,
                 high=4.0, slow=1.0, fast=32.0, device="cuda"):
        if scaling == "yarn":
            low, high = slow, fast
        turns, self.mult = qspec_rotary_turns(rot, base, scaling, factor, original, low, high)
        self.turns = turns.to(device)
        self.rot, self.interleaved = int(rot), bool(interleaved)
        self.plan = RotaryPlan(_ptr(self.turns), self.rot, int(self.interleaved), self.mult, 0)
        self.ref = ctypes.addressof(self.plan)


def qspec_rotary(x, pos, rotary, out, inverse=False, stream=None):
    """Rotate x bf16 [T, heads, dim] (any token and head strides) by pos int32 [T] into out (may be x)."""
    _dt(x, _bf16, "x"); _dt(out, _bf16, "out"); _dt(pos, _int32, "pos")
    shape = x.shape
    if len(shape) != 3 or out.shape != shape:
        raise ValueError("x and out must be [T, heads, dim]")
    T, H, D = shape
    xs, os_ = x.stride(), out.stride()
    if not (x.is_cuda and out.is_cuda):
        raise ValueError("tensor must live on the GPU")
    if D > 1 and (xs[2] != 1 or os_[2] != 1):
        raise ValueError("the values of a head of x and of out must be contiguous")
    _need(pos, T, "pos")
    xt, ot = (xs[0], os_[0]) if T > 1 else (0, 0)
    xh, oh = (xs[1], os_[1]) if H > 1 else (0, 0)
    _check("qspec_rotary", load().qspec_rotary(x.data_ptr(), xt, xh, _ptr(pos), T, H, D, rotary.ref, 1 if inverse else 0,
                                               out.data_ptr(), ot, oh, _stream(stream)))


class KVCacheDesc(ctypes.Structure):
    """The C struct qspec_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("heads", ctypes.c_int32), ("page", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class KVBatchDesc(ctypes.Structure):
    """The C struct qspec_kv_batch."""
    _fields_ = [("cu_tok", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("max_tok", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("T", ctypes.c_int64)]
    refs = None   # copies given to calls, by their T

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        self.__dict__["refs"] = {}   # what is written counts from the next call on


class KVCache:
    """A paged key/value cache: k, v uint8 [pages, heads, page, dim] of e4m3 codes, k_exp, v_exp int8 [pages, heads]."""

    def __init__(self, k, v, k_exp, v_exp):
        for name, t in (("k", k), ("v", v)):
            _dt(t, torch.uint8, name)
            if t.dim() != 4 or t.shape != k.shape:
                raise ValueError("k and v must be [pages, heads, page, dim]")
        _dt(k_exp, torch.int8, "k_exp"); _dt(v_exp, torch.int8, "v_exp")
        n, self.heads, self.page, self.dim = k.shape
        _need(k_exp, n * self.heads, "k_exp"); _need(v_exp, n * self.heads, "v_exp")
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.desc = KVCacheDesc(_ptr(k), _ptr(v), _ptr(k_exp), _ptr(v_exp), n, self.heads, self.page, self.dim, 0)
        self.ref = ctypes.addressof(self.desc)

    def values(self, which="k"):
        """The cached values as fp32 [pages, heads, page, dim] (a torch expression, for inspection)."""
        codes, exps = (self.k, self.k_exp) if which == "k" else (self.v, self.v_exp)
        return codes.view(torch.float8_e4m3fn).float() * torch.exp2(exps.float())[..., None, None]


def new_kv_cache(n_pages, heads, page, dim, device="cuda"):
    """An empty cache of n_pages pages."""
    def codes():
        return torch.zeros(n_pages, heads, page, dim, dtype=torch.uint8, device=device)

    def exps():
        return torch.zeros(n_pages, heads, dtype=torch.int8, device=device)
    return KVCache(codes(), codes(), exps(), exps())


class KVBatch:
    """The sequences of a step: cu_tok int32 [B+1], kv_len int32 [B], pages int32 [B, max_pages], max_tok.

    The tensors are read by the kernels: update them in place between steps (graph replays included).
    """

    def __init__(self, cu_tok, kv_len, pages, max_tok):
        _dt(cu_tok, torch.int32, "cu_tok"); _dt(kv_len, torch.int32, "kv_len"); _dt(pages, torch.int32, "pages")
        if pages.dim() != 2:
            raise ValueError("pages must be [B, max_pages]")
        B, max_pages = pages.shape
        _need(cu_tok, B + 1, "cu_tok"); _need(kv_len, B, "kv_len")
        self.cu_tok, self.kv_len, self.pages = cu_tok, kv_len, pages
        self.desc = KVBatchDesc(_ptr(cu_tok), _ptr(kv_len), _ptr(pages), B, max_pages, _arg32(max_tok, "max_tok"), 0, 0)

    def ref(self, T):
        """The descriptor for a step of T new tokens, to be passed to a call.  Each T has a copy of its own that stays as it
        is: threads may use one batch for steps of different sizes at once (ctypes lets go of the interpreter's lock
        while a call runs)."""
        refs = self.desc.refs
        ref = refs.get(T)
        if ref is None:
            desc = KVBatchDesc.from_buffer_copy(self.desc)
            desc.T = T
            if len(refs) >= 64:
                refs.clear()
            ref = refs[T] = ctypes.byref(desc)
        return ref


def qspec_kv_append(cache, batch, k, v, rotary=None, pos=None, q=None, q_out=None, stream=None):
    """Write the step's k and v (bf16 [T, heads, dim]) into the cache; rotate k and q [T, heads_q, dim] (into
    q_out, q itself when omitted) with a Rotary at pos int32 [T] (cache positions when omitted)."""
    _dt(k, _bf16, "k"); _dt(v, _bf16, "v"); _dt(q, _bf16, "q"); _dt(q_out, _bf16, "q_out"); _dt(pos, _int32, "pos")
    T = k.shape[0]
    if v.shape[0] != T or (q is not None and q.shape[0] != T):
        raise ValueError("k, v and q must have the same number of tokens")
    _need(pos, T, "pos")
    kp, ks = _rows(k, cache.heads, cache.dim, "k")
    vp, vs = _rows(v, cache.heads, cache.dim, "v")
    qp = qs = qop = qos = hq = 0
    if q is not None:
        q_out = q if q_out is None else q_out
        if q_out.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
        hq = q.shape[1]
        qp, qs = _rows(q, hq, cache.dim, "q")
        qop, qos = _rows(q_out, hq, cache.dim, "q_out")
    _check("qspec_kv_append",
           load().qspec_kv_append(cache.ref, batch.ref(T), kp, ks, vp, vs, rotary.ref if rotary is not None else None,
                                  _ptr(pos), qp or None, qs, hq, qop or None, qos, _stream(stream)))


def qspec_kv_attention_workspace_size():
    return int(load().qspec_kv_attention_workspace_size())


def new_kv_attention_workspace(device="cuda"):
    """A zero-filled attention workspace (zero once; it serves every shape, calls keep it ready)."""
    return torch.zeros(qspec_kv_attention_workspace_size(), dtype=torch.uint8, device=device)


def qspec_kv_attention(cache, batch, q, out, ws, scale=None, window=0, tree=None, lse=None, stream=None):
    """out = causal attention of q (bf16 [T, heads_q, dim]) over the cache; scale defaults to dim^-0.5, tree:
    int64 [T] words of visible new tokens, lse: fp32 [T, heads_q]."""
    _dt(q, _bf16, "q"); _dt(out, _bf16, "out"); _dt(tree, torch.int64, "tree"); _dt(lse, _f32, "lse")
    _dt(ws, torch.uint8, "ws")
    T, hq = q.shape[:2]
    if out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    _need(tree, T, "tree"); _need(lse, T * hq, "lse")
    qp, qs = _rows(q, hq, cache.dim, "q")
    op, os_ = _rows(out, hq, cache.dim, "out")
    window = int(window)
    if not 0 <= window < 2 ** 31:  # (one beyond every position hides none)
        window = _arg32(min(window, 2 ** 31 - 1), "window")
    _check("qspec_kv_attention",
           load().qspec_kv_attention(cache.ref, batch.ref(T), qp, qs, hq,
                                     cache.dim ** -0.5 if scale is None else float(scale), window, _ptr(tree), op, os_,
                                     _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


class KVPrefixesDesc(ctypes.Structure):
    """The C struct qspec_kv_prefixes."""
    _fields_ = [("cu_seq", ctypes.c_void_p), ("len", ctypes.c_void_p), ("n_groups", ctypes.c_int32), ("max_tok", ctypes.c_int32)]


class KVPrefixes:
    """Groups of a batch's sequences that share a prefix: cu_seq int32 [groups + 1], lengths int32 [groups], max_tok new tokens
    of a group at most.  The tensors are read by the kernels, as a KVBatch's are."""

    def __init__(self, cu_seq, lengths, max_tok):
        _dt(cu_seq, _int32, "cu_seq"); _dt(lengths, _int32, "lengths")
        n = lengths.numel()
        _need(cu_seq, n + 1, "cu_seq")
        self.cu_seq, self.lengths = cu_seq, lengths
        self.desc = KVPrefixesDesc(_ptr(cu_seq), _ptr(lengths), n, _arg32(max_tok, "max_tok"))
        self.ref = ctypes.addressof(self.desc)


def qspec_kv_attention_shared(cache, batch, prefixes, q, out, ws, scale=None, window=0, tree=None, lse=None, stream=None):
    """qspec_kv_attention where the sequences of each group of a KVPrefixes share their first positions, read once for all."""
    _dt(q, _bf16, "q"); _dt(out, _bf16, "out"); _dt(tree, torch.int64, "tree"); _dt(lse, _f32, "lse")
    _dt(ws, torch.uint8, "ws")
    T, hq = q.shape[:2]
    if out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    _need(tree, T, "tree"); _need(lse, T * hq, "lse")
    qp, qs = _rows(q, hq, cache.dim, "q")
    op, os_ = _rows(out, hq, cache.dim, "out")
    window = int(window)
    if not 0 <= window < 2 ** 31:  # (one beyond every position hides none)
        window = _arg32(min(window, 2 ** 31 - 1), "window")
    _check("qspec_kv_attention_shared",
           load().qspec_kv_attention_shared(cache.ref, batch.ref(T), prefixes.ref, qp, qs, hq,
                                            cache.dim ** -0.5 if scale is None else float(scale), window, _ptr(tree), op, os_,
                                            _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


def qspec_beam_workspace_size(B, beams, V, n):
    return int(load().qspec_beam_workspace_size(B, beams, V, n))


def new_beam_workspace(B, beams, V, n, device="cuda"):
    """A zero-filled beam-selection workspace (zero once; calls keep it ready, for this shape and smaller ones)."""
    size = qspec_beam_workspace_size(B, beams, V, n)
    if size == 0:
        raise ValueError("invalid beam shape")
    return torch.zeros(size, dtype=torch.uint8, device=device)


def qspec_beam_select(logits, scores, parent, tok, score, ws, done=None, end_tok=0, weights=None, stream=None):
    """The n best of each sequence's beams times tokens: logits bf16 [B, beams, V], scores fp32 [B, beams] (summed log probabilities)
    -> parent (row of logits), tok int32 [B, n], score fp32 [B, n].  done int32 [B, beams]: finished beams, which offer end_tok at
    their own score; weights fp32 [B, beams]: candidates compare by score times weight."""
    _dt(logits, _bf16, "logits"); _dt(scores, _f32, "scores"); _dt(parent, _int32, "parent"); _dt(tok, _int32, "tok")
    _dt(score, _f32, "score"); _dt(done, _int32, "done"); _dt(weights, _f32, "weights"); _dt(ws, torch.uint8, "ws")
    B, K, V = logits.shape
    if parent.dim() != 2 or parent.shape[0] != B:
        raise ValueError(f"parent must be [{B}, n]")
    n = parent.shape[1]
    _need(scores, B * K, "scores"); _need(done, B * K, "done"); _need(weights, B * K, "weights")
    _need(tok, B * n, "tok"); _need(score, B * n, "score")
    _check("qspec_beam_select",
           load().qspec_beam_select(_ptr(logits), _ptr(scores), _ptr(done), _arg32(end_tok, "end_tok"), _ptr(weights), B, K, V, n,
                                    _ptr(parent), _ptr(tok), _ptr(score), _ptr(ws), ws.numel(), _stream(stream)))


class KVLayers:
    """The caches of a model's layers, which share page tables: KVCaches of one shape."""

    def __init__(self, caches):
        self.caches = list(caches)
        if not self.caches:
            raise ValueError("at least one cache")
        self.arr = (KVCacheDesc * len(self.caches))(*[c.desc for c in self.caches])
        self.n, self.page, self.ref = len(self.caches), self.caches[0].page, ctypes.addressof(self.arr)


def _layers(caches):
    """(address, number, page) of the descriptors of a KVCache or KVLayers."""
    return (caches.ref, caches.n if isinstance(caches, KVLayers) else 1, caches.page)


def qspec_kv_pages(pages, room, keep, need, refs, page, new_pages, new_refs, copy_src, copy_dst, copy_len, left, parent=None,
                   stream=None):
    """The next step's page tables: new row r (of new_pages [R, W]) keeps keep[r] positions of row parent[r] (r when omitted) of
    pages and has room for need[r]; refs / new_refs [n_pages] count each page's holders (may be one tensor), and
    (copy_src, copy_dst, copy_len) [R] say what qspec_kv_copy_pages has to copy.  left [1]: free pages, or minus those that lack."""
    for name, t in (("pages", pages), ("room", room), ("keep", keep), ("need", need), ("refs", refs), ("new_pages", new_pages),
                    ("new_refs", new_refs), ("copy_src", copy_src), ("copy_dst", copy_dst), ("copy_len", copy_len),
                    ("left", left), ("parent", parent)):
        _dt(t, _int32, name)
    if pages.dim() != 2 or new_pages.dim() != 2:
        raise ValueError("pages and new_pages must be [rows, max_pages]")
    (B, W), (R, NW), n_pages = pages.shape, new_pages.shape, refs.numel()
    _need(room, B, "room"); _need(keep, R, "keep"); _need(need, R, "need"); _need(new_refs, n_pages, "new_refs"); _need(left, 1, "left")
    _need(copy_src, R, "copy_src"); _need(copy_dst, R, "copy_dst"); _need(copy_len, R, "copy_len"); _need(parent, R, "parent")
    _check("qspec_kv_pages",
           load().qspec_kv_pages(_ptr(pages) or None, _ptr(room) or None, B, W, _ptr(parent) or None, _ptr(keep) or None,
                                 _ptr(need) or None, R, NW, _ptr(refs), n_pages, _arg32(page, "page"), _ptr(new_pages) or None,
                                 _ptr(new_refs), _ptr(copy_src) or None, _ptr(copy_dst) or None, _ptr(copy_len) or None,
                                 _ptr(left), _stream(stream)))


def qspec_kv_copy_pages(caches, src, dst, lengths=None, stream=None):
    """Page src[i] -> dst[i] (int32; src < 0: none) in a KVCache or all of a KVLayers: scales and the first lengths[i] slots (all)."""
    _dt(src, _int32, "src"); _dt(dst, _int32, "dst"); _dt(lengths, _int32, "lengths")
    n = src.numel()
    _need(dst, n, "dst"); _need(lengths, n, "lengths")
    if n == 0:                     # (the last rows have ended: no pairs, no arrays)
        src = dst = lengths = None
    ref, layers, _ = _layers(caches)
    _check("qspec_kv_copy_pages", load().qspec_kv_copy_pages(ref, layers, _ptr(src), _ptr(dst), _ptr(lengths), n, _stream(stream)))


def qspec_kv_compact(caches, batch, nodes, count, first=1, stream=None):
    """The accepted nodes (int32 [B, T], count [B] of them) of the tree that the batch's append wrote, `first` tokens behind each
    sequence's first new one, move behind it: in a KVCache or all of a KVLayers."""
    _dt(nodes, _int32, "nodes"); _dt(count, _int32, "count")
    B, T = nodes.shape
    if B < batch.desc.B:
        raise ValueError(f"nodes must be [{batch.desc.B}, T]")
    _need(count, batch.desc.B, "count")
    ref, layers, _ = _layers(caches)
    tokens = batch.desc.max_tok * batch.desc.B  # (the call reads no tokens: an upper bound of their number)
    _check("qspec_kv_compact", load().qspec_kv_compact(ref, layers, batch.ref(tokens), _ptr(nodes), _ptr(count), T,
                                                       _arg32(first, "first"), _stream(stream)))


def qspec_logits_adjust(logits, out, draft_tok=None, hist=None, hist_len=None, prompt_len=None, penalties=None,
                        bias_ids=None, bias=None, mask=None, stream=None):
    """Penalties, biases and a grammar mask on logits bf16 [B, rows, V] into out (may be logits)."""
    _dt(logits, _bf16, "logits"); _dt(out, _bf16, "out"); _dt(draft_tok, _int32, "draft_tok"); _dt(hist, _int32, "hist")
    _dt(hist_len, _int32, "hist_len"); _dt(prompt_len, _int32, "prompt_len"); _dt(bias_ids, _int32, "bias_ids")
    _dt(mask, _int32, "mask"); _dt(penalties, _f32, "penalties"); _dt(bias, _f32, "bias")
    B, rows, V = logits.shape
    n_bias = bias_ids.shape[1] if bias_ids is not None else 0
    _need(out, B * rows * V, "out"); _need(draft_tok, B * (rows - 1), "draft_tok"); _need(hist_len, B, "hist_len")
    _need(prompt_len, B, "prompt_len"); _need(penalties, 3 * B, "penalties"); _need(bias_ids, B * n_bias, "bias_ids")
    _need(bias, B * n_bias, "bias"); _need(mask, B * rows * ((V + 31) // 32), "mask")
    if hist is not None and (hist.dim() != 2 or hist.shape[0] < B):
        raise ValueError("hist must be [B, length]")
    _check("qspec_logits_adjust",
           load().qspec_logits_adjust(_ptr(logits), B, rows, V, _ptr(draft_tok), _ptr(hist),
                                      hist.shape[1] if hist is not None else 0, _ptr(hist_len), _ptr(prompt_len),
                                      _ptr(penalties), _ptr(bias_ids), _ptr(bias), n_bias, _ptr(mask), _ptr(out),
                                      _stream(stream)))


def _ptr_any(t, name):
    """Pointer of a contiguous device tensor or pinned host tensor (qspec_copy's operands)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda and not t.is_pinned():
        raise ValueError(f"{name} must live on the GPU or in pinned host memory")
    return t.data_ptr()


def qspec_copy(dst, src, stream=None):
    """Copy src into dst (same number of bytes, device or pinned host tensors) with one kernel."""
    nb = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nb:
        raise ValueError(f"dst holds {dst.numel() * dst.element_size()} bytes, src {nb}")
    _check("qspec_copy", load().qspec_copy(_ptr_any(dst, "dst"), _ptr_any(src, "src"), nb, _stream(stream)))


def qspec_check_status(ws=None, stream=None):
    """Synchronise the stream and raise on device-side errors (timeouts, invalid draft tokens)."""
    _check("qspec_check_status", load().qspec_check_status(_ptr(ws), _stream(stream)))


def qspec_status_string(code: int) -> str:
    return load().qspec_status_string(int(code)).decode()


def new_verify_workspace(B, gamma, V, device="cuda"):
    """A zero-filled verify workspace of the required size (zero once; calls keep it ready)."""
    n = qspec_verify_workspace_size(B, gamma, V)
    if n == 0:
        raise ValueError("invalid verify shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)
