"""ctypes binding of libdiffattn_v2.so: the same entry points as include/diffattn_v2.h.

Argument marshalling only: every step of the operator runs in the CUDA library. The
wrappers take torch CUDA tensors, check dtype/shape/contiguity, pass data pointers and the
current (or given) stream, and raise on a non-OK status. Output tensors and the decode
workspace are allocated with torch when the caller does not pass them.

There is no CPU fallback: if the library is missing, importing fails with an error that
says how to build it; if only the binding's native half is, the calls that go through it (with
sinks, rotary positions, cache pages) fail with one.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import build

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdiffattn_v2.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE = 0, -1, -2, -3, -4

_vp, _i, _f, _sz, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
_ip = ctypes.POINTER(ctypes.c_int)

_SIGNATURES = {
    "diffattn_v2_version": (_i, []),
    "diffattn_v2_status_string": (ctypes.c_char_p, [_i]),
    "diffattn_v2_prefill": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "diffattn_v2_prefill_f32": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "diffattn_v2_prefill_window": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "diffattn_v2_prefill_varlen": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]),
    "diffattn_v2_prefill_train": (_i, [_vp] * 7 + [_i] * 6 + [_vp]),
    "diffattn_v2_backward_workspace_size": (_sz, [_i, _i, _i]),
    "diffattn_v2_backward": (_i, [_vp] * 11 + [_i] * 6 + [_vp, _sz, _vp]),
    "diffattn_v2_prefill_window_train": (_i, [_vp] * 7 + [_i] * 6 + [_vp]),
    "diffattn_v2_backward_window": (_i, [_vp] * 11 + [_i] * 6 + [_vp, _sz, _vp]),
    "diffattn_v2_prefill_varlen_train": (_i, [_vp] * 8 + [_i] * 7 + [_vp]),
    "diffattn_v2_backward_varlen_workspace_size": (_sz, [_i, _i, _i]),
    "diffattn_v2_backward_varlen": (_i, [_vp] * 12 + [_i] * 7 + [_vp, _sz, _vp]),
    "diffattn_v2_prefill_varlen_window_train": (_i, [_vp] * 8 + [_i] * 7 + [_vp]),
    "diffattn_v2_backward_varlen_window": (_i, [_vp] * 12 + [_i] * 7 + [_vp, _sz, _vp]),
    "diffattn_v2_decode_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "diffattn_v2_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "diffattn_v2_decode_window": (_i, [_vp] * 6 + [_i] * 6 + [_vp, _sz, _vp]),
    "diffattn_v2_decode_f32": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "diffattn_v2_decode_paged": (_i, [_vp] * 7 + [_i] * 7 + [_vp, _sz, _vp]),
    "diffattn_v2_decode_paged_window": (_i, [_vp] * 7 + [_i] * 8 + [_vp, _sz, _vp]),
    "diffattn_v2_decode_multi_workspace_size": (_sz, [_i] * 6),
    "diffattn_v2_decode_multi": (_i, [_vp] * 6 + [_i] * 6 + [_vp, _sz, _vp]),
    "diffattn_v2_lambda_v1": (_i, [_vp, _vp, _vp, _vp, _f, _i, _i, _i, _vp, _vp]),
    "diffattn_v2_lambda_v2": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp]),
    "diffattn_v2_prefill_fused_lambda": (_i, [_vp] * 8 + [_i] * 7 + [_vp]),
    "diffattn_v2_prefill_varlen_window": (_i, [_vp] * 6 + [_i] * 7 + [_vp]),
    "diffattn_v2_prefill_window_sink": (_i, [_vp] * 5 + [_i] * 7 + [_vp]),
    "diffattn_v2_prefill_varlen_window_sink": (_i, [_vp] * 6 + [_i] * 8 + [_vp]),
    "diffattn_v2_prefill_window_sink_train": (_i, [_vp] * 7 + [_i] * 7 + [_vp]),
    "diffattn_v2_prefill_varlen_window_sink_train": (_i, [_vp] * 8 + [_i] * 8 + [_vp]),
    "diffattn_v2_backward_window_sink_workspace_size": (_sz, [_i] * 6),
    "diffattn_v2_backward_window_sink": (_i, [_vp] * 11 + [_i] * 7 + [_vp, _sz, _vp]),
    "diffattn_v2_backward_varlen_window_sink_workspace_size": (_sz, [_i] * 7),
    "diffattn_v2_backward_varlen_window_sink": (_i, [_vp] * 12 + [_i] * 8 + [_vp, _sz, _vp]),
    "diffattn_v2_decode_window_sink": (_i, [_vp] * 6 + [_i] * 7 + [_vp]),
    "diffattn_v2_decode_paged_window_sink": (_i, [_vp] * 7 + [_i] * 9 + [_vp]),
    "diffattn_v2_rope": (_i, [_vp] * 6 + [_ip] + [_i] * 5 + [_i64] * 4 + [_i] * 3 + [_vp]),
    "diffattn_v2_rope_append_paged": (_i, [_vp] * 6 + [_ip, _i] + [_vp] * 5 + [_i] * 8 + [_i64] * 4 + [_i] * 2 + [_vp]),
    "diffattn_v2_cache_extend": (_i, [_vp] * 5 + [_i] * 4 + [_vp]),
    "diffattn_v2_cache_fork": (_i, [_vp] * 7 + [_i] * 5 + [_vp]),
    "diffattn_v2_cache_trim": (_i, [_vp] * 4 + [_i] * 6 + [_vp]),
    "diffattn_v2_cache_free": (_i, [_vp] * 5 + [_i] * 4 + [_vp]),
    "diffattn_v2_cache_compact": (_i, [_vp] * 6 + [_i] * 3 + [_vp]),
    "diffattn_v2_cache_copy_pages": (_i, [_vp] * 3 + [_i] * 2 + [_sz, _vp]),
    "diffattn_v2_device_error": (_i, [ctypes.POINTER(_i), _vp]),
    "diffattn_v2_decode_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
}
EXPORTED = tuple(_SIGNATURES)


def load(path=LIB_PATH):
    """Load a build of the library (the default, or e.g. its bounds-checking twin
    libdiffattn_v2_debug.so) with the entry points' argument and result types set. The
    wrappers below call the module's LIB."""
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing; build it with `python -m differential_attention_v2_b200.build` "
            "(nvcc, sm_100a). There is no fallback implementation.")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    # addresses of the entry points that are called through the native half
    lib.addresses = {name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _SIGNATURES}
    return lib


LIB = load()


class DiffAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {LIB.diffattn_v2_status_string(status).decode()} ({status})")


def _check(status: int, what: str):
    if status != OK:
        raise DiffAttnError(status, what)


def _load_native():
    """(the native half of the binding, "") or (None, why there is none): the calls that go through it
    raise then, the others work."""
    if not os.path.exists(build.NATIVE_PATH):
        return None, f"{build.NATIVE_PATH} is missing"
    if build.native_built_for() not in ("", build.native_stamp()):
        return None, f"{build.NATIVE_PATH} was built for {build.native_built_for()}, this is {build.native_stamp()}"
    spec = importlib.util.spec_from_file_location(__package__ + "._native", build.NATIVE_PATH)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        return None, str(e)
    module.on_error(_check)
    return module, ""


_native, _why_not_native = _load_native()


def _no_native(*_):
    raise ImportError(f"{_why_not_native}; build it with `python -m differential_attention_v2_b200.build`. "
                      "There is no fallback implementation.")


_invoke = _native.invoke if _native else _no_native


def _check_description(name, description):
    """The native half passes every C argument as a word, whatever the prototype says: the description has
    to name as many as the prototype has, pointers where it has pointers."""
    arguments, words = description.split("=>")[0].split("->")
    tensors = {a.lstrip(">@").split(":")[0].split("(")[0] for a in arguments.split() if ":" in a or a[0] == "@"}
    got = ["pointer" if w in tensors or w == "%" else "integer" for w in words.split()] + ["pointer"]  # the stream
    want = ["pointer" if t in (_vp, _ip) else "integer" for t in _SIGNATURES[name][1]]
    sizes = [a.count(",") + 1 for a in arguments.split() if a[0] == "@"]
    if got != want or any(n != len(_SIGNATURES[name + "_workspace_size"][1]) for n in sizes):
        raise TypeError(f"{name}: the description passes {got}, the prototype takes {want}")


def _entry(name, description):
    """An entry point of short calls: the native half checks its tensors, allocates the outputs that
    are not given and calls it on their device and the given or current stream, as described (see
    csrc/binding.cpp for the notation)."""
    _check_description(name, description)
    return _native.define(name, description) if _native else None


def _stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _torch_stream(stream, device):
    """A given stream as a torch stream."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)


def _empty(stream, shape, dtype, device):
    """An output or workspace of a call on `stream` (None: the current one), from that stream's memory
    pool: a block of the current stream's pool may still be in use by work queued there, which the
    given stream does not wait for. It is recorded on the current stream, where the caller reads it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    if t.numel():
        t.record_stream(caller)
    return t


def _empty_like(stream, t):
    return _empty(stream, t.shape, dtype=t.dtype, device=t.device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, ndim):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def version() -> int:
    return LIB.diffattn_v2_version()


def _window_of_sink(window, causal):
    if window is None or not causal:
        raise ValueError("sink needs a causal window")
    return int(window)


def prefill(q, k, v, lam, out=None, causal=True, stream=None):
    """bf16 prefill: q [B,S,Hq,D], k/v [B,S,Hkv,D], lam fp32 [B,S,Hq/2] -> out bf16 [B,S,Hq/2,D]."""
    for t, n, nd in ((q, "q", 4), (k, "k", 4), (v, "v", 4)):
        _need(t, n, torch.bfloat16, nd)
    _need(lam, "lam", torch.float32, 3)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    if out is None:
        out = _empty(stream, (B, S, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 4)
    st = LIB.diffattn_v2_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out), B, S, Hq, Hkv, D,
                                 1 if causal else 0, _stream(stream, q.device))
    _check(st, "diffattn_v2_prefill")
    return out


def prefill_window(q, k, v, lam, window, out=None, stream=None, sink=None):
    """bf16 causal prefill where query i sees only keys i-window+1 .. i, and with `sink` the
    first `sink` keys too."""
    if sink is not None:
        return _invoke(_PREFILL_SINK, LIB.addresses["diffattn_v2_prefill_window_sink"], q, k, v, lam, window, sink, out,
                       stream)
    for t, n, nd in ((q, "q", 4), (k, "k", 4), (v, "v", 4)):
        _need(t, n, torch.bfloat16, nd)
    _need(lam, "lam", torch.float32, 3)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    if out is None:
        out = _empty(stream, (B, S, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 4)
    st = LIB.diffattn_v2_prefill_window(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out), B, S, Hq, Hkv, D,
                                        int(window), _stream(stream, q.device))
    _check(st, "diffattn_v2_prefill_window")
    return out


def prefill_varlen(q, k, v, lam, cu_seqlens, max_seqlen, out=None, causal=True, stream=None):
    """bf16 prefill of packed sequences: q [T,Hq,D], k/v [T,Hkv,D], lam fp32 [T,Hq/2],
    cu_seqlens int32 [B+1] on the device; max_seqlen >= the longest sequence."""
    for t, n, nd in ((q, "q", 3), (k, "k", 3), (v, "v", 3)):
        _need(t, n, torch.bfloat16, nd)
    _need(lam, "lam", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    if out is None:
        out = _empty(stream, (T, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 3)
    st = LIB.diffattn_v2_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out), _ptr(cu_seqlens), B,
                                        int(max_seqlen), T, Hq, Hkv, D, 1 if causal else 0, _stream(stream, q.device))
    _check(st, "diffattn_v2_prefill_varlen")
    return out


def prefill_varlen_window(q, k, v, lam, cu_seqlens, max_seqlen, window, out=None, stream=None, sink=None):
    """Causal sliding-window prefill of packed sequences (layouts of prefill_varlen): query i
    of a sequence sees that sequence's keys i-window+1 .. i, and with `sink` its first `sink`
    keys too."""
    if sink is not None:
        return _invoke(_PREFILL_VARLEN_SINK, LIB.addresses["diffattn_v2_prefill_varlen_window_sink"], q, k, v, lam,
                       cu_seqlens, max_seqlen, window, sink, out, stream)
    for t, n, nd in ((q, "q", 3), (k, "k", 3), (v, "v", 3)):
        _need(t, n, torch.bfloat16, nd)
    _need(lam, "lam", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    if out is None:
        out = _empty(stream, (T, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 3)
    st = LIB.diffattn_v2_prefill_varlen_window(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out), _ptr(cu_seqlens), B,
                                               int(max_seqlen), T, Hq, Hkv, D, int(window), _stream(stream, q.device))
    _check(st, "diffattn_v2_prefill_varlen_window")
    return out


def prefill_f32(q, k, v, lam, out=None, causal=True, stream=None):
    """fp32 prefill on CUDA cores; same layout as prefill with fp32 tensors."""
    for t, n, nd in ((q, "q", 4), (k, "k", 4), (v, "v", 4), (lam, "lam", 3)):
        _need(t, n, torch.float32, nd)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    if out is None:
        out = _empty(stream, (B, S, Hq // 2, D), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, 4)
    st = LIB.diffattn_v2_prefill_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out), B, S, Hq, Hkv, D,
                                     1 if causal else 0, _stream(stream, q.device))
    _check(st, "diffattn_v2_prefill_f32")
    return out


def prefill_train(q, k, v, lam, out=None, o_branch=None, lse=None, causal=True, window=None, stream=None, sink=None):
    """Training forward: prefill plus the per-head normalised O_b (bf16 [B,S,Hq,D]) and the
    log2-domain row log-sum-exp (fp32 [B,S,Hq]) that backward reads. Returns (out, o_branch, lse).
    With `window` the causal sliding-window prefill (query i sees keys i-window+1 .. i); with
    `sink` besides, the first `sink` keys stay visible and o_branch is fp32."""
    if sink is not None:
        return _invoke(_TRAIN_SINK, LIB.addresses["diffattn_v2_prefill_window_sink_train"], q, k, v, lam,
                       _window_of_sink(window, causal), sink, out, o_branch, lse, stream)
    for t, n, nd in ((q, "q", 4), (k, "k", 4), (v, "v", 4)):
        _need(t, n, torch.bfloat16, nd)
    _need(lam, "lam", torch.float32, 3)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    if out is None:
        out = _empty(stream, (B, S, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    if o_branch is None:
        o_branch = _empty(stream, (B, S, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = _empty(stream, (B, S, Hq), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.bfloat16, 4)
    _need(o_branch, "o_branch", torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    if window is not None:
        st = LIB.diffattn_v2_prefill_window_train(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out), _ptr(o_branch),
                                                  _ptr(lse), B, S, Hq, Hkv, D, int(window), _stream(stream, q.device))
        _check(st, "diffattn_v2_prefill_window_train")
        return out, o_branch, lse
    st = LIB.diffattn_v2_prefill_train(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out), _ptr(o_branch), _ptr(lse),
                                       B, S, Hq, Hkv, D, 1 if causal else 0, _stream(stream, q.device))
    _check(st, "diffattn_v2_prefill_train")
    return out, o_branch, lse


def backward_workspace_size(B, S, Hq) -> int:
    return int(LIB.diffattn_v2_backward_workspace_size(B, S, Hq))


def backward(q, k, v, lam, o_branch, lse, dout, causal=True, dq=None, dk=None, dv=None, dlam=None,
             workspace=None, window=None, stream=None, sink=None):
    """Gradients of the bf16 prefill: returns (dq, dk, dv, dlam) with the layouts of q, k, v, lam.
    With `window` the gradients of the causal sliding-window prefill, with `sink` besides those
    of the window with sinks (o_branch fp32)."""
    if sink is not None:
        return _invoke(_BACKWARD_SINK, LIB.addresses["diffattn_v2_backward_window_sink"], q, k, v, lam, o_branch, lse, dout,
                       _window_of_sink(window, causal), sink, dq, dk, dv, dlam,
                       LIB.addresses["diffattn_v2_backward_window_sink_workspace_size"], workspace, stream)
    for t, n, nd in ((q, "q", 4), (k, "k", 4), (v, "v", 4), (o_branch, "o_branch", 4), (dout, "dout", 4)):
        _need(t, n, torch.bfloat16, nd)
    _need(lam, "lam", torch.float32, 3)
    _need(lse, "lse", torch.float32, 3)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    dq = _empty_like(stream, q) if dq is None else dq
    dk = _empty_like(stream, k) if dk is None else dk
    dv = _empty_like(stream, v) if dv is None else dv
    dlam = _empty_like(stream, lam) if dlam is None else dlam
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, n, torch.bfloat16, 4)
    _need(dlam, "dlam", torch.float32, 3)
    ws_bytes = backward_workspace_size(B, S, Hq)
    if workspace is None:
        workspace = _empty(stream, max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    if window is not None:
        st = LIB.diffattn_v2_backward_window(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(o_branch), _ptr(lse),
                                             _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlam), B, S, Hq, Hkv, D,
                                             int(window), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                             _stream(stream, q.device))
        _check(st, "diffattn_v2_backward_window")
        return dq, dk, dv, dlam
    st = LIB.diffattn_v2_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(o_branch), _ptr(lse), _ptr(dout),
                                  _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlam), B, S, Hq, Hkv, D, 1 if causal else 0,
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream, q.device))
    _check(st, "diffattn_v2_backward")
    return dq, dk, dv, dlam


def prefill_varlen_train(q, k, v, lam, cu_seqlens, max_seqlen, out=None, o_branch=None, lse=None, causal=True,
                         stream=None, window=None, sink=None):
    """Training forward of packed sequences (layouts of prefill_varlen): returns
    (out [T,Hq/2,D], o_branch [T,Hq,D], lse [T,Hq]). With `window` the causal sliding window
    inside every sequence."""
    if sink is not None:  # with a window: the first `sink` keys stay visible, o_branch fp32
        return _invoke(_TRAIN_VARLEN_SINK, LIB.addresses["diffattn_v2_prefill_varlen_window_sink_train"], q, k, v, lam,
                       cu_seqlens, max_seqlen, _window_of_sink(window, causal), sink, out, o_branch, lse, stream)
    for t, n, nd in ((q, "q", 3), (k, "k", 3), (v, "v", 3)):
        _need(t, n, torch.bfloat16, nd)
    _need(lam, "lam", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    out = _empty(stream, (T, Hq // 2, D), dtype=torch.bfloat16, device=q.device) if out is None else out
    o_branch = _empty(stream, (T, Hq, D), dtype=torch.bfloat16, device=q.device) if o_branch is None else o_branch
    lse = _empty(stream, (T, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", torch.bfloat16, 3)
    _need(o_branch, "o_branch", torch.bfloat16, 3)
    _need(lse, "lse", torch.float32, 2)
    if window is not None:
        st = LIB.diffattn_v2_prefill_varlen_window_train(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out),
                                                         _ptr(o_branch), _ptr(lse), _ptr(cu_seqlens), B,
                                                         int(max_seqlen), T, Hq, Hkv, D, int(window),
                                                         _stream(stream, q.device))
        _check(st, "diffattn_v2_prefill_varlen_window_train")
        return out, o_branch, lse
    st = LIB.diffattn_v2_prefill_varlen_train(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out), _ptr(o_branch),
                                              _ptr(lse), _ptr(cu_seqlens), B, int(max_seqlen), T, Hq, Hkv, D,
                                              1 if causal else 0, _stream(stream, q.device))
    _check(st, "diffattn_v2_prefill_varlen_train")
    return out, o_branch, lse


def backward_varlen_workspace_size(B, total_tokens, Hq) -> int:
    return int(LIB.diffattn_v2_backward_varlen_workspace_size(B, total_tokens, Hq))


def backward_varlen(q, k, v, lam, o_branch, lse, dout, cu_seqlens, max_seqlen, causal=True, workspace=None,
                    stream=None, window=None, sink=None):
    """Gradients of the packed-sequence prefill: returns (dq, dk, dv, dlam) in the packed layouts.
    With `window` the gradients of the causal sliding-window packed prefill."""
    if sink is not None:  # with a window: the first `sink` keys stay visible, o_branch fp32
        return _invoke(_BACKWARD_VARLEN_SINK, LIB.addresses["diffattn_v2_backward_varlen_window_sink"], q, k, v, lam,
                       cu_seqlens, max_seqlen, o_branch, lse, dout, _window_of_sink(window, causal), sink, None, None,
                       None, None, LIB.addresses["diffattn_v2_backward_varlen_window_sink_workspace_size"], workspace,
                       stream)
    for t, n, nd in ((q, "q", 3), (k, "k", 3), (v, "v", 3), (o_branch, "o_branch", 3), (dout, "dout", 3)):
        _need(t, n, torch.bfloat16, nd)
    _need(lam, "lam", torch.float32, 2)
    _need(lse, "lse", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    dq, dk, dv, dlam = (_empty_like(stream, t) for t in (q, k, v, lam))
    ws_bytes = backward_varlen_workspace_size(B, T, Hq)
    if workspace is None:
        workspace = _empty(stream, max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    ws_given = workspace.numel() * workspace.element_size()
    if window is not None:
        st = LIB.diffattn_v2_backward_varlen_window(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(o_branch), _ptr(lse),
                                                    _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlam),
                                                    _ptr(cu_seqlens), B, int(max_seqlen), T, Hq, Hkv, D, int(window),
                                                    _ptr(workspace), ws_given, _stream(stream, q.device))
        _check(st, "diffattn_v2_backward_varlen_window")
        return dq, dk, dv, dlam
    st = LIB.diffattn_v2_backward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(o_branch), _ptr(lse),
                                         _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlam), _ptr(cu_seqlens), B,
                                         int(max_seqlen), T, Hq, Hkv, D, 1 if causal else 0, _ptr(workspace),
                                         ws_given, _stream(stream, q.device))
    _check(st, "diffattn_v2_backward_varlen")
    return dq, dk, dv, dlam


def decode_workspace_size(B, Smax, Hq, Hkv, D) -> int:
    return int(LIB.diffattn_v2_decode_workspace_size(B, Smax, Hq, Hkv, D))


def decode(q, kcache, vcache, seqlens, lam, out=None, workspace=None, stream=None, window=None, sink=None):
    """bf16 decode step: q [B,Hq,D], caches [B,Smax,Hkv,D], seqlens int32 [B], lam fp32 [B,Hq/2].
    With `window` the new token sees only its sequence's last `window` keys, with `sink` besides
    the first `sink` ones (no workspace)."""
    if sink is not None:
        return _invoke(_DECODE_SINK, LIB.addresses["diffattn_v2_decode_window_sink"], q, kcache, vcache, seqlens, lam,
                       _window_of_sink(window, True), sink, out, stream)
    _need(q, "q", torch.bfloat16, 3)
    _need(kcache, "kcache", torch.bfloat16, 4)
    _need(vcache, "vcache", torch.bfloat16, 4)
    _need(seqlens, "seqlens", torch.int32, 1)
    _need(lam, "lam", torch.float32, 2)
    B, Hq, D = q.shape
    Smax, Hkv = kcache.shape[1], kcache.shape[2]
    if out is None:
        out = _empty(stream, (B, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 3)
    need = decode_workspace_size(B, Smax, Hq, Hkv, D)
    if workspace is None:
        workspace = _empty(stream, max(need, 16), dtype=torch.uint8, device=q.device)
    if window is not None:
        st = LIB.diffattn_v2_decode_window(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(lam), _ptr(out), B,
                                           Smax, Hq, Hkv, D, int(window), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream, q.device))
        _check(st, "diffattn_v2_decode_window")
        return out
    st = LIB.diffattn_v2_decode(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(lam), _ptr(out), B, Smax,
                                Hq, Hkv, D, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream, q.device))
    _check(st, "diffattn_v2_decode")
    return out


def decode_multi(q, kcache, vcache, seqlens, lam, out=None, workspace=None, stream=None):
    """bf16 decode of T new tokens per sequence: q [B,T,Hq,D], lam fp32 [B,T,Hq/2] ->
    out bf16 [B,T,Hq/2,D]; token t sees keys [0, seqlens[b] - T + t + 1)."""
    _need(q, "q", torch.bfloat16, 4)
    _need(kcache, "kcache", torch.bfloat16, 4)
    _need(vcache, "vcache", torch.bfloat16, 4)
    _need(seqlens, "seqlens", torch.int32, 1)
    _need(lam, "lam", torch.float32, 3)
    B, T, Hq, D = q.shape
    Smax, Hkv = kcache.shape[1], kcache.shape[2]
    if out is None:
        out = _empty(stream, (B, T, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 4)
    need = int(LIB.diffattn_v2_decode_multi_workspace_size(B, T, Smax, Hq, Hkv, D))
    if workspace is None:
        workspace = _empty(stream, max(need, 16), dtype=torch.uint8, device=q.device)
    st = LIB.diffattn_v2_decode_multi(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(lam), _ptr(out), B, T,
                                      Smax, Hq, Hkv, D, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(stream, q.device))
    _check(st, "diffattn_v2_decode_multi")
    return out


def decode_paged(q, kpages, vpages, block_table, seqlens, lam, out=None, workspace=None, stream=None, window=None,
                 sink=None):
    """bf16 decode over a paged cache: kpages/vpages [num_pages, page_size, Hkv, D],
    block_table int32 [B, max_pages], seqlens int32 [B], lam fp32 [B, Hq/2]. With `window`
    the new token sees only its sequence's last `window` keys, with `sink` besides the first
    `sink` ones (no workspace; entries of pages without a visible key may be -1)."""
    if sink is not None:
        return _invoke(_DECODE_PAGED_SINK, LIB.addresses["diffattn_v2_decode_paged_window_sink"], q, kpages, vpages,
                       block_table, seqlens, lam, _window_of_sink(window, True), sink, out, stream)
    _need(q, "q", torch.bfloat16, 3)
    _need(kpages, "kpages", torch.bfloat16, 4)
    _need(vpages, "vpages", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seqlens, "seqlens", torch.int32, 1)
    _need(lam, "lam", torch.float32, 2)
    B, Hq, D = q.shape
    num_pages, page_size, Hkv = kpages.shape[0], kpages.shape[1], kpages.shape[2]
    max_pages = block_table.shape[1]
    if out is None:
        out = _empty(stream, (B, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 3)
    need = decode_workspace_size(B, max_pages * page_size, Hq, Hkv, D)
    if workspace is None:
        workspace = _empty(stream, max(need, 16), dtype=torch.uint8, device=q.device)
    if window is not None:
        st = LIB.diffattn_v2_decode_paged_window(_ptr(q), _ptr(kpages), _ptr(vpages), _ptr(block_table), _ptr(seqlens),
                                                 _ptr(lam), _ptr(out), B, max_pages, page_size, num_pages, Hq, Hkv, D,
                                                 int(window), _ptr(workspace),
                                                 workspace.numel() * workspace.element_size(), _stream(stream, q.device))
        _check(st, "diffattn_v2_decode_paged_window")
        return out
    st = LIB.diffattn_v2_decode_paged(_ptr(q), _ptr(kpages), _ptr(vpages), _ptr(block_table), _ptr(seqlens), _ptr(lam),
                                      _ptr(out), B, max_pages, page_size, num_pages, Hq, Hkv, D, _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream, q.device))
    _check(st, "diffattn_v2_decode_paged")
    return out


def decode_f32(q, kcache, vcache, seqlens, lam, out=None, stream=None):
    """fp32 decode step on CUDA cores; same layout as decode with fp32 tensors."""
    _need(q, "q", torch.float32, 3)
    _need(kcache, "kcache", torch.float32, 4)
    _need(vcache, "vcache", torch.float32, 4)
    _need(seqlens, "seqlens", torch.int32, 1)
    _need(lam, "lam", torch.float32, 2)
    B, Hq, D = q.shape
    Smax, Hkv = kcache.shape[1], kcache.shape[2]
    if out is None:
        out = _empty(stream, (B, Hq // 2, D), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, 3)
    st = LIB.diffattn_v2_decode_f32(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(lam), _ptr(out), B,
                                    Smax, Hq, Hkv, D, _stream(stream, q.device))
    _check(st, "diffattn_v2_decode_f32")
    return out


def lambda_v1(lq1, lk1, lq2, lk2, lambda_init=0.8, rows=1, out=None, stream=None):
    """V1 lambda per pair, broadcast to `rows` rows: out fp32 [rows, n_pairs]."""
    for t, n in ((lq1, "lq1"), (lk1, "lk1"), (lq2, "lq2"), (lk2, "lk2")):
        _need(t, n, torch.float32, 2)
    n_pairs, d = lq1.shape
    if out is None:
        out = _empty(stream, (rows, n_pairs), dtype=torch.float32, device=lq1.device)
    if out.dtype != torch.float32 or not out.is_contiguous() or out.numel() != rows * n_pairs:
        raise ValueError("out must be a contiguous fp32 tensor with rows*n_pairs elements")
    st = LIB.diffattn_v2_lambda_v1(_ptr(lq1), _ptr(lk1), _ptr(lq2), _ptr(lk2), float(lambda_init), n_pairs, d, rows,
                                   _ptr(out), _stream(stream, lq1.device))
    _check(st, "diffattn_v2_lambda_v1")
    return out


def lambda_v2(x, w_lambda, bias=None, out=None, stream=None):
    """V2 lambda sigmoid(x @ w_lambda + bias): x bf16 [T, d_model], w_lambda bf16
    [d_model, n_pairs], bias fp32 [n_pairs] or None -> fp32 [T, n_pairs]."""
    _need(x, "x", torch.bfloat16, 2)
    _need(w_lambda, "w_lambda", torch.bfloat16, 2)
    if bias is not None:
        _need(bias, "bias", torch.float32, 1)
    T, d = x.shape
    n_pairs = w_lambda.shape[1]
    if out is None:
        out = _empty(stream, (T, n_pairs), dtype=torch.float32, device=x.device)
    st = LIB.diffattn_v2_lambda_v2(_ptr(x), _ptr(w_lambda), _ptr(bias), T, d, n_pairs, _ptr(out),
                                   _stream(stream, x.device))
    _check(st, "diffattn_v2_lambda_v2")
    return out


def prefill_fused_lambda(q, k, v, x, w_lambda_t, bias=None, out=None, lambda_out=None, causal=True, stream=None):
    """bf16 prefill with the V2 lambda sigmoid(x . w_lambda_t[p] + bias[p]) computed inside the
    kernel: q [B,S,Hq,D], k/v [B,S,Hkv,D], x bf16 [B,S,d_model], w_lambda_t bf16 [Hq/2, d_model]
    (the projection transposed), bias fp32 [Hq/2] or None; lambda_out fp32 [B,S,Hq/2] receives
    the lambda when given. Returns out bf16 [B,S,Hq/2,D]."""
    for t, n, nd in ((q, "q", 4), (k, "k", 4), (v, "v", 4), (x, "x", 3), (w_lambda_t, "w_lambda_t", 2)):
        _need(t, n, torch.bfloat16, nd)
    if bias is not None:
        _need(bias, "bias", torch.float32, 1)
    if lambda_out is not None:
        _need(lambda_out, "lambda_out", torch.float32, 3)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    d_model = x.shape[2]
    if out is None:
        out = _empty(stream, (B, S, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 4)
    st = LIB.diffattn_v2_prefill_fused_lambda(_ptr(q), _ptr(k), _ptr(v), _ptr(x), _ptr(w_lambda_t), _ptr(bias),
                                              _ptr(out), _ptr(lambda_out), B, S, Hq, Hkv, D, d_model,
                                              1 if causal else 0, _stream(stream, q.device))
    _check(st, "diffattn_v2_prefill_fused_lambda")
    return out


def device_error(stream=None, device=None) -> int:
    """Synchronise the stream and return (and clear) the kernels' device error word."""
    code = ctypes.c_int(0)
    st = LIB.diffattn_v2_device_error(ctypes.byref(code), _stream(stream, device))
    if st == ERR_CUDA:
        raise DiffAttnError(st, "diffattn_v2_device_error")
    return code.value


def decode_noalloc(q, kcache, vcache, seqlens, lam, out=None, stream=None):
    """bf16 decode step whose partials live in the library's fixed 16 MiB device array.

    For callers that cannot allocate device memory (a KV-cache pool or caching allocator
    that owns nearly all HBM, plugin interfaces without a workspace). The library allocates
    nothing; calls that overlap on the GPU share the array and race, so serialise them.
    Sizes needing more than 16 MiB of partials raise (DA2_ERR_UNSUPPORTED)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(kcache, "kcache", torch.bfloat16, 4)
    _need(vcache, "vcache", torch.bfloat16, 4)
    _need(seqlens, "seqlens", torch.int32, 1)
    _need(lam, "lam", torch.float32, 2)
    B, Hq, D = q.shape
    Smax, Hkv = kcache.shape[1], kcache.shape[2]
    if out is None:
        out = _empty(stream, (B, Hq // 2, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 3)
    st = LIB.diffattn_v2_decode_noalloc(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(lam), _ptr(out),
                                        B, Smax, Hq, Hkv, D, _stream(stream, q.device))
    _check(st, "diffattn_v2_decode_noalloc")
    return out


def rope(q, k, positions, inv_freq, sections, q_out=None, k_out=None, inverse=False, interleaved=False, stream=None):
    """Rotary positions with len(sections) axes (1 to 4): q [T,Hq,D], k [T,Hkv,D] or None, bf16 or
    fp32 (heads of a token contiguous, any token stride), positions int32 [n_axes, T], inv_freq
    fp32 [sum(sections)]; pair c turns by positions[axis(c)] * inv_freq[c]. Pairs are dimensions
    (c, c + P), interleaved (2c, 2c + 1); `inverse` turns back (the gradient). Outputs may be the
    inputs. Returns (q_out, k_out)."""
    return _invoke(_ROPE, LIB.addresses["diffattn_v2_rope"], q, k, positions, inv_freq, sections, q_out, k_out, inverse,
                   interleaved, stream)


def rope_append_paged(q, k, v, positions, inv_freq, sections, kpages, vpages, block_table, seqlens, cu_seqlens=None,
                      q_out=None, interleaved=False, stream=None):
    """Rotary positions of a serving step's new tokens, with k (turned) and v written to their rows
    of the paged cache: token i of sequence b's n_b new ones is logical position
    seqlens[b] - n_b + i. q [T,Hq,D], k and v [T,Hkv,D] as in rope, caches
    [num_pages, page_size, Hkv, D] of the same dtype; cu_seqlens int32 [B+1] tells the sequences'
    new tokens (None: one each). Rows of q_out behind the last sequence are not written. Returns
    q_out."""
    return _invoke(_ROPE_APPEND, LIB.addresses["diffattn_v2_rope_append_paged"], q, k, v, positions, inv_freq, sections,
                   kpages, vpages, block_table, seqlens, cu_seqlens, q_out, interleaved, stream)


def _of_nothing(result, nothing, stream):
    """The result of a bookkeeping call, checked and allocated by it. One on nothing launches nothing:
    its result is 0, written on the call's stream."""
    if nothing:
        with torch.cuda.stream(None if stream is None else _torch_stream(stream, result.device)):
            result.zero_()
    return result


def cache_extend(block_table, seqlens, refs, n_new, page_size, result=None, stream=None):
    """n_new[b] more tokens for every sequence: seqlens grows and the pages that are missing are
    taken from the free ones (refs == 0), lowest first. Returns result int32 [1] on the device:
    pages taken, or -1 (too few free pages or a full row; nothing changed)."""
    result = _invoke(_CACHE_EXTEND, LIB.addresses["diffattn_v2_cache_extend"], block_table, seqlens, refs, n_new,
                     page_size, result, stream)
    return _of_nothing(result, seqlens.numel() == 0, stream)


def cache_fork(block_table, seqlens, refs, parents, children, page_size, copies=None, result=None, stream=None):
    """Row children[i] (empty) continues what row parents[i] holds: whole pages are shared, a partly
    filled last page gets a page of its own. Returns (copies int32 [n,2] for cache_copy_pages, -1
    where there is none; result int32 [1]: pages taken, -1 too few free pages, -2 a bad pair)."""
    copies, result = _invoke(_CACHE_FORK, LIB.addresses["diffattn_v2_cache_fork"], block_table, seqlens, refs, parents,
                             children, page_size, copies, result, stream)
    return copies, _of_nothing(result, parents.numel() == 0, stream)


def cache_trim(block_table, seqlens, refs, page_size, window, sink, result=None, stream=None):
    """Pages that hold neither one of the first `sink` keys nor one of the last `window` leave their
    sequence. Returns result int32 [1]: pages that became free."""
    result = _invoke(_CACHE_TRIM, LIB.addresses["diffattn_v2_cache_trim"], block_table, seqlens, refs, page_size, window,
                     sink, result, stream)
    return _of_nothing(result, seqlens.numel() == 0, stream)


def cache_free(block_table, seqlens, refs, seqs, result=None, stream=None):
    """The listed sequences (int32; negative entries are padding) give their pages back and become
    empty. Returns result int32 [1]: pages that became free, or -2 (an index >= B; nothing changed)."""
    result = _invoke(_CACHE_FREE, LIB.addresses["diffattn_v2_cache_free"], block_table, seqlens, refs, seqs, result, stream)
    return _of_nothing(result, seqs.numel() == 0, stream)


def cache_compact(block_table, refs, block_table_out=None, refs_out=None, moves=None, result=None, stream=None):
    """A plan that brings the L pages in use to the front of the pool. Returns (block_table, refs,
    moves int32 [num_pages // 2, 2] for cache_copy_pages, result int32 [1] = L); the outputs may be
    the inputs' own tensors."""
    return _invoke(_CACHE_COMPACT, LIB.addresses["diffattn_v2_cache_compact"], block_table, refs, block_table_out,
                   refs_out, moves, result, stream)


def cache_copy_pages(kpages, vpages, copies, stream=None):
    """Copies page copies[i][0] to page copies[i][1] in both caches [num_pages, ...]; pairs with a
    negative entry are skipped. No page may be a destination twice, or a source and a destination."""
    _invoke(_CACHE_COPY, LIB.addresses["diffattn_v2_cache_copy_pages"], kpages, vpages, copies, stream)


_BATCH = "q:bf16[B,S,Hq,D] k:bf16[B,S,Hkv,D] v:bf16[B,S,Hkv,D] lam:f32[B,S,Hq/2] "
_PACKED = "q:bf16[T,Hq,D] k:bf16[T,Hkv,D] v:bf16[T,Hkv,D] lam:f32[T,Hq/2] cu_seqlens:i32[B+1] #max_seqlen "
_POOL = "block_table:i32[B,max_pages] seqlens:i32[B] refs:i32[N] "
_PREFILL_SINK = _entry("diffattn_v2_prefill_window_sink", _BATCH + """#window #sink >out:bf16[B,S,Hq/2,D]
    -> q k v lam out B S Hq Hkv D window sink => out""")
_PREFILL_VARLEN_SINK = _entry("diffattn_v2_prefill_varlen_window_sink", _PACKED + """#window #sink
    >out:bf16[T,Hq/2,D] -> q k v lam out cu_seqlens B max_seqlen T Hq Hkv D window sink => out""")
_TRAIN_SINK = _entry("diffattn_v2_prefill_window_sink_train", _BATCH + """#window #sink >out:bf16[B,S,Hq/2,D]
    >o_branch:f32[B,S,Hq,D] >lse:f32[B,S,Hq] -> q k v lam out o_branch lse B S Hq Hkv D window sink
    => out o_branch lse""")
_TRAIN_VARLEN_SINK = _entry("diffattn_v2_prefill_varlen_window_sink_train", _PACKED + """#window #sink
    >out:bf16[T,Hq/2,D] >o_branch:f32[T,Hq,D] >lse:f32[T,Hq]
    -> q k v lam out o_branch lse cu_seqlens B max_seqlen T Hq Hkv D window sink => out o_branch lse""")
_BACKWARD_SINK = _entry("diffattn_v2_backward_window_sink", _BATCH + """o_branch:f32[B,S,Hq,D] lse:f32[B,S,Hq]
    dout:bf16[B,S,Hq/2,D] #window #sink >dq:bf16[B,S,Hq,D] >dk:bf16[B,S,Hkv,D] >dv:bf16[B,S,Hkv,D] >dlam:f32[B,S,Hq/2]
    @workspace(B,S,Hq,Hkv,window,sink)
    -> q k v lam o_branch lse dout dq dk dv dlam B S Hq Hkv D window sink workspace workspace.n => dq dk dv dlam""")
_BACKWARD_VARLEN_SINK = _entry("diffattn_v2_backward_varlen_window_sink", _PACKED + """o_branch:f32[T,Hq,D] lse:f32[T,Hq]
    dout:bf16[T,Hq/2,D] #window #sink >dq:bf16[T,Hq,D] >dk:bf16[T,Hkv,D] >dv:bf16[T,Hkv,D] >dlam:f32[T,Hq/2]
    @workspace(B,max_seqlen,T,Hq,Hkv,window,sink)
    -> q k v lam o_branch lse dout dq dk dv dlam cu_seqlens B max_seqlen T Hq Hkv D window sink workspace workspace.n
    => dq dk dv dlam""")
_DECODE_SINK = _entry("diffattn_v2_decode_window_sink", """q:bf16[B,Hq,D] kcache:bf16[B,Smax,Hkv,D]
    vcache:bf16[B,Smax,Hkv,D] seqlens:i32[B] lam:f32[B,Hq/2] #window #sink >out:bf16[B,Hq/2,D]
    -> q kcache vcache seqlens lam out B Smax Hq Hkv D window sink => out""")
_DECODE_PAGED_SINK = _entry("diffattn_v2_decode_paged_window_sink", """q:bf16[B,Hq,D] kpages:bf16[N,ps,Hkv,D]
    vpages:bf16[N,ps,Hkv,D] block_table:i32[B,max_pages] seqlens:i32[B] lam:f32[B,Hq/2] #window #sink
    >out:bf16[B,Hq/2,D] -> q kpages vpages block_table seqlens lam out B max_pages ps N Hq Hkv D window sink => out""")
_ROPE = _entry("diffattn_v2_rope", """q:io<T,Hq,D> k:io<T,Hkv,D>? positions:i32[%.n,T] inv_freq:f32[%.sum] %sections
    >q_out:io<T,Hq,D> >k_out:io<T,Hkv,D>?k !inverse !interleaved
    -> q k q_out k_out positions inv_freq % %.n T Hq Hkv D q.s k.s q_out.s k_out.s io interleaved inverse
    => q_out k_out""")
_ROPE_APPEND = _entry("diffattn_v2_rope_append_paged", """q:io<T,Hq,D> k:io<T,Hkv,D> v:io<T,Hkv,D>
    positions:i32[%.n,T] inv_freq:f32[%.sum] %sections kpages:io[N,ps,Hkv,D] vpages:io[N,ps,Hkv,D]
    block_table:i32[B,max_pages] seqlens:i32[B] cu_seqlens:i32[B+1]? >q_out:io<T,Hq,D> !interleaved
    -> q k v q_out positions inv_freq % %.n kpages vpages block_table seqlens cu_seqlens T B max_pages ps N Hq Hkv D
    q.s k.s v.s q_out.s io interleaved => q_out""")
_CACHE_EXTEND = _entry("diffattn_v2_cache_extend", _POOL + """n_new:i32[B] #page_size >result:i32[1]
    -> block_table seqlens refs n_new result B max_pages page_size N => result""")
_CACHE_FORK = _entry("diffattn_v2_cache_fork", _POOL + """parents:i32[n] children:i32[n] #page_size >copies:i32[n,2]
    >result:i32[1] -> block_table seqlens refs parents children copies result n B max_pages page_size N
    => copies result""")
_CACHE_TRIM = _entry("diffattn_v2_cache_trim", _POOL + """#page_size #window #sink >result:i32[1]
    -> block_table seqlens refs result B max_pages page_size N window sink => result""")
_CACHE_FREE = _entry("diffattn_v2_cache_free", _POOL + """seqs:i32[n] >result:i32[1]
    -> block_table seqlens refs seqs result n B max_pages N => result""")
_CACHE_COMPACT = _entry("diffattn_v2_cache_compact", """block_table:i32[B,max_pages] refs:i32[N]
    >block_table_out:i32[B,max_pages] >refs_out:i32[N] >moves:i32[N/2,2] >result:i32[1]
    -> block_table refs block_table_out refs_out moves result B max_pages N
    => block_table_out refs_out moves result""")
_CACHE_COPY = _entry("diffattn_v2_cache_copy_pages", """kpages:any[N,...] vpages:any[N,...] copies:i32[n,2]
    -> kpages vpages copies n N kpages.size =>""")
