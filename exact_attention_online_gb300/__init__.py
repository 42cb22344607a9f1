"""GB300-native exact attention: online-softmax forward and recomputation
backward, as hand-written sm_103a kernels behind the C ABI of include/fa.h.

This module is the thin Python binding: each function has the name of the C
entry point it calls and does argument marshalling only (tensor -> pointer,
shape -> ints, current CUDA stream).  Every step of the computation runs in
libfa.so; there is no other code path.  A nonzero fa_status raises FAError.

Layouts (as in include/fa.h): q, o, dout, dq bf16 [B, H, N, d]; k, v, dk, dv
bf16 [B, Hkv, N, d]; lse fp32 [B, H, N]; all contiguous CUDA tensors.
"""
from __future__ import annotations

import ctypes

from ._native import EXPORTS, LIB_PATH, binding, build, lib

FA_OK = 0
FA_ERR_INVALID_ARG = -1
FA_ERR_UNSUPPORTED = -2
FA_ERR_ALIGNMENT = -3
FA_ERR_WORKSPACE = -4
FA_ERR_CUDA = -5
FA_ERR_TIMEOUT = -6

__all__ = ["build", "lib", "LIB_PATH", "EXPORTS", "FAError", "fa_fwd", "fa_fwd_precise", "fa_bwd",
           "fa_bwd_workspace_size", "fa_bwd_precise", "fa_bwd_preprocess",
           "fa_bwd_preprocess_precise", "fa_bwd_dkdv", "fa_bwd_dq_convert",
           "fa_device_status", "fa_device_status_detail", "fa_status_string",
           "fa_kernel_launches", "fa_watchdog_selftest", "attention", "attention_backward",
           "fa_fwd_window", "fa_bwd_window", "fa_bwd_dkdv_window", "attention_window",
           "attention_window_backward", "fa_fwd_varlen", "fa_bwd_varlen",
           "fa_bwd_varlen_workspace_size", "attention_varlen", "attention_varlen_backward",
           "fa_fp8_buffer_size", "fa_fp8_quantize", "fa_fwd_fp8", "attention_fp8",
           "fa_fwd_decode_workspace_size", "fa_fwd_decode", "attention_decode",
           "fa_fwd_train", "fa_bwd_train", "fa_bwd_preprocess_train", "fa_exp2_check",
           "fa_ex2_rate",
           "fa_fwd_window_train", "fa_bwd_window_train",
           "fa_kv_append", "fa_kv_append_varlen", "fa_kv_gather", "fa_kv_gather_varlen",
           "fa_fwd_decode_paged_workspace_size", "fa_fwd_decode_paged", "attention_decode_paged",
           "fa_kv_reserve", "fa_kv_release", "fa_kv_slots", "fa_kv_slots_varlen",
           "rope_frequencies", "fa_rope", "rope", "fa_rope_append",
           "fa_fwd_cross_workspace_size", "fa_fwd_cross", "fa_fwd_cross_varlen",
           "fa_bwd_cross_workspace_size", "fa_bwd_cross", "fa_bwd_cross_varlen",
           "fa_fwd_cross_decode_workspace_size", "fa_fwd_cross_decode", "attention_cross",
           "attention_cross_backward", "attention_cross_varlen",
           "attention_cross_varlen_backward", "attention_cross_decode"]


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_status_string(status)} ({status})")


def fa_status_string(status: int) -> str:
    return lib().fa_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != FA_OK:
        raise FAError(status, where)


_cuda = None   # (current device, raw current stream of a device), once CUDA is up


def _runtime():
    """torch's short forms of the two where it has them, as a small call's time is the host's; they
    are not part of its public interface, which answers else."""
    global _cuda
    if _cuda is None:
        import torch
        torch.cuda.current_device()   # raises without a CUDA runtime
        _cuda = (getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device,
                 getattr(torch._C, "_cuda_getCurrentRawStream", None) or
                 (lambda device: torch.cuda.current_stream(device).cuda_stream))
    return _cuda


def _current_index() -> int:
    """Index of the current CUDA device: every pointer the library receives
    must be memory of this device (its kernels and tensor maps are built
    there)."""
    try:
        return _runtime()[0]()
    except Exception:   # no CUDA runtime in this process: the library rejects the call
        return 0


# What a function of binding() returns for arguments that are not exactly what the call takes:
# the wrapper's own checks then find what is wrong with them, or nothing (a size that is no int).
_EXPLAIN = 1


def _done(status: int, where: str) -> bool:
    """Whether binding() has made the call; raises where the library refused it."""
    if status == _EXPLAIN:
        return False
    if status != FA_OK:
        raise FAError(status, where)
    return True


def _handle(stream):
    """A stream for binding(): None is the current one."""
    return None if stream is None else _stream(stream)


def _on_current_device(t, name) -> None:
    dev = getattr(t, "device", None)
    idx = getattr(dev, "index", None)
    cur = _current_index()
    if idx is not None and idx != cur:
        raise ValueError(f"{name} is on cuda:{idx} but the current device is cuda:{cur}")


def _stream(stream):
    if stream is None:
        device, raw_stream = _runtime()
        return raw_stream(device())
    if hasattr(stream, "cuda_stream"):
        _on_current_device(stream, "stream")
        return stream.cuda_stream
    return int(stream)


def _ptr(t, name, dtype, shape):
    """Device pointer of t after checking its shape (the C entry points see
    only pointers, so a short buffer would be read or written past its end),
    dtype, contiguity and device: a CUDA tensor of the current device, so that
    every operand of a call shares one device."""
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {str(dtype)[6:]} tensor")
    _on_current_device(t, name)
    return t.data_ptr()


def _c_int(x, name) -> int:
    """x for a C int argument, which would take the lower 32 bits of a larger one."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} = {x} is out of range")
    return x


def _bytes(size_of, *sizes) -> int:
    return int(size_of(*(_c_int(x, "a size") for x in sizes)))


def _bf16(t, name, shape=None):
    import torch
    return _ptr(t, name, torch.bfloat16, shape)


def _f32(t, name, shape=None):
    import torch
    return _ptr(t, name, torch.float32, shape)


def _dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be 4-D [B, H(kv), N, d]")
    B, H, N, d = q.shape
    if k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree")
    return B, H, k.shape[1], N, d


def _shapes(B, H, Hkv, N, d):
    """Shapes of the query-side tensors (q, o, dout, dq), the key-side tensors
    (k, v, dk, dv) and lse: [B, H, N, d], [B, Hkv, N, d], [B, H, N]."""
    return (B, H, N, d), (B, Hkv, N, d), (B, H, N)


def fa_fwd(q, k, v, o, lse, causal: bool, scale: float, stream=None) -> None:
    B, H, Hkv, N, d = _dims(q, k)
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    _check(lib().fa_fwd(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _bf16(o, "o", qs),
                        _f32(lse, "lse", ls), B, H, Hkv, N, d, int(bool(causal)), float(scale),
                        _stream(stream)), "fa_fwd")


def fa_fwd_precise(q, k, v, o, lse, causal: bool, scale: float, stream=None) -> None:
    """o: fp32 [B, H, N, d]."""
    B, H, Hkv, N, d = _dims(q, k)
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    _check(lib().fa_fwd_precise(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _f32(o, "o", qs),
                                _f32(lse, "lse", ls), B, H, Hkv, N, d, int(bool(causal)),
                                float(scale), _stream(stream)), "fa_fwd_precise")


def fa_fwd_window(q, k, v, o, lse, window: int, scale: float, stream=None) -> None:
    """Causal sliding window: query i attends to keys i - window < j <= i."""
    B, H, Hkv, N, d = _dims(q, k)
    window = _c_int(window, "window")
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    _check(lib().fa_fwd_window(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _bf16(o, "o", qs),
                               _f32(lse, "lse", ls), B, H, Hkv, N, d, window, float(scale),
                               _stream(stream)), "fa_fwd_window")


def _i32(t, name, shape=None):
    import torch
    return _ptr(t, name, torch.int32, shape)


def _varlen_dims(q, k, cu_seqlens):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("packed q and k must be 3-D [H(kv), total, d]")
    H, total, d = q.shape
    if k.shape[1] != total or k.shape[2] != d:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree")
    if cu_seqlens.dim() != 1:
        raise ValueError("cu_seqlens must be 1-D [B + 1]")
    return cu_seqlens.numel() - 1, H, k.shape[0], total, d


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, max_seqlen: int, causal: bool, scale: float,
                  stream=None) -> None:
    """Packed sequences: q, o [H, total, d], k, v [Hkv, total, d], lse [H, total],
    cu_seqlens int32 [B + 1] on the device."""
    B, H, Hkv, total, d = _varlen_dims(q, k, cu_seqlens)
    max_seqlen = _c_int(max_seqlen, "max_seqlen")
    qs, ks = (H, total, d), (Hkv, total, d)
    _check(lib().fa_fwd_varlen(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _bf16(o, "o", qs),
                               _f32(lse, "lse", (H, total)), _i32(cu_seqlens, "cu_seqlens"), B,
                               max_seqlen, total, H, Hkv, d, int(bool(causal)),
                               float(scale), _stream(stream)), "fa_fwd_varlen")


def fa_bwd_varlen_workspace_size(B: int, H: int, Hkv: int, max_seqlen: int, d: int) -> int:
    return _bytes(lib().fa_bwd_varlen_workspace_size, B, H, Hkv, max_seqlen, d)


def fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens, max_seqlen: int,
                  causal: bool, scale: float, stream=None) -> None:
    B, H, Hkv, total, d = _varlen_dims(q, k, cu_seqlens)
    max_seqlen = _c_int(max_seqlen, "max_seqlen")
    qs, ks = (H, total, d), (Hkv, total, d)
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_varlen(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _bf16(o, "o", qs),
                               _bf16(dout, "dout", qs), _f32(lse, "lse", (H, total)),
                               _bf16(dq, "dq", qs), _bf16(dk, "dk", ks), _bf16(dv, "dv", ks),
                               wp, wb,
                               _i32(cu_seqlens, "cu_seqlens"), B, max_seqlen, total, H, Hkv,
                               d, int(bool(causal)), float(scale), _stream(stream)),
           "fa_bwd_varlen")


def fa_bwd_workspace_size(B: int, H: int, Hkv: int, N: int, d: int) -> int:
    return _bytes(lib().fa_bwd_workspace_size, B, H, Hkv, N, d)


def _ws(workspace):
    import torch
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _on_current_device(workspace, "workspace")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal: bool, scale: float,
           stream=None) -> None:
    B, H, Hkv, N, d = _dims(q, k)
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _bf16(o, "o", qs),
                        _bf16(dout, "dout", qs), _f32(lse, "lse", ls), _bf16(dq, "dq", qs),
                        _bf16(dk, "dk", ks), _bf16(dv, "dv", ks), wp, wb, B, H, Hkv, N, d,
                        int(bool(causal)),
                        float(scale), _stream(stream)), "fa_bwd")


def fa_bwd_precise(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal: bool, scale: float,
                   stream=None) -> None:
    """o: the fp32 output of fa_fwd_precise."""
    B, H, Hkv, N, d = _dims(q, k)
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_precise(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _f32(o, "o", qs),
                                _bf16(dout, "dout", qs), _f32(lse, "lse", ls), _bf16(dq, "dq", qs),
                                _bf16(dk, "dk", ks), _bf16(dv, "dv", ks), wp, wb, B, H, Hkv, N, d,
                                int(bool(causal)), float(scale), _stream(stream)),
           "fa_bwd_precise")


def fa_fwd_train(q, k, v, o, lse, workspace, causal: bool, scale: float, stream=None) -> None:
    """fa_fwd, plus the backward's workspace prepared for fa_bwd_train; o is
    bf16, or fp32 (the precise forward)."""
    B, H, Hkv, N, d = _dims(q, k)
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    wp, wb = _ws(workspace)
    import torch
    if o.dtype == torch.float32:
        fn, op, name = lib().fa_fwd_train_precise, _f32(o, "o", qs), "fa_fwd_train_precise"
    else:
        fn, op, name = lib().fa_fwd_train, _bf16(o, "o", qs), "fa_fwd_train"
    _check(fn(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), op, _f32(lse, "lse", ls), wp, wb,
              B, H, Hkv, N, d, int(bool(causal)), float(scale), _stream(stream)), name)


def fa_bwd_train(q, k, v, o, dout, dq, dk, dv, workspace, causal: bool, scale: float,
                 stream=None) -> None:
    """The backward of fa_fwd_train, on the workspace it prepared; o is bf16 or
    fp32 as that forward wrote it."""
    B, H, Hkv, N, d = _dims(q, k)
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    wp, wb = _ws(workspace)
    import torch
    if o.dtype == torch.float32:
        fn, op, name = lib().fa_bwd_train_precise, _f32(o, "o", qs), "fa_bwd_train_precise"
    else:
        fn, op, name = lib().fa_bwd_train, _bf16(o, "o", qs), "fa_bwd_train"
    _check(fn(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), op, _bf16(dout, "dout", qs),
              _bf16(dq, "dq", qs), _bf16(dk, "dk", ks), _bf16(dv, "dv", ks), wp, wb,
              B, H, Hkv, N, d, int(bool(causal)), float(scale), _stream(stream)), name)


def fa_exp2_check(x, y_fma, y_ex2, stream=None) -> None:
    """2^x on the FMA pipe (y_fma) and from ex2.approx (y_ex2) for fp32 CUDA x."""
    n = x.numel()
    _check(lib().fa_exp2_check(_f32(x, "x"), _f32(y_fma, "y_fma", tuple(x.shape)),
                               _f32(y_ex2, "y_ex2", tuple(x.shape)), n, _stream(stream)),
           "fa_exp2_check")


def fa_ex2_rate(out, blocks: int, iters: int, stream=None) -> None:
    """One launch of the exponential-unit microbenchmark: blocks x 256 threads,
    8 x iters ex2.approx each; out is an fp32 CUDA tensor of blocks x 256."""
    if out.numel() < int(blocks) * 256:
        raise ValueError(f"out must hold blocks x 256 = {int(blocks) * 256} floats")
    _check(lib().fa_ex2_rate(_f32(out, "out"), int(blocks), int(iters), _stream(stream)),
           "fa_ex2_rate")


def fa_bwd_preprocess_train(o, dout, workspace, Hkv: int, stream=None) -> None:
    """Stage 1 of fa_bwd_train: -D into the workspace fa_fwd_train prepared (o
    bf16, or fp32 from the precise forward)."""
    import torch
    if o.dim() != 4:
        raise ValueError("o must be 4-D [B, H, N, d]")
    B, H, N, d = o.shape
    wp, wb = _ws(workspace)
    if o.dtype == torch.float32:
        fn, op, name = (lib().fa_bwd_preprocess_train_precise, _f32(o, "o"),
                        "fa_bwd_preprocess_train_precise")
    else:
        fn, op, name = lib().fa_bwd_preprocess_train, _bf16(o, "o"), "fa_bwd_preprocess_train"
    _check(fn(op, _bf16(dout, "dout", (B, H, N, d)), wp, wb, B, H, int(Hkv), N, d,
              _stream(stream)), name)


def fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, workspace, window: int, scale: float,
                  stream=None) -> None:
    """Backward of fa_fwd_window."""
    B, H, Hkv, N, d = _dims(q, k)
    window = _c_int(window, "window")
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_window(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _bf16(o, "o", qs),
                               _bf16(dout, "dout", qs), _f32(lse, "lse", ls), _bf16(dq, "dq", qs),
                               _bf16(dk, "dk", ks), _bf16(dv, "dv", ks), wp, wb, B, H, Hkv, N, d,
                               window, float(scale), _stream(stream)), "fa_bwd_window")


def fa_fwd_window_train(q, k, v, o, lse, workspace, window: int, scale: float,
                        stream=None) -> None:
    """fa_fwd_window, plus the backward's workspace prepared for
    fa_bwd_window_train."""
    B, H, Hkv, N, d = _dims(q, k)
    window = _c_int(window, "window")
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    wp, wb = _ws(workspace)
    _check(lib().fa_fwd_window_train(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks),
                                     _bf16(o, "o", qs), _f32(lse, "lse", ls), wp, wb, B, H, Hkv,
                                     N, d, window, float(scale), _stream(stream)),
           "fa_fwd_window_train")


def fa_bwd_window_train(q, k, v, o, dout, dq, dk, dv, workspace, window: int, scale: float,
                        stream=None) -> None:
    """The backward of fa_fwd_window_train, on the workspace it prepared."""
    B, H, Hkv, N, d = _dims(q, k)
    window = _c_int(window, "window")
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_window_train(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks),
                                     _bf16(o, "o", qs), _bf16(dout, "dout", qs),
                                     _bf16(dq, "dq", qs), _bf16(dk, "dk", ks), _bf16(dv, "dv", ks),
                                     wp, wb, B, H, Hkv, N, d, window, float(scale),
                                     _stream(stream)), "fa_bwd_window_train")


def _dims_of(t, name):
    if t.dim() != 4:
        raise ValueError(f"{name} must be 4-D [B, H, N, d]")
    return tuple(t.shape)


def fa_bwd_preprocess(o, dout, lse, workspace, Hkv: int, stream=None) -> None:
    B, H, N, d = _dims_of(o, "o")
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_preprocess(_bf16(o, "o"), _bf16(dout, "dout", (B, H, N, d)),
                                   _f32(lse, "lse", (B, H, N)), wp, wb,
                                   B, H, Hkv, N, d, _stream(stream)), "fa_bwd_preprocess")


def fa_bwd_preprocess_precise(o, dout, lse, workspace, Hkv: int, stream=None) -> None:
    """o: the fp32 output of fa_fwd_precise."""
    B, H, N, d = _dims_of(o, "o")
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_preprocess_precise(_f32(o, "o"), _bf16(dout, "dout", (B, H, N, d)),
                                           _f32(lse, "lse", (B, H, N)),
                                           wp, wb, B, H, Hkv, N, d, _stream(stream)),
           "fa_bwd_preprocess_precise")


def fa_bwd_dkdv(q, k, v, dout, dk, dv, workspace, causal: bool, scale: float,
                stream=None) -> None:
    B, H, Hkv, N, d = _dims(q, k)
    qs, ks, _ = _shapes(B, H, Hkv, N, d)
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_dkdv(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks),
                             _bf16(dout, "dout", qs), _bf16(dk, "dk", ks), _bf16(dv, "dv", ks),
                             wp, wb, B, H, Hkv, N, d,
                             int(bool(causal)), float(scale), _stream(stream)), "fa_bwd_dkdv")


def fa_bwd_dkdv_window(q, k, v, dout, dk, dv, workspace, window: int, scale: float,
                       stream=None) -> None:
    B, H, Hkv, N, d = _dims(q, k)
    window = _c_int(window, "window")
    qs, ks, _ = _shapes(B, H, Hkv, N, d)
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_dkdv_window(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks),
                                    _bf16(dout, "dout", qs), _bf16(dk, "dk", ks),
                                    _bf16(dv, "dv", ks), wp, wb,
                                    B, H, Hkv, N, d, window, float(scale), _stream(stream)),
           "fa_bwd_dkdv_window")


def fa_bwd_dq_convert(workspace, dq, Hkv: int, scale: float, stream=None) -> None:
    B, H, N, d = _dims_of(dq, "dq")
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_dq_convert(wp, wb, _bf16(dq, "dq"), B, H, Hkv, N, d, float(scale),
                                   _stream(stream)), "fa_bwd_dq_convert")


def fa_device_status(stream=None) -> int:
    return int(lib().fa_device_status(_stream(stream)))


def fa_device_status_detail():
    site, block = ctypes.c_int(0), ctypes.c_int(0)
    lib().fa_device_status_detail(ctypes.byref(site), ctypes.byref(block))
    return site.value, block.value


def fa_kernel_launches() -> int:
    return int(lib().fa_kernel_launches())


def fa_watchdog_selftest(timeout_ns: int, stream=None) -> None:
    _check(lib().fa_watchdog_selftest(int(timeout_ns), _stream(stream)), "fa_watchdog_selftest")


# Convenience wrappers that allocate outputs with PyTorch (the library itself
# never allocates).
class _Outputs:
    """Context in which a wrapper allocates for a call on `stream`: memory of that stream, so
    that nothing the current stream still has to do can touch it, and a workspace that the
    wrapper drops is handed out again behind the call.  What it returns goes through `out`:
    the current stream, where the caller may use it, is told to the allocator too."""

    def __init__(self, stream):
        import torch
        self.side = self.ctx = None
        if stream is not None and _stream(stream) != _stream(None):
            self.side = stream if isinstance(stream, torch.cuda.Stream) else \
                torch.cuda.ExternalStream(_stream(stream))

    def __enter__(self):
        import torch
        if self.side is not None:
            self.ctx = torch.cuda.stream(self.side)
            self.ctx.__enter__()
        return self

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)

    def kept(self, workspace):
        """A workspace that may be the caller's: the call's stream is told to the allocator."""
        if self.side is not None:
            workspace.record_stream(self.side)

    def out(self, *tensors):
        import torch
        if self.side is not None:
            for t in tensors:
                t.record_stream(torch.cuda.current_stream())
        return tensors


def fa_fp8_buffer_size(B: int, H: int, Hkv: int, N: int, d: int) -> int:
    return _bytes(lib().fa_fp8_buffer_size, B, H, Hkv, N, d)


def fa_fp8_quantize(v, fp8_buf, H: int, stream=None) -> None:
    """e4m3 codes (transposed) and block scales of v [B, Hkv, N, d] into fp8_buf,
    a contiguous CUDA tensor of at least fa_fp8_buffer_size() bytes; H is the
    number of query heads (checked against Hkv)."""
    B, Hkv, N, d = _dims_of(v, "v")
    bp, bb = _ws(fp8_buf)
    _check(lib().fa_fp8_quantize(_bf16(v, "v"), bp, bb, B, int(H), Hkv, N, d, _stream(stream)),
           "fa_fp8_quantize")


def fa_fwd_fp8(q, k, fp8_buf, o, lse, causal: bool, scale: float, stream=None) -> None:
    """S from the bf16 q, k; P V in e4m3 with V from fp8_buf; o: bf16 [B, H, N, d],
    lse: fp32 [B, H, N]."""
    B, H, Hkv, N, d = _dims(q, k)
    qs, ks, ls = _shapes(B, H, Hkv, N, d)
    bp, bb = _ws(fp8_buf)
    _check(lib().fa_fwd_fp8(_bf16(q, "q"), _bf16(k, "k"), bp, bb, _bf16(o, "o", qs),
                            _f32(lse, "lse", ls), B, H, Hkv, N, d, int(bool(causal)),
                            float(scale), _stream(stream)), "fa_fwd_fp8")


def attention_fp8(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """FP8 forward: quantize V (into a new buffer) and attend; returns (O, LSE, buffer)."""
    import torch
    B, H, Hkv, N, d = _dims(q, k)
    if scale is None:
        scale = d ** -0.5
    n = fa_fp8_buffer_size(B, H, Hkv, N, d)
    if n == 0:
        raise FAError(FA_ERR_UNSUPPORTED, "fa_fp8_buffer_size")
    with _Outputs(stream) as on:
        buf = torch.empty(n, dtype=torch.uint8, device=q.device)
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fp8_quantize(v, buf, H, stream)
    fa_fwd_fp8(q, k, buf, o, lse, causal, scale, stream)
    return on.out(o, lse, buf)


def fa_fwd_decode_workspace_size(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    return _bytes(lib().fa_fwd_decode_workspace_size, B, H, Hkv, Nq, Nk, d)


def fa_fwd_decode(q, k, v, o, lse, workspace, causal: bool, scale: float, stream=None) -> None:
    """q, o: bf16 [B, H, Nq, d]; k, v: bf16 [B, Hkv, Nk, d]; lse: fp32 [B, H, Nq]."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be 4-D")
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != d or v.shape != k.shape:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)} disagree")
    wp, wb = _ws(workspace)
    _check(lib().fa_fwd_decode(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"),
                               _bf16(o, "o", (B, H, Nq, d)), _f32(lse, "lse", (B, H, Nq)),
                               wp, wb, B, H, Hkv, Nq, Nk, d,
                               int(bool(causal)), float(scale), _stream(stream)), "fa_fwd_decode")


def attention_decode(q, k, v, causal: bool = True, scale: float | None = None, stream=None):
    """Decoding forward; allocates the output, LSE and workspace."""
    import torch
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = d ** -0.5
    n = fa_fwd_decode_workspace_size(B, H, Hkv, Nq, Nk, d)
    if n == 0:
        raise FAError(FA_ERR_UNSUPPORTED, "fa_fwd_decode_workspace_size")
    with _Outputs(stream) as on:
        work = torch.empty(n, dtype=torch.uint8, device=q.device)
        o = torch.empty_like(q)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    fa_fwd_decode(q, k, v, o, lse, work, causal, scale, stream)
    return on.out(o, lse)


# ------------------------------------------------------------- paged cache
# A decoding step makes these calls once a layer on little data, so their checks,
# those of _ptr, are spelled out in one expression a call (a function call a tensor
# was a quarter of a small call's time); _explain finds what is wrong.
def _explain(*args):
    for t, name, dtype, shape in args:
        _ptr(t, name, dtype, shape)
    raise ValueError("tensors disagree")


def _pool(k_pages, block_table, kv_scales):
    """Shapes of a paged cache and the type of its pages: k_pages, v_pages [n_pages, Hkv,
    page_size, d] (bf16; torch.float8_e4m3fn with kv_scales fp32 [n_pages, Hkv, 2,
    page_size]), block_table int32 [B, max_pages]."""
    import torch
    pool, table = k_pages.shape, block_table.shape
    if len(pool) != 4:
        raise ValueError("k_pages must be 4-D [n_pages, Hkv, page_size, d]")
    if len(table) != 2:
        raise ValueError("block_table must be 2-D [B, max_pages]")
    return pool, table, torch.bfloat16 if kv_scales is None else torch.float8_e4m3fn


def _scales(kv_scales, pool, cur):
    import torch
    if kv_scales is None:
        return None
    shape = (pool[0], pool[1], 2, pool[2])
    if kv_scales.dtype is torch.float32 and kv_scales.shape == shape and \
            kv_scales.get_device() == cur and kv_scales.is_contiguous():
        return kv_scales.data_ptr()
    return _ptr(kv_scales, "kv_scales", torch.float32, shape)


def _move(call, append, k, v, k_pages, v_pages, block_table, starts, counts, kv_scales, stream,
          max_seqlen=None):
    """fa_kv_append and fa_kv_gather, dense (k [B, Hkv, N, d], counts [B]) or, with max_seqlen,
    packed (k [Hkv, total, d], counts = cu_seqlens [B + 1])."""
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    pool, table, kd = _pool(k_pages, block_table, kv_scales)
    cur = _current_index()
    shape = k.shape
    B = table[0]
    if max_seqlen is None:
        n, good = B, len(shape) == 4 and shape[0] == B
    else:
        n, good = B + 1, len(shape) == 3
    if not good or shape[-3] != pool[1] or shape[-1] != pool[3]:
        raise ValueError(f"k has shape {tuple(shape)}, expected "
                         f"{'[B, Hkv, N, d]' if max_seqlen is None else '[Hkv, total, d]'} of "
                         f"k_pages {tuple(pool)} and block_table {tuple(table)}")
    if not (k.dtype is bf and v.dtype is bf and v.shape == shape and k_pages.dtype is kd and
            v_pages.dtype is kd and v_pages.shape == pool and block_table.dtype is i32 and
            starts.dtype is i32 and starts.shape == (B,) and counts.dtype is i32 and
            counts.shape == (n,) and k.get_device() == cur and v.get_device() == cur and
            k_pages.get_device() == cur and v_pages.get_device() == cur and
            block_table.get_device() == cur and starts.get_device() == cur and
            counts.get_device() == cur and k.is_contiguous() and v.is_contiguous() and
            k_pages.is_contiguous() and v_pages.is_contiguous() and
            block_table.is_contiguous() and starts.is_contiguous() and counts.is_contiguous()):
        _explain((k, "k", bf, shape), (v, "v", bf, shape), (k_pages, "k_pages", kd, pool),
                 (v_pages, "v_pages", kd, pool), (block_table, "block_table", i32, table),
                 (starts, "starts", i32, (B,)),
                 (counts, "counts" if max_seqlen is None else "cu_seqlens", i32, (n,)))
    sp = _scales(kv_scales, pool, cur)
    rows, pages = (k.data_ptr(), v.data_ptr()), (k_pages.data_ptr(), v_pages.data_ptr(), sp)
    sizes = (B, pool[1], shape[2]) if max_seqlen is None else (B, max_seqlen, shape[1], pool[1])
    first, then = (rows, pages) if append else (pages, rows)
    return call(*first, *then, block_table.data_ptr(), starts.data_ptr(), counts.data_ptr(),
                *sizes, pool[0], pool[2], table[1], pool[3], _stream(stream))


def fa_kv_append(k, v, k_pages, v_pages, block_table, starts, counts, kv_scales=None,
                 stream=None) -> None:
    """Rows i < counts[b] of k, v [B, Hkv, N, d] to positions starts[b] + i of sequence b;
    quantised to e4m3 when kv_scales is given.  starts, counts: int32 [B]."""
    _check(_move(lib().fa_kv_append, True, k, v, k_pages, v_pages, block_table, starts, counts,
                 kv_scales, stream), "fa_kv_append")


def fa_kv_append_varlen(k, v, k_pages, v_pages, block_table, starts, cu_seqlens, max_seqlen: int,
                        kv_scales=None, stream=None) -> None:
    """fa_kv_append from a packed batch: k, v [Hkv, total, d], cu_seqlens int32 [B + 1]."""
    _check(_move(lib().fa_kv_append_varlen, True, k, v, k_pages, v_pages, block_table, starts,
                 cu_seqlens, kv_scales, stream, _c_int(max_seqlen, "max_seqlen")),
           "fa_kv_append_varlen")


def fa_kv_gather(k_pages, v_pages, k, v, block_table, starts, counts, kv_scales=None,
                 stream=None) -> None:
    """Positions starts[b] .. starts[b] + counts[b] - 1 of sequence b into rows 0 ..
    counts[b] - 1 of bf16 k, v [B, Hkv, N, d]; the rows behind stay as they are."""
    _check(_move(lib().fa_kv_gather, False, k, v, k_pages, v_pages, block_table, starts, counts,
                 kv_scales, stream), "fa_kv_gather")


def fa_kv_gather_varlen(k_pages, v_pages, k, v, block_table, starts, cu_seqlens, max_seqlen: int,
                        kv_scales=None, stream=None) -> None:
    """fa_kv_gather into a packed batch: k, v [Hkv, total, d], cu_seqlens int32 [B + 1]."""
    _check(_move(lib().fa_kv_gather_varlen, False, k, v, k_pages, v_pages, block_table, starts,
                 cu_seqlens, kv_scales, stream, _c_int(max_seqlen, "max_seqlen")),
           "fa_kv_gather_varlen")


def fa_fwd_decode_paged_workspace_size(B: int, H: int, Hkv: int, Nq: int, d: int) -> int:
    return _bytes(lib().fa_fwd_decode_paged_workspace_size, B, H, Hkv, Nq, d)


def fa_fwd_decode_paged(q, k_pages, v_pages, o, lse, block_table, seqlens, workspace,
                        causal: bool, scale: float, kv_scales=None, stream=None) -> None:
    """q, o: bf16 [B, H, Nq, d]; lse: fp32 [B, H, Nq]; seqlens: int32 [B], the cached
    positions of each sequence, its Nq new ones included."""
    import torch
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    pool, table, kd = _pool(k_pages, block_table, kv_scales)
    cur = _current_index()
    qs = q.shape
    if len(qs) != 4:
        raise ValueError("q must be 4-D [B, H, Nq, d]")
    B, H, Nq, d = qs
    if pool[3] != d or table[0] != B:
        raise ValueError(f"q {tuple(qs)}, k_pages {tuple(pool)} and block_table {tuple(table)} "
                         "disagree")
    if not (q.dtype is bf and o.dtype is bf and o.shape == qs and lse.dtype is f32 and
            lse.shape == (B, H, Nq) and k_pages.dtype is kd and v_pages.dtype is kd and
            v_pages.shape == pool and block_table.dtype is i32 and seqlens.dtype is i32 and
            seqlens.shape == (B,) and q.get_device() == cur and o.get_device() == cur and
            lse.get_device() == cur and k_pages.get_device() == cur and
            v_pages.get_device() == cur and block_table.get_device() == cur and
            seqlens.get_device() == cur and q.is_contiguous() and o.is_contiguous() and
            lse.is_contiguous() and k_pages.is_contiguous() and v_pages.is_contiguous() and
            block_table.is_contiguous() and seqlens.is_contiguous()):
        _explain((q, "q", bf, qs), (k_pages, "k_pages", kd, pool), (v_pages, "v_pages", kd, pool),
                 (o, "o", bf, qs), (lse, "lse", f32, (B, H, Nq)),
                 (block_table, "block_table", i32, table), (seqlens, "seqlens", i32, (B,)))
    sp = _scales(kv_scales, pool, cur)
    if workspace.get_device() == cur and workspace.is_contiguous():
        wp, wb = workspace.data_ptr(), workspace.nbytes
    else:
        wp, wb = _ws(workspace)
    _check(lib().fa_fwd_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), sp,
                                     o.data_ptr(), lse.data_ptr(), block_table.data_ptr(),
                                     seqlens.data_ptr(), wp, wb, B, H, pool[1], Nq, pool[0],
                                     pool[2], table[1], d, 1 if causal else 0, float(scale),
                                     _stream(stream)), "fa_fwd_decode_paged")


def attention_decode_paged(q, k_pages, v_pages, block_table, seqlens, causal: bool = True,
                           scale: float | None = None, kv_scales=None, workspace=None,
                           stream=None):
    """Decoding over a paged cache; allocates the output and LSE, and the workspace unless it
    is given; returns (o, lse)."""
    import torch
    B, H, Nq, d = _dims_of(q, "q")
    pool, _, _ = _pool(k_pages, block_table, kv_scales)
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        if workspace is None:
            n = fa_fwd_decode_paged_workspace_size(B, H, pool[1], Nq, d)
            if n == 0:
                raise FAError(FA_ERR_UNSUPPORTED, "fa_fwd_decode_paged_workspace_size")
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    fa_fwd_decode_paged(q, k_pages, v_pages, o, lse, block_table, seqlens, workspace, causal,
                        scale, kv_scales, stream)
    if on.side is not None:
        workspace.record_stream(on.side)       # the caller's, if it is given
    return on.out(o, lse)


# --------------------------------------------- block tables and slot maps
def _all_i32(*args):
    """Pointers of int32 tensors, (tensor, name, shape) each."""
    return [_i32(t, name, shape) for t, name, shape in args]


def _map(positions, slots, shape):
    import torch
    return _i32(positions, "positions", shape), _ptr(slots, "slots", torch.int64, shape)


def _table(block_table):
    if block_table.dim() != 2:
        raise ValueError("block_table must be 2-D [B, max_pages]")
    return block_table.shape


def fa_kv_reserve(block_table, seqlens, free_pages, n_free, new_tokens, starts, counts,
                  cu_seqlens, page_size: int, positions=None, slots=None, stream=None) -> None:
    """Room for new_tokens [B] more tokens a sequence: block_table [B, max_pages], seqlens [B],
    free_pages [n_pages] and n_free [1] in place; starts, counts [B] and cu_seqlens [B + 1]
    written; positions, slots (int64) [B, N] or packed [total]: the new tokens' map.  All
    int32 but slots."""
    if _done(binding().kv_reserve(block_table, seqlens, free_pages, n_free, new_tokens, starts,
                                  counts, cu_seqlens, positions, slots, page_size,
                                  _handle(stream)), "fa_kv_reserve"):
        return
    B, mp = table = _table(block_table)
    one = (B,)
    n_pages = free_pages.numel()
    ptrs = _all_i32((block_table, "block_table", table), (seqlens, "seqlens", one),
                          (free_pages, "free_pages", (n_pages,)), (n_free, "n_free", (1,)),
                          (new_tokens, "new_tokens", one), (starts, "starts", one),
                          (counts, "counts", one), (cu_seqlens, "cu_seqlens", (B + 1,)))
    N, total, at = 0, 0, (None, None)
    if positions is not None or slots is not None:
        if positions is None or slots is None:
            raise ValueError("positions and slots come together")
        shape = slots.shape
        if len(shape) == 2:
            N, shape = shape[1], (B, shape[1])
            if N < 1:
                raise ValueError("slots has no rows")
        else:
            total, shape = slots.numel(), (slots.numel(),)
        at = _map(positions, slots, shape)
    _check(lib().fa_kv_reserve(*ptrs, *at, B, N, total, n_pages, _c_int(page_size, "page_size"),
                               mp, _stream(stream)), "fa_kv_reserve")


def fa_kv_release(block_table, seqlens, free_pages, n_free, keep, page_size: int, pinned=None,
                  stream=None) -> None:
    """Every sequence cut back to its first keep [B] tokens, the pages behind them free again
    (but for the first pinned [B] pages of each, if given)."""
    if _done(binding().kv_release(block_table, seqlens, free_pages, n_free, keep, pinned, page_size,
                                  _handle(stream)), "fa_kv_release"):
        return
    B, mp = table = _table(block_table)
    one = (B,)
    n_pages = free_pages.numel()
    ptrs = _all_i32((block_table, "block_table", table), (seqlens, "seqlens", one),
                          (free_pages, "free_pages", (n_pages,)), (n_free, "n_free", (1,)),
                          (keep, "keep", one),
                    *(() if pinned is None else ((pinned, "pinned", one),)))
    if pinned is None:
        ptrs.append(None)
    _check(lib().fa_kv_release(*ptrs, B, n_pages, _c_int(page_size, "page_size"), mp,
                               _stream(stream)), "fa_kv_release")


def fa_kv_slots(block_table, starts, counts, positions, slots, page_size: int,
                stream=None) -> None:
    """Positions and slots [B, N] of rows i < counts[b] at positions starts[b] + i."""
    B, mp = table = _table(block_table)
    ptrs = _all_i32((block_table, "block_table", table), (starts, "starts", (B,)),
                    (counts, "counts", (B,)))
    if slots.dim() != 2:
        raise ValueError("slots must be 2-D [B, N]")
    N = slots.shape[1]
    at = _map(positions, slots, (B, N))
    _check(lib().fa_kv_slots(*ptrs, *at, B, N, _c_int(page_size, "page_size"), mp,
                             _stream(stream)), "fa_kv_slots")


def fa_kv_slots_varlen(block_table, starts, cu_seqlens, positions, slots, page_size: int,
                       stream=None) -> None:
    """The same of a packed batch: positions, slots [total], cu_seqlens [B + 1]."""
    B, mp = table = _table(block_table)
    ptrs = _all_i32((block_table, "block_table", table), (starts, "starts", (B,)),
                    (cu_seqlens, "cu_seqlens", (B + 1,)))
    if slots.dim() != 1:
        raise ValueError("slots must be 1-D [total]")
    at = _map(positions, slots, slots.shape)
    _check(lib().fa_kv_slots_varlen(*ptrs, *at, B, slots.numel(), _c_int(page_size, "page_size"),
                                    mp, _stream(stream)), "fa_kv_slots_varlen")


# ------------------------------------------------------- rotary positions
_SCALINGS = {None: 0, "none": 0, "linear": 1, "ntk": 2, "parts": 3}


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None,
                     factor: float = 1.0, original_length: int = 0, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, device=None):
    """(freqs, amplitude) for fa_rope and fa_rope_append: an int64 tensor [rot / 2] on `device`
    (default: the current CUDA device) and a number, from fa_rope_freqs.  scaling: "linear",
    "ntk" or "parts"."""
    import torch
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(k for k in _SCALINGS if k)}")
    rot = _c_int(rot, "rot")
    freqs = torch.zeros(max(rot // 2, 1), dtype=torch.int64)
    amplitude = ctypes.c_float()
    _check(lib().fa_rope_freqs(freqs.data_ptr(), ctypes.byref(amplitude), rot, float(base),
                               _SCALINGS[scaling], float(factor),
                               _c_int(original_length, "original_length"), float(beta_fast),
                               float(beta_slow)), "fa_rope_freqs")
    return freqs.to("cuda" if device is None else device), amplitude.value


_STRIDES = ctypes.c_longlong * 12


def _rows(t, name, shape):
    """Device pointer and strides of rows t, contiguous each."""
    import torch
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != torch.bfloat16 or not t.is_cuda or t.stride(3) != 1:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor with contiguous rows")
    _on_current_device(t, name)
    return t.data_ptr(), t.stride()[:3]


def _rope_args(q, positions, freqs):
    """B, H, N, d, rot of a call, and the pointers of positions and freqs."""
    import torch
    B, H, N, d = _dims_of(q, "q")
    return (B, H, N, d, 2 * freqs.numel(), _i32(positions, "positions", (B, N)),
            _ptr(freqs, "freqs", torch.int64, (freqs.numel(),)))


def fa_rope(q, k, q_out, k_out, positions, freqs, interleaved: bool = False,
            inverse: bool = False, amplitude: float = 1.0, stream=None) -> None:
    """q [B, H, N, d] and k [B, Hkv, N, d] (or None, with k_out) turned by their positions
    int32 [B, N] into q_out and k_out; any strides over B, H and N.  freqs, amplitude: from
    rope_frequencies; inverse: for gradients."""
    if _done(binding().rope(q, k, q_out, k_out, positions, freqs, interleaved, inverse, amplitude,
                            _handle(stream)), "fa_rope"):
        return
    B, H, N, d, rot, pp, fp = _rope_args(q, positions, freqs)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out come together")
    (qp, qs), (qop, qos) = _rows(q, "q", q.shape), _rows(q_out, "q_out", q.shape)
    Hkv, kp, kop, ks, kos = 0, None, None, (0, 0, 0), (0, 0, 0)
    if k is not None:
        Hkv = _dims_of(k, "k")[1]
        (kp, ks), (kop, kos) = (_rows(t, n, (B, Hkv, N, d)) for t, n in ((k, "k"), (k_out, "k_out")))
    strides = _STRIDES(*qs, *ks, *qos, *kos)
    _check(lib().fa_rope(qp, kp, qop, kop, pp, fp, strides, B, H, Hkv, N, d, rot,
                         1 if interleaved else 0, 1 if inverse else 0, float(amplitude),
                         _stream(stream)), "fa_rope")


def rope(q, k, positions, freqs, interleaved: bool = False, inverse: bool = False,
         amplitude: float = 1.0, stream=None):
    """fa_rope into new contiguous tensors; returns (q_out, k_out)."""
    import torch
    with _Outputs(stream) as on:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
    fa_rope(q, k, q_out, k_out, positions, freqs, interleaved, inverse, amplitude, stream)
    on.out(*(t for t in (q_out, k_out) if t is not None))
    return q_out, k_out


def fa_rope_append(q, k, v, q_out, k_pages, v_pages, positions, slots, freqs,
                   interleaved: bool = False, amplitude: float = 1.0, kv_scales=None,
                   stream=None) -> None:
    """q [B, H, N, d] turned into q_out; k [B, Hkv, N, d] turned, and v, into the pages at
    slots int64 [B, N] (negative: not written); a packed batch is B = 1.  Any strides over
    B, H and N of q, k, v and q_out."""
    if _done(binding().rope_append(q, k, v, q_out, k_pages, v_pages, positions, slots, freqs,
                                   interleaved, amplitude, kv_scales, _handle(stream)),
             "fa_rope_append"):
        return
    import torch
    B, H, N, d, rot, pp, fp = _rope_args(q, positions, freqs)
    pool = k_pages.shape
    if len(pool) != 4 or pool[3] != d:
        raise ValueError(f"k_pages must be 4-D [n_pages, Hkv, page_size, {d}]")
    kd = torch.bfloat16 if kv_scales is None else torch.float8_e4m3fn
    kv = (B, pool[1], N, d)
    rows = [_rows(*x) for x in ((q, "q", q.shape), (k, "k", kv), (v, "v", kv),
                                (q_out, "q_out", q.shape))]
    strides = _STRIDES(*(x for _, s in rows for x in s))
    _check(lib().fa_rope_append(*(x for x, _ in rows), _ptr(k_pages, "k_pages", kd, pool),
                                _ptr(v_pages, "v_pages", kd, pool),
                                _scales(kv_scales, pool, _current_index()), pp,
                                _ptr(slots, "slots", torch.int64, (B, N)), fp, strides, B, H,
                                pool[1], N, pool[0], pool[2], d, rot, 1 if interleaved else 0,
                                float(amplitude), _stream(stream)), "fa_rope_append")


# --------------------------------------- queries and keys of two lengths
def fa_fwd_cross_workspace_size(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    return _bytes(lib().fa_fwd_cross_workspace_size, B, H, Hkv, Nq, Nk, d)


def fa_bwd_cross_workspace_size(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    return _bytes(lib().fa_bwd_cross_workspace_size, B, H, Hkv, Nq, Nk, d)


def fa_fwd_cross_decode_workspace_size(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    return _bytes(lib().fa_fwd_cross_decode_workspace_size, B, H, Hkv, Nq, Nk, d)


def _cross_dims(q, k, kv_lens):
    """Shapes of the query side, the key side and lse; B, H, Hkv, Nq, Nk, d; kv_lens' pointer."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be 4-D [B, H(kv), N, d]")
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree")
    lens = None if kv_lens is None else _i32(kv_lens, "kv_lens", (B,))
    return (B, H, Nq, d), (B, Hkv, Nk, d), (B, H, Nq), (B, H, Hkv, Nq, Nk, d), lens


def _cross_varlen_dims(q, k, cu_q, cu_k, max_q, max_k):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("packed q and k must be 3-D [H(kv), total, d]")
    if cu_q.dim() != 1 or cu_k.shape != cu_q.shape:
        raise ValueError("cu_q and cu_k must be 1-D [B + 1]")
    H, total_q, d = q.shape
    Hkv, total_k, dk = k.shape
    if dk != d:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree")
    sizes = (cu_q.numel() - 1, _c_int(max_q, "max_q"), _c_int(max_k, "max_k"), total_q, total_k, H,
             Hkv, d)
    return (H, total_q, d), (Hkv, total_k, d), (H, total_q), sizes, \
        (_i32(cu_q, "cu_q"), _i32(cu_k, "cu_k"))


def fa_fwd_cross(q, k, v, o, lse, workspace, causal: bool, scale: float, kv_lens=None,
                 stream=None) -> None:
    """q, o: bf16 [B, H, Nq, d]; k, v: bf16 [B, Hkv, Nk, d]; lse: fp32 [B, H, Nq]; kv_lens:
    int32 [B], the keys of each sequence (default: Nk)."""
    if _done(binding().cross_forward(q, k, v, o, lse, workspace, causal, scale, kv_lens,
                                     _handle(stream)), "fa_fwd_cross"):
        return
    qs, ks, ls, sizes, lens = _cross_dims(q, k, kv_lens)
    wp, wb = _ws(workspace)
    _check(lib().fa_fwd_cross(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _bf16(o, "o", qs),
                              _f32(lse, "lse", ls), lens, wp, wb, *sizes, int(bool(causal)),
                              float(scale), _stream(stream)), "fa_fwd_cross")


def fa_bwd_cross(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal: bool, scale: float,
                 kv_lens=None, stream=None) -> None:
    """The gradients of fa_fwd_cross."""
    if _done(binding().cross_backward(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal, scale,
                                      kv_lens, _handle(stream)), "fa_bwd_cross"):
        return
    qs, ks, ls, sizes, lens = _cross_dims(q, k, kv_lens)
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_cross(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks), _bf16(o, "o", qs),
                              _bf16(dout, "dout", qs), _f32(lse, "lse", ls), _bf16(dq, "dq", qs),
                              _bf16(dk, "dk", ks), _bf16(dv, "dv", ks), lens, wp, wb, *sizes,
                              int(bool(causal)), float(scale), _stream(stream)), "fa_bwd_cross")


def fa_fwd_cross_varlen(q, k, v, o, lse, workspace, cu_q, cu_k, max_q: int, max_k: int,
                        causal: bool, scale: float, stream=None) -> None:
    """Packed: q, o [H, total_q, d], k, v [Hkv, total_k, d], lse [H, total_q]; cu_q, cu_k int32
    [B + 1]."""
    if _done(binding().cross_forward_varlen(q, k, v, o, lse, workspace, causal, scale, cu_q, cu_k,
                                            max_q, max_k, _handle(stream)), "fa_fwd_cross_varlen"):
        return
    qs, ks, ls, sizes, cu = _cross_varlen_dims(q, k, cu_q, cu_k, max_q, max_k)
    wp, wb = _ws(workspace)
    _check(lib().fa_fwd_cross_varlen(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks),
                                     _bf16(o, "o", qs), _f32(lse, "lse", ls), *cu, wp, wb, *sizes,
                                     int(bool(causal)), float(scale), _stream(stream)),
           "fa_fwd_cross_varlen")


def fa_bwd_cross_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_q, cu_k, max_q: int,
                        max_k: int, causal: bool, scale: float, stream=None) -> None:
    """The gradients of fa_fwd_cross_varlen."""
    if _done(binding().cross_backward_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal,
                                             scale, cu_q, cu_k, max_q, max_k, _handle(stream)),
             "fa_bwd_cross_varlen"):
        return
    qs, ks, ls, sizes, cu = _cross_varlen_dims(q, k, cu_q, cu_k, max_q, max_k)
    wp, wb = _ws(workspace)
    _check(lib().fa_bwd_cross_varlen(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks),
                                     _bf16(o, "o", qs), _bf16(dout, "dout", qs),
                                     _f32(lse, "lse", ls), _bf16(dq, "dq", qs),
                                     _bf16(dk, "dk", ks), _bf16(dv, "dv", ks), *cu, wp, wb, *sizes,
                                     int(bool(causal)), float(scale), _stream(stream)),
           "fa_bwd_cross_varlen")


def fa_fwd_cross_decode(q, k, v, o, lse, workspace, causal: bool, scale: float, kv_lens=None,
                        stream=None) -> None:
    """fa_fwd_cross for a few queries a sequence, (H / Hkv) * Nq <= 32."""
    if _done(binding().cross_decode(q, k, v, o, lse, workspace, causal, scale, kv_lens,
                                    _handle(stream)), "fa_fwd_cross_decode"):
        return
    qs, ks, ls, sizes, lens = _cross_dims(q, k, kv_lens)
    wp, wb = _ws(workspace)
    _check(lib().fa_fwd_cross_decode(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v", ks),
                                     _bf16(o, "o", qs), _f32(lse, "lse", ls), lens, wp, wb, *sizes,
                                     int(bool(causal)), float(scale), _stream(stream)),
           "fa_fwd_cross_decode")


def _workspace_of(size_of, where, *sizes):
    import torch
    n = size_of(*sizes)
    if n == 0:
        raise FAError(FA_ERR_UNSUPPORTED, where)
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def attention_cross(q, k, v, kv_lens=None, causal: bool = False, scale: float | None = None,
                    workspace=None, stream=None):
    """Attention of q [B, H, Nq, d] to k, v [B, Hkv, Nk, d]; returns (o, lse)."""
    import torch
    B, H, Nq, d = _dims_of(q, "q")
    _, Hkv, Nk, _ = _dims_of(k, "k")
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = _workspace_of(fa_fwd_cross_workspace_size, "fa_fwd_cross_workspace_size",
                                      B, H, Hkv, Nq, Nk, d)
    fa_fwd_cross(q, k, v, o, lse, workspace, causal, scale, kv_lens, stream)
    on.kept(workspace)
    return on.out(o, lse)


def attention_cross_backward(q, k, v, o, lse, dout, kv_lens=None, causal: bool = False,
                             scale: float | None = None, workspace=None, stream=None):
    """Returns (dq, dk, dv) for attention_cross."""
    import torch
    B, H, Nq, d = _dims_of(q, "q")
    _, Hkv, Nk, _ = _dims_of(k, "k")
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        if workspace is None:
            workspace = _workspace_of(fa_bwd_cross_workspace_size, "fa_bwd_cross_workspace_size",
                                      B, H, Hkv, Nq, Nk, d)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd_cross(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal, scale, kv_lens, stream)
    on.kept(workspace)
    return on.out(dq, dk, dv)


def attention_cross_varlen(q, k, v, cu_q, cu_k, max_q: int, max_k: int, causal: bool = False,
                           scale: float | None = None, workspace=None, stream=None):
    """Packed: q [H, total_q, d], k, v [Hkv, total_k, d]; returns (o, lse [H, total_q])."""
    import torch
    _, _, _, sizes, _ = _cross_varlen_dims(q, k, cu_q, cu_k, max_q, max_k)
    B, mq, mk, _, _, H, Hkv, d = sizes
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = _workspace_of(fa_fwd_cross_workspace_size, "fa_fwd_cross_workspace_size",
                                      B, H, Hkv, mq, mk, d)
    fa_fwd_cross_varlen(q, k, v, o, lse, workspace, cu_q, cu_k, max_q, max_k, causal, scale, stream)
    on.kept(workspace)
    return on.out(o, lse)


def attention_cross_varlen_backward(q, k, v, o, lse, dout, cu_q, cu_k, max_q: int, max_k: int,
                                    causal: bool = False, scale: float | None = None,
                                    workspace=None, stream=None):
    """Returns (dq, dk, dv) for attention_cross_varlen."""
    import torch
    _, _, _, sizes, _ = _cross_varlen_dims(q, k, cu_q, cu_k, max_q, max_k)
    B, mq, mk, _, _, H, Hkv, d = sizes
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        if workspace is None:
            workspace = _workspace_of(fa_bwd_cross_workspace_size, "fa_bwd_cross_workspace_size",
                                      B, H, Hkv, mq, mk, d)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd_cross_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_q, cu_k, max_q, max_k,
                        causal, scale, stream)
    on.kept(workspace)
    return on.out(dq, dk, dv)


def attention_cross_decode(q, k, v, kv_lens=None, causal: bool = False, scale: float | None = None,
                           workspace=None, stream=None):
    """attention_cross for a few queries a sequence; returns (o, lse)."""
    import torch
    B, H, Nq, d = _dims_of(q, "q")
    _, Hkv, Nk, _ = _dims_of(k, "k")
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = _workspace_of(fa_fwd_cross_decode_workspace_size,
                                      "fa_fwd_cross_decode_workspace_size", B, H, Hkv, Nq, Nk, d)
    fa_fwd_cross_decode(q, k, v, o, lse, workspace, causal, scale, kv_lens, stream)
    on.kept(workspace)
    return on.out(o, lse)


def attention(q, k, v, causal: bool = False, scale: float | None = None, stream=None,
              precise: bool = False):
    """Returns (o, lse) for bf16 CUDA q [B,H,N,d], k/v [B,Hkv,N,d]; o is bf16, or
    fp32 from fa_fwd_precise when precise=True."""
    import torch
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        o = torch.empty(q.shape, dtype=torch.float32, device=q.device) if precise else \
            torch.empty_like(q)
    (fa_fwd_precise if precise else fa_fwd)(q, k, v, o, lse, causal, scale, stream)
    return on.out(o, lse)


def attention_window(q, k, v, window: int, scale: float | None = None, stream=None):
    """Causal sliding-window attention (query i sees keys i - window < j <= i);
    returns (o, lse)."""
    import torch
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        o = torch.empty_like(q)
    fa_fwd_window(q, k, v, o, lse, window, scale, stream)
    return on.out(o, lse)


def attention_window_backward(q, k, v, o, lse, dout, window: int, scale: float | None = None,
                              workspace=None, stream=None):
    """Returns (dq, dk, dv) for attention_window."""
    import torch
    B, H, Hkv, N, d = _dims(q, k)
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        if workspace is None:
            workspace = torch.empty(fa_bwd_workspace_size(B, H, Hkv, N, d), dtype=torch.uint8,
                                    device=q.device)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, workspace, window, scale, stream)
    return on.out(dq, dk, dv)


def attention_varlen(q, k, v, cu_seqlens, max_seqlen: int, causal: bool = False,
                     scale: float | None = None, stream=None):
    """Packed variable-length sequences; returns (o [H, total, d], lse [H, total])."""
    import torch
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, max_seqlen, causal, scale, stream)
    return on.out(o, lse)


def attention_varlen_backward(q, k, v, o, lse, dout, cu_seqlens, max_seqlen: int,
                              causal: bool = False, scale: float | None = None, workspace=None,
                              stream=None):
    """Returns (dq, dk, dv) for attention_varlen."""
    import torch
    B, H, Hkv, total, d = _varlen_dims(q, k, cu_seqlens)
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        if workspace is None:
            workspace = torch.empty(fa_bwd_varlen_workspace_size(B, H, Hkv, max_seqlen, d),
                                    dtype=torch.uint8, device=q.device)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens, max_seqlen, causal,
                  scale, stream)
    return on.out(dq, dk, dv)


def attention_backward(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None,
                       workspace=None, stream=None):
    """Returns (dq, dk, dv)."""
    import torch
    B, H, Hkv, N, d = _dims(q, k)
    scale = d ** -0.5 if scale is None else scale
    with _Outputs(stream) as on:
        if workspace is None:
            workspace = torch.empty(fa_bwd_workspace_size(B, H, Hkv, N, d), dtype=torch.uint8,
                                    device=q.device)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if o.dtype == torch.float32:
        fa_bwd_precise(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal, scale, stream)
    else:
        fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal, scale, stream)
    return on.out(dq, dk, dv)
