"""ctypes binding of libfa8.so (include/fa8.h): argument marshalling only.

Every step of the attention runs in the library's CUDA kernels.  This module turns torch
tensors into ``fa8_tensor`` views, allocates outputs and the split-KV workspace with torch
(device memory is the only thing torch provides here), and raises ``Fa8Error`` on any
non-zero status.  There is no fallback: if the library is missing or fails to load, every
call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

from .build import args_path

_HERE = os.path.dirname(os.path.abspath(__file__))
# FA8_LIBRARY may point at another build of the same library (e.g. one with FA8_TRACE)
LIB_PATH = os.environ.get("FA8_LIBRARY") or os.path.join(_HERE, "_build", "libfa8.so")

FA8_SUCCESS = 0
FA8_ERR_INVALID_ARG = 1
FA8_ERR_UNSUPPORTED = 2
FA8_ERR_WORKSPACE = 3
FA8_ERR_CUDA = 4
FA8_ERR_DEVICE_TIMEOUT = 5
FA8_ERR_DEVICE_BOUNDS = 6

_DTYPES = {
    torch.float8_e4m3fn: 1,
    torch.float8_e5m2: 2,
    torch.bfloat16: 3,
    torch.float16: 4,
    torch.float32: 5,
    torch.int32: 6,
    torch.float64: 7,
}

# name -> (restype, argtypes); every function declared in include/fa8.h
_T = None  # filled after the struct is defined


class Fa8Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


_P = ctypes.POINTER(Fa8Tensor)
SIGNATURES = {
    "fa8_fwd": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int,
                               ctypes.c_int, _P, ctypes.c_float, ctypes.c_int, ctypes.c_void_p,
                               ctypes.c_size_t, ctypes.c_void_p]),
    "fa8_fwd_workspace_size": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int,
                                              ctypes.POINTER(ctypes.c_int),
                                              ctypes.POINTER(ctypes.c_size_t)]),
    "fa8_fwd_plan": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                    ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_size_t),
                                    ctypes.POINTER(ctypes.c_int64)]),
    "fa8_fwd_static_scratch": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int,
                                              ctypes.c_int, ctypes.c_int, _P, ctypes.c_float, ctypes.c_int,
                                              ctypes.c_void_p]),
    "fa8_rope_inv_freq": (ctypes.c_int, [ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_double,
                                         ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                         ctypes.POINTER(ctypes.c_double)]),
    "fa8_rope_append": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_float, _P, _P, _P,
                                       _P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_void_p]),
    "fa8_page_bounds": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "fa8_select_pages": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_void_p]),
    "fa8_fwd_pages": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int, _P,
                                     ctypes.c_float, ctypes.c_void_p]),
    "fa8_fwd_scored": (ctypes.c_int, [_P] * 11 + [ctypes.c_int] * 3 + [_P, _P, ctypes.c_float, _P, ctypes.c_float,
                                      ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "fa8_fwd_scored_workspace_size": (ctypes.c_int, [_P] * 6 + [ctypes.c_int, _P, ctypes.POINTER(ctypes.c_size_t)]),
    "fa8_fwd_tree": (ctypes.c_int, [_P] * 12 + [ctypes.c_int, ctypes.c_float, _P, ctypes.c_float, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]),
    "fa8_tree_masks": (ctypes.c_int, [_P] * 5 + [ctypes.c_void_p]),
    "fa8_keep_tokens": (ctypes.c_int, [_P] * 6 + [ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "fa8_check": (ctypes.c_int, [ctypes.c_void_p]),
    "fa8_set_wait_timeout_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "fa8_set_decode_kernel": (ctypes.c_int, [ctypes.c_int]),
    "fa8_debug_wait_probe": (ctypes.c_int, [ctypes.c_void_p]),
    "fa8_debug_set_trace_buffer": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t]),
    "fa8_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fa8_last_error": (ctypes.c_char_p, []),
    "fa8_version": (ctypes.c_int, []),
}

_lib = None


class Fa8Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"fa8 status {status}: {msg}")
        self.status = status


def lib():
    """Loads libfa8.so (built by ``fp8_attention_forward_gb300.build``); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfa8.so not built ({LIB_PATH}); run fp8_attention_forward_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _view(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    if t.dim() > 4:
        raise ValueError("at most 4 dims")
    v = Fa8Tensor()
    v.data = t.data_ptr()
    v.dtype = _DTYPES[t.dtype]
    v.ndim = t.dim()
    for i in range(t.dim()):
        v.shape[i] = t.shape[i]
        v.stride[i] = t.stride(i)
    return v


def _ref(v):
    return None if v is None else ctypes.byref(v)


def _raise(st: int):
    if st != FA8_SUCCESS:
        raise Fa8Error(st, lib().fa8_last_error().decode())


def _on_device(device):
    """Makes ``device`` current for the library call: the library plans for, and looks up its
    per-device state on, the current CUDA device."""
    import contextlib

    if device.type != "cuda":
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def plan(q, k, v, *, cu_seqlens_q=None, cu_seqlens_k=None, block_table=None, page_size=0,
         num_splits=0, sm_count=None):
    """(splits, workspace_bytes, grid) chosen for these shapes; host-only when sm_count is given."""
    views = [_view(x) for x in (q, k, v, cu_seqlens_q, cu_seqlens_k, block_table)]
    splits = ctypes.c_int(0)
    nbytes = ctypes.c_size_t(0)
    if sm_count is None:
        with _on_device(q.device):
            st = lib().fa8_fwd_workspace_size(*[_ref(x) for x in views], int(page_size), int(num_splits),
                                              ctypes.byref(splits), ctypes.byref(nbytes))
        _raise(st)
        return splits.value, nbytes.value, None
    grid = (ctypes.c_int64 * 2)()
    st = lib().fa8_fwd_plan(*[_ref(x) for x in views], int(page_size), int(num_splits), int(sm_count),
                            ctypes.byref(splits), ctypes.byref(nbytes), grid)
    _raise(st)
    return splits.value, nbytes.value, (grid[0], grid[1])


def fwd(q, k, v, *, descale_q=None, descale_k=None, descale_v=None, out=None, lse=None,
        cu_seqlens_q=None, cu_seqlens_k=None, block_table=None, page_size=0, causal=False,
        window_left=-1, sink=None, softmax_scale=0.0, num_splits=0, workspace=None,
        out_dtype=torch.bfloat16, return_lse=True, stream=None):
    """Fused FP8 attention forward; returns (out, lse).  See include/fa8.h for layouts."""
    dev = q.device
    dv = v.shape[-1]
    if out is None:
        out = torch.empty(tuple(q.shape[:-1]) + (dv,), dtype=out_dtype, device=dev)
    if lse is None and return_lse:
        if q.dim() == 4:
            lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=dev)
        else:
            lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=dev)
    if workspace is None:
        _, nbytes, _ = plan(q, k, v, cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k,
                            block_table=block_table, page_size=page_size, num_splits=num_splits)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev) if nbytes else None
    views = dict(q=_view(q), k=_view(k), v=_view(v), dq=_view(descale_q), dk=_view(descale_k),
                 dv=_view(descale_v), out=_view(out), lse=_view(lse), cq=_view(cu_seqlens_q),
                 ck=_view(cu_seqlens_k), bt=_view(block_table), sink=_view(sink))
    ws_ptr = ctypes.c_void_p(workspace.data_ptr() if workspace is not None else 0)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    with _on_device(dev):
        st = lib().fa8_fwd(_ref(views["q"]), _ref(views["k"]), _ref(views["v"]), _ref(views["dq"]),
                           _ref(views["dk"]), _ref(views["dv"]), _ref(views["out"]), _ref(views["lse"]),
                           _ref(views["cq"]), _ref(views["ck"]), _ref(views["bt"]), int(page_size),
                           int(bool(causal)), int(window_left), _ref(views["sink"]), float(softmax_scale),
                           int(num_splits), ws_ptr, ws_bytes,
                           _stream_handle(stream, dev) if dev.type == "cuda" else ctypes.c_void_p(0))
    _raise(st)
    return out, lse


STATIC_SCRATCH_BYTES = 32 * 1024 * 1024  # FA8_STATIC_SCRATCH_BYTES in include/fa8.h (a CPU test compares them)


def fwd_static_scratch(q, k, v, *, out, lse=None, descale_q=None, descale_k=None, descale_v=None,
                       cu_seqlens_q=None, cu_seqlens_k=None, block_table=None, page_size=0, causal=False,
                       window_left=-1, sink=None, softmax_scale=0.0, num_splits=0, stream=None):
    """``fa8_fwd_static_scratch``: the forward with split partials in the library's static
    device scratch.  ``out`` (and ``lse`` if wanted) are caller-provided; nothing is allocated."""
    views = dict(q=_view(q), k=_view(k), v=_view(v), dq=_view(descale_q), dk=_view(descale_k),
                 dv=_view(descale_v), out=_view(out), lse=_view(lse), cq=_view(cu_seqlens_q),
                 ck=_view(cu_seqlens_k), bt=_view(block_table), sink=_view(sink))
    with _on_device(q.device):
        st = lib().fa8_fwd_static_scratch(_ref(views["q"]), _ref(views["k"]), _ref(views["v"]),
                                          _ref(views["dq"]), _ref(views["dk"]), _ref(views["dv"]),
                                          _ref(views["out"]), _ref(views["lse"]), _ref(views["cq"]),
                                          _ref(views["ck"]), _ref(views["bt"]), int(page_size), int(bool(causal)),
                                          int(window_left), _ref(views["sink"]), float(softmax_scale),
                                          int(num_splits), _stream_handle(stream, q.device))
    _raise(st)
    return out, lse


# ------------------------------------------------------------------ around the paged cache
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}  # fa8_rope_scaling


def rope_inv_freq(rotary_dim, base=10000.0, *, scaling="none", factor=1.0, original_len=0.0, low=1.0,
                  high=None, device="cpu"):
    """The rotary_dim / 2 frequencies (fp64) that ``rope_append`` takes, stretched for long
    contexts as ``fa8_rope_scaling`` in include/fa8.h says."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    if high is None:
        high = 4.0 if scaling == "bands" else 32.0
    out = torch.empty(max(int(rotary_dim), 0) // 2, dtype=torch.float64)
    _raise(lib().fa8_rope_inv_freq(int(rotary_dim), float(base), ROPE_SCALINGS[scaling], float(factor),
                                   float(original_len), float(low), float(high),
                                   ctypes.cast(out.data_ptr(), ctypes.POINTER(ctypes.c_double))))
    return out.to(device)


_ARG = [struct.Struct("Qii%dq%dx%dq%dx" % (n, 32 - 8 * n, n, 32 - 8 * n)) for n in range(5)]  # fa8_tensor of n dims
_ARGS = ctypes.c_char * (ctypes.sizeof(Fa8Tensor) * 16)
_SCALARS = (type(None), int, float)


def _packed(name):
    """The entry point as a function of tensors and numbers, the views packed into one buffer here."""
    res, types = SIGNATURES[name]
    fn = lib()[name]
    fn.restype, fn.argtypes = res, [ctypes.c_void_p if t in (_P, ctypes.POINTER(ctypes.c_size_t)) else t for t in types]
    sizes = {i for i, t in enumerate(types) if t in (ctypes.c_void_p, ctypes.c_size_t)}

    def call(*args):
        buf = _ARGS()
        at = start = ctypes.addressof(buf)
        passed = []
        device = None
        for i, a in enumerate(args[:-1]):
            if type(a) in _SCALARS:
                if type(a) is int and i not in sizes and not -(1 << 31) <= a < 1 << 31:
                    raise OverflowError("argument does not fit 32 bits")
                passed.append(a)
                continue
            shape = a.shape
            n = len(shape)
            if a.dtype not in _DTYPES:
                raise TypeError(f"unsupported dtype {a.dtype}")
            if n > 4:
                raise ValueError("at most 4 dims")
            if a.get_device() != (a.get_device() if device is None else device):
                raise ValueError("all tensors must be on one device")
            device = a.get_device()
            _ARG[n].pack_into(buf, at - start, a.data_ptr(), _DTYPES[a.dtype], n, *shape, *a.stride())
            passed.append(at)
            at += 80
        return fn(*passed, args[-1])

    return call


def _args_module():
    """The module that packs the views in C++, or None where it was not built for this Python and torch."""
    from importlib.machinery import ExtensionFileLoader
    from importlib.util import module_from_spec, spec_from_file_location

    path = args_path(torch.__version__)
    if not os.path.exists(path):
        return None
    return module_from_spec(spec_from_file_location("fa8_args", path, loader=ExtensionFileLoader("fa8_args", path)))


_entries = {}  # what the calls below use, by name; "": the module


def _module():
    if "" not in _entries:
        _entries[""] = _args_module()
    return _entries[""]


def _entry(name):
    fn = _entries.get(name)
    if fn is None:
        module = _module()
        if module is None:
            fn = _packed(name)
        else:
            import functools

            fn = functools.partial(getattr(module, name), ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value)
        _entries[name] = fn
    return fn


def _beside(stream, make, *args):
    """make(*args), on ``stream`` where one is given: memory that work queued on the current stream may
    still use must not reach a kernel that does not wait for that work."""
    if stream is None:
        return make(*args)
    with torch.cuda.stream(stream):
        return make(*args)


def _empty(q, dtype, drop, *dims):
    """A new tensor beside q, of its shape with the last ``drop`` dims replaced."""
    module = _module()
    if module is not None and dtype in _DTYPES:
        try:
            return module.empty(q, _DTYPES[dtype], drop, *dims)
        except RuntimeError:
            pass  # torch raises its own error, e.g. OutOfMemoryError
    return torch.empty((*q.shape[:len(q.shape) - drop], *dims), dtype=dtype, device=q.device)


def _empty_lse(q):
    module = _module()
    if module is not None:
        try:
            return module.empty_lse(q)
        except RuntimeError:
            pass
    shape = (q.shape[0], q.shape[2], q.shape[1]) if q.dim() == 4 else (q.shape[1], q.shape[0])
    return torch.empty(shape, dtype=torch.float32, device=q.device)


def _zero_bounds(k):
    return torch.zeros((k.shape[0], k.shape[2], 2, k.shape[3]), dtype=torch.uint8,
                       device=k.device).view(torch.float8_e4m3fn)


def _call(name, index, stream, *args):
    """One library call on CUDA device ``index`` (-1: host tensors); tensors are passed as views, the
    stream goes last."""
    _run(_entries.get(name) or _entry(name), index, stream, *args)


def _run(fn, index, stream, *args):
    if index < 0:
        if torch.cuda.is_available():
            raise ValueError("the tensors must be on a CUDA device")
        status = fn(*args, 0)  # refuses what it would refuse, else says that there is no device
    else:
        handle = _raw_stream(index) if stream is None else stream.cuda_stream
        if _current_device() == index:
            status = fn(*args, handle)
        else:
            with torch.cuda.device(index):
                status = fn(*args, handle)
    if status:
        _raise(status)


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)  # no Stream object per call
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def rope_append(q, k, v, inv_freq, *, k_out, v_out, q_out=None, positions=None, interleaved=False,
                rotary_offset=0, rot_scale=1.0, descale_q=None, descale_k=None, descale_v=None,
                cu_seqlens_q=None, cu_seqlens_k=None, block_table=None, page_size=0, stream=None):
    """Rotates Q and K, rounds Q, K and V to E4M3, appends K and V to k_out / v_out (dense,
    varlen or paged, as in ``fwd``) and returns E4M3 Q."""
    if q_out is None:
        q_out = _beside(stream, _empty, q, torch.float8_e4m3fn, 1, q.shape[-1])
    _call("fa8_rope_append", q.get_device(), stream, q, k, v, inv_freq, positions, int(bool(interleaved)),
          int(rotary_offset), float(rot_scale), descale_q, descale_k, descale_v, q_out, k_out, v_out, cu_seqlens_q,
          cu_seqlens_k, block_table, int(page_size))
    return q_out


def page_bounds(k, bounds=None, *, cu_seqlens_k, block_table, page_size, cu_seqlens_q=None, new_tokens=-1,
                stream=None):
    """Updates the per-channel key bounds of the pages that hold the last new_tokens keys of each
    request (cu_seqlens_q: its new tokens; neither: all pages).  Without ``bounds`` a zeroed
    (num_pages, Hkv, 2, D) tensor is made."""
    if bounds is None:
        bounds = _beside(stream, _zero_bounds, k)
    _call("fa8_page_bounds", k.get_device(), stream, k, bounds, cu_seqlens_q, cu_seqlens_k, block_table, int(page_size),
          int(new_tokens))
    return bounds


def select_pages(q, bounds, top_k, *, cu_seqlens_k, block_table, page_size, cu_seqlens_q=None, causal=True,
                 keep_first=1, keep_last=1, pages=None, stream=None):
    """For every token and kv-head the top_k pages by bounded score: int32 (.., Hkv, top_k),
    ascending, -1 behind the last."""
    if pages is None:
        pages = _beside(stream, _empty, q, torch.int32, 2, bounds.shape[1], int(top_k))
    elif pages.shape[-1] != top_k:
        raise ValueError("pages must hold top_k entries")
    _call("fa8_select_pages", q.get_device(), stream, q, bounds, pages, cu_seqlens_q, cu_seqlens_k, block_table,
          int(page_size), int(bool(causal)), int(keep_first), int(keep_last))
    return pages


def fwd_pages(q, k, v, pages, *, cu_seqlens_k, block_table, page_size, descale_q=None, descale_k=None,
              descale_v=None, out=None, lse=None, cu_seqlens_q=None, causal=True, sink=None, softmax_scale=0.0,
              out_dtype=torch.bfloat16, return_lse=True, stream=None):
    """Attention over the listed pages of a paged cache; returns (out, lse) as ``fwd`` does."""
    if out is None:
        out = _beside(stream, _empty, q, out_dtype, 1, v.shape[-1])
    if lse is None and return_lse:
        lse = _beside(stream, _empty_lse, q)
    _call("fa8_fwd_pages", q.get_device(), stream, q, k, v, pages, descale_q, descale_k, descale_v, out, lse, cu_seqlens_q,
          cu_seqlens_k, block_table, int(page_size), int(bool(causal)), sink, float(softmax_scale))
    return out, lse


# ------------------------------------------------------------------ changed scores, drafted trees
def scored_workspace_size(q, k, v, *, cu_seqlens_q=None, cu_seqlens_k=None, block_table=None, page_size=0, ranges=None):
    """Bytes of workspace that ``fwd_scored`` and (without ranges) ``fwd_tree`` need for these shapes."""
    size = ctypes.c_size_t(0)
    views = [_view(t) for t in (q, k, v, cu_seqlens_q, cu_seqlens_k, block_table, ranges)]
    with _on_device(q.device):
        _raise(lib().fa8_fwd_scored_workspace_size(*map(_ref, views[:6]), int(page_size), _ref(views[6]), ctypes.byref(size)))
    return size.value


def _scored(name, stream, tensors, out, lse, placed, args, workspace, out_dtype, return_lse):
    """fa8_fwd_scored or fa8_fwd_tree, on the stream that its new tensors belong to.  ``tensors`` come before out,
    ``placed`` (packing and pages) and the rest after lse."""
    q, k, v = tensors[:3]
    index, module = q.get_device(), _module()
    if module is not None and index >= 0 and out_dtype in (torch.bfloat16, torch.float16):
        fn = _entries.get(name)
        if fn is None:
            import functools

            both = (ctypes.cast(getattr(lib(), x), ctypes.c_void_p).value for x in (name, "fa8_fwd_scored_workspace_size"))
            fn = _entries[name] = functools.partial(getattr(module, name), *both)
        got = None
        try:
            if stream is None and _current_device() == index:
                got = fn(*tensors, out, lse, *placed, *args, workspace, _DTYPES[out_dtype], return_lse, _raw_stream(index))
            else:
                handle = _raw_stream(index) if stream is None else stream.cuda_stream
                with torch.cuda.stream(stream), torch.cuda.device(index):
                    got = fn(*tensors, out, lse, *placed, *args, workspace, _DTYPES[out_dtype], return_lse, handle)
        except RuntimeError:
            pass  # torch raises its own error below, e.g. OutOfMemoryError
        if got is not None:
            if got[0]:
                _raise(got[0])
            return got[1:]
    if out is None:
        out = _beside(stream, _empty, q, out_dtype, 1, v.shape[-1])
    if lse is None and return_lse:
        lse = _beside(stream, _empty_lse, q)
    if workspace is None:
        n = 0
        if index >= 0:
            ranges = args[2] if name == "fa8_fwd_scored" else None
            n = scored_workspace_size(q, k, v, cu_seqlens_q=placed[0], cu_seqlens_k=placed[1], block_table=placed[2],
                                      page_size=placed[3], ranges=ranges)
        if n:
            workspace = _beside(stream, _empty, q, torch.float32, q.dim(), n // 4)
    elif not workspace.is_contiguous() or workspace.device != q.device:
        raise ValueError("workspace must be a contiguous tensor on q's device")
    ptr, size = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    fn = _entries.get((name,))
    if fn is None:
        fn = _entries[(name,)] = _packed(name)
    _run(fn, index, stream, *tensors, out, lse, *placed, *args, ptr, size)
    return out, lse


def fwd_scored(q, k, v, *, causal=False, window_left=-1, ranges=None, slopes=None, softcap=0.0, descale_q=None,
               descale_k=None, descale_v=None, out=None, lse=None, cu_seqlens_q=None, cu_seqlens_k=None,
               block_table=None, page_size=0, sink=None, softmax_scale=0.0, out_dtype=torch.bfloat16, return_lse=True,
               workspace=None, stream=None):
    """``fwd`` with scores capped by a tanh (``softcap``), less ``slopes`` times the distance, and for each token
    only the keys of its range (``ranges``: documents, prefixes, spans); returns (out, lse)."""
    return _scored("fa8_fwd_scored", stream, (q, k, v, descale_q, descale_k, descale_v), out, lse,
                   (cu_seqlens_q, cu_seqlens_k, block_table, int(page_size)),
                   (int(bool(causal)), int(window_left), ranges, slopes, float(softcap), sink, float(softmax_scale)),
                   workspace, out_dtype, return_lse)


def fwd_tree(q, k, v, masks, *, softcap=0.0, descale_q=None, descale_k=None, descale_v=None, out=None, lse=None,
             cu_seqlens_q=None, cu_seqlens_k=None, block_table=None, page_size=0, sink=None, softmax_scale=0.0,
             out_dtype=torch.bfloat16, return_lse=True, workspace=None, stream=None):
    """Attention of a tree of drafted tokens, the requests' last keys: each sees all keys before them and those
    of its mask; returns (out, lse)."""
    return _scored("fa8_fwd_tree", stream, (q, k, v, masks, descale_q, descale_k, descale_v), out, lse,
                   (cu_seqlens_q, cu_seqlens_k, block_table, int(page_size)), (float(softcap), sink, float(softmax_scale)),
                   workspace, out_dtype, return_lse)


def tree_masks(parents, *, cu_seqlens_k=None, cu_seqlens_q=None, max_tokens=None, masks=None, positions=None,
               stream=None):
    """Masks and positions of drafted tokens from their parents (negative: the text before them); returns
    (masks, positions).  Packed parents need ``max_tokens``, the most of a request (or ``masks``)."""
    if masks is None:
        if cu_seqlens_q is None:
            max_tokens = parents.shape[-1]
        elif max_tokens is None:
            raise ValueError("packed parents need max_tokens or masks")
    words = 0 if masks is not None else (int(max_tokens) + 31) // 32
    index = parents.get_device()
    if stream is None and index >= 0 and _module() is not None and _current_device() == index:
        fn = _entries.get("fa8_tree_masks") or _entry("fa8_tree_masks")
        got = None
        try:
            got = fn(parents, masks, positions, cu_seqlens_q, cu_seqlens_k, words, _raw_stream(index))
        except RuntimeError:
            pass  # torch raises its own error below, e.g. OutOfMemoryError
        if got is not None:
            if got[0]:
                _raise(got[0])
            return got[1:]
    if masks is None:
        masks = _beside(stream, _empty, parents, torch.int32, 0, words)
    if positions is None:
        positions = _beside(stream, _empty, parents, torch.int32, 0)
    fn = _entries.get(("fa8_tree_masks",))
    if fn is None:
        fn = _entries[("fa8_tree_masks",)] = _packed("fa8_tree_masks")
    _run(fn, index, stream, parents, masks, positions, cu_seqlens_q, cu_seqlens_k)
    return masks, positions


def keep_tokens(k, v, kept, *, new_tokens=0, cu_seqlens_q=None, cu_seqlens_k=None, block_table=None, page_size=0,
                stream=None):
    """Moves the accepted drafted tokens' K and V (``kept``: their indices, -1: none) to the first drafted slots of
    the caches, in place; returns (k, v)."""
    _call("fa8_keep_tokens", k.get_device(), stream, k, v, kept, cu_seqlens_q, cu_seqlens_k, block_table, int(page_size),
          int(new_tokens))
    return k, v


def fwd_case(case, **kw):
    """Runs ``fwd`` on an ``inputs.Case`` (tensors already on the GPU)."""
    args = dict(descale_q=case.descale_q, descale_k=case.descale_k, descale_v=case.descale_v,
                cu_seqlens_q=case.cu_seqlens_q, cu_seqlens_k=case.cu_seqlens_k,
                block_table=case.block_table, page_size=case.page_size, causal=case.causal,
                window_left=case.window_left, sink=case.sink, softmax_scale=case.softmax_scale,
                out_dtype=case.out_dtype)
    args.update(kw)
    return fwd(case.q, case.k, case.v, **args)


def check(stream=None) -> int:
    """Synchronises and returns (and clears) the device status word; raises on a CUDA error."""
    dev = torch.device("cuda", torch.cuda.current_device())
    st = lib().fa8_check(_stream_handle(stream, dev))
    if st == FA8_ERR_CUDA:
        _raise(st)
    return st


def set_wait_timeout_ns(ns: int):
    _raise(lib().fa8_set_wait_timeout_ns(int(ns)))


def set_decode_kernel(enable: bool):
    """Routes decode shapes (<= 16 query rows per kv-head) to the decode kernel (default)."""
    _raise(lib().fa8_set_decode_kernel(1 if enable else 0))


def debug_wait_probe(stream=None) -> int:
    dev = torch.device("cuda", torch.cuda.current_device())
    return lib().fa8_debug_wait_probe(_stream_handle(stream, dev))


def version() -> int:
    return lib().fa8_version()
