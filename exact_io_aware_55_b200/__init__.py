"""Exact IO-aware attention for B200 (sm_100a).

The compute lives in ``libfa.so`` (C ABI, ``include/fa.h``); this package is
its Python binding.  Functions named like the C entry points take torch CUDA
tensors and pass their pointers through unchanged; PyTorch only provides the
device memory and the stream.  ``attention_forward`` / ``attention_backward``
additionally allocate the outputs (and the backward workspace) with torch.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import FA_OK, FAError, LIB_PATH, STATUS_CODES, STATUS_NAMES, check, lib, strerror

__all__ = [
    "FAError", "LIB_PATH", "fa_fwd", "fa_fwd_fp8", "fa_bwd", "fa_bwd_deterministic", "fa_bwd_workspace_size",
    "fa_bwd_events", "fa_fwd_plan", "fa_bwd_fp8", "fa_bwd_fp8_workspace_size", "attention_backward_fp8", "fa_get_device_status", "fa_device_status", "fa_fwd_decode", "fa_fwd_decode_workspace_size", "attention_decode",
    "fa_fwd_standard", "fa_fwd_standard_workspace_size", "attention_forward_standard",
    "fa_watchdog_selftest", "attention_forward", "attention_backward", "attention_forward_fp8", "lib",
    "STATUS_NAMES", "STATUS_CODES", "strerror",
    "ROPE_SCALINGS", "rope_frequencies", "fa_rope", "rope_forward", "rope_backward", "fa_page_tables",
    "fa_cache_append_fp8", "fa_fwd_decode_paged_fp8", "fa_fwd_decode_paged_fp8_workspace_size",
    "attention_decode_paged_fp8",
]


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _shape(q):
    if q.dim() != 4:
        raise ValueError("tensors must be [B, H, N, d]")
    return tuple(int(x) for x in q.shape)


def _check_tensors(ref_shape, dtype, *ts):
    for t in ts:
        if t.device.type != "cuda":
            raise ValueError("tensors must be CUDA tensors")
        if tuple(t.shape) != ref_shape or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"expected contiguous {dtype} {ref_shape}, got {t.dtype} {tuple(t.shape)}")


def fa_fwd(q, k, v, o, lse, scale: float, causal: bool, stream=None) -> None:
    """O, LSE <- attention(q, k, v) (bf16 in/out, LSE fp32 [B,H,N])."""
    B, H, N, d = _shape(q)
    _check_tensors((B, H, N, d), torch.bfloat16, q, k, v, o)
    _check_tensors((B, H, N), torch.float32, lse)
    check(lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale), int(bool(causal)),
                     _stream_ptr(stream)))


def fa_fwd_fp8(q8, k8, v8, q_descale, k_descale, v_descale, o, lse, scale: float, causal: bool,
               stream=None) -> None:
    """Forward with e4m3 inputs (uint8 or float8_e4m3fn tensors) and per-tensor descales."""
    B, H, N, d = _shape(q8)
    for t in (q8, k8, v8):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or tuple(t.shape) != (B, H, N, d) \
                or not t.is_contiguous() or t.device.type != "cuda":
            raise ValueError("e4m3 inputs must be contiguous CUDA uint8/float8_e4m3fn [B,H,N,d]")
    _check_tensors((B, H, N, d), torch.bfloat16, o)
    _check_tensors((B, H, N), torch.float32, lse)
    check(lib.fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), float(q_descale), float(k_descale), float(v_descale),
                         _ptr(o), _ptr(lse), B, H, N, d, float(scale), int(bool(causal)), _stream_ptr(stream)))


def fa_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    n = int(lib.fa_bwd_workspace_size(B, H, N, d))
    if n == ctypes.c_size_t(-1).value:
        raise FAError(1, "invalid shape for fa_bwd_workspace_size")
    return n


def fa_bwd(q, k, v, o, do, lse, dq, dk, dv, scale: float, causal: bool, workspace, stream=None) -> None:
    """dQ, dK, dV <- backward of attention; workspace is a CUDA uint8 tensor."""
    B, H, N, d = _shape(q)
    _check_tensors((B, H, N, d), torch.bfloat16, q, k, v, o, do, dq, dk, dv)
    _check_tensors((B, H, N), torch.float32, lse)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                     B, H, N, d, float(scale), int(bool(causal)), _ptr(workspace), wbytes, _stream_ptr(stream)))


def fa_bwd_events(q, k, v, o, do, lse, dq, dk, dv, scale: float, causal: bool, workspace, events,
                  stream=None) -> None:
    """fa_bwd that also records four torch.cuda.Event objects on the stream:
    before the preprocess, before and after the main kernel, after the last launch."""
    B, H, N, d = _shape(q)
    _check_tensors((B, H, N, d), torch.bfloat16, q, k, v, o, do, dq, dk, dv)
    _check_tensors((B, H, N), torch.float32, lse)
    if len(events) != 4:
        raise ValueError("fa_bwd_events takes four events")
    for e in events:
        if int(e.cuda_event) == 0:         # torch creates the CUDA event at its first record
            e.record(torch.cuda.current_stream() if stream is None else stream)
    arr = (ctypes.c_void_p * 4)(*(int(e.cuda_event) for e in events))
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.fa_bwd_events(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                            B, H, N, d, float(scale), int(bool(causal)), _ptr(workspace), wbytes, arr,
                            _stream_ptr(stream)))


def fa_bwd_fp8_workspace_size(B: int, H: int, N: int, d: int) -> int:
    n = int(lib.fa_bwd_fp8_workspace_size(B, H, N, d))
    if n == ctypes.c_size_t(-1).value:
        raise FAError(1, "invalid shape for fa_bwd_fp8_workspace_size (d must be 128)")
    return n


def _check_e4m3(shape, *ts):
    for t in ts:
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or tuple(t.shape) != shape \
                or not t.is_contiguous() or t.device.type != "cuda":
            raise ValueError("e4m3 inputs must be contiguous CUDA uint8/float8_e4m3fn [B,H,N,d]")


def fa_bwd_fp8(q8, k8, v8, q_descale, k_descale, v_descale, o, do, lse, dq, dk, dv, scale: float, causal: bool,
               workspace, stream=None) -> None:
    """dQ, dK, dV (real units) <- backward of the e4m3 forward; workspace is a CUDA uint8 tensor."""
    B, H, N, d = _shape(q8)
    _check_e4m3((B, H, N, d), q8, k8, v8)
    _check_tensors((B, H, N, d), torch.bfloat16, o, do, dq, dk, dv)
    _check_tensors((B, H, N), torch.float32, lse)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.fa_bwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), float(q_descale), float(k_descale), float(v_descale),
                         _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                         int(bool(causal)), _ptr(workspace), wbytes, _stream_ptr(stream)))


def fa_fwd_plan(B: int, H: int, N: int, d: int, causal: bool):
    """(ctas, items, pair_items) of the forward's launch for this shape."""
    c, it, pi = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    check(lib.fa_fwd_plan(B, H, N, d, int(bool(causal)), ctypes.byref(c), ctypes.byref(it), ctypes.byref(pi)))
    return c.value, it.value, pi.value


def fa_bwd_deterministic(q, k, v, o, do, lse, dq, dk, dv, scale: float, causal: bool, workspace,
                         stream=None) -> None:
    """As fa_bwd, with dQ from a separate atomic-free pass: bit-reproducible results."""
    B, H, N, d = _shape(q)
    _check_tensors((B, H, N, d), torch.bfloat16, q, k, v, o, do, dq, dk, dv)
    _check_tensors((B, H, N), torch.float32, lse)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.fa_bwd_deterministic(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
                                   _ptr(dv), B, H, N, d, float(scale), int(bool(causal)), _ptr(workspace), wbytes,
                                   _stream_ptr(stream)))


def fa_fwd_decode_workspace_size(B: int, H: int, Nq: int, Nk: int, d: int) -> int:
    n = int(lib.fa_fwd_decode_workspace_size(B, H, Nq, Nk, d))
    if n == ctypes.c_size_t(-1).value:
        raise FAError(1, "invalid shape for fa_fwd_decode_workspace_size")
    return n


def fa_fwd_decode(q, k, v, o, lse, scale: float, causal: bool, workspace, stream=None) -> None:
    """O, LSE <- attention of q [B,H,Nq,d] (Nq <= 16) over a KV cache k, v [B,H,Nk,d]."""
    B, H, Nq, d = _shape(q)
    Nk = int(k.shape[2])
    _check_tensors((B, H, Nk, d), torch.bfloat16, k, v)
    _check_tensors((B, H, Nq, d), torch.bfloat16, q, o)
    _check_tensors((B, H, Nq), torch.float32, lse)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.fa_fwd_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d, float(scale),
                            int(bool(causal)), _ptr(workspace), wbytes, _stream_ptr(stream)))


def attention_decode(q, k, v, scale: float | None = None, causal: bool = False, workspace=None, stream=None):
    """Allocates O, LSE (and the split workspace unless given) with torch and runs fa_fwd_decode."""
    B, H, Nq, d = _shape(q)
    Nk = int(k.shape[2])
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(16, fa_fwd_decode_workspace_size(B, H, Nq, Nk, d)), dtype=torch.uint8,
                                device=q.device)
    fa_fwd_decode(q, k, v, o, lse, _default_scale(d) if scale is None else scale, causal, workspace, stream)
    return o, lse


def fa_fwd_standard_workspace_size(B: int, H: int, N: int, d: int) -> int:
    n = int(lib.fa_fwd_standard_workspace_size(B, H, N, d))
    if n == ctypes.c_size_t(-1).value:
        raise FAError(1, "invalid shape for fa_fwd_standard_workspace_size")
    return n


def fa_fwd_standard(q, k, v, o, lse, scale: float, causal: bool, workspace, stream=None) -> None:
    """Standard attention with S and P materialised in the workspace (the IO baseline)."""
    B, H, N, d = _shape(q)
    _check_tensors((B, H, N, d), torch.bfloat16, q, k, v, o)
    _check_tensors((B, H, N), torch.float32, lse)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.fa_fwd_standard(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
                              int(bool(causal)), _ptr(workspace), wbytes, _stream_ptr(stream)))


def attention_forward_standard(q, k, v, scale: float | None = None, causal: bool = False, workspace=None,
                               stream=None):
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(256, fa_fwd_standard_workspace_size(B, H, N, d)), dtype=torch.uint8,
                                device=q.device)
    fa_fwd_standard(q, k, v, o, lse, _default_scale(d) if scale is None else scale, causal, workspace, stream)
    return o, lse


def fa_device_status(stream=None):
    """(status, where) of the device status word; synchronises the stream and clears it."""
    where = ctypes.c_uint32(0)
    st = lib.fa_device_status(_stream_ptr(stream), ctypes.byref(where))
    return st, int(where.value)


def fa_watchdog_selftest(limit_us: int, stream=None) -> None:
    check(lib.fa_watchdog_selftest(int(limit_us), _stream_ptr(stream)))


def _default_scale(d: int) -> float:
    return d ** -0.5


def attention_forward(q, k, v, scale: float | None = None, causal: bool = False, stream=None):
    """Allocates O (bf16) and LSE (fp32) with torch and runs fa_fwd."""
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, _default_scale(d) if scale is None else scale, causal, stream)
    return o, lse


def attention_forward_fp8(q8, k8, v8, q_descale, k_descale, v_descale, scale: float | None = None,
                          causal: bool = False, stream=None):
    B, H, N, d = _shape(q8)
    o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    fa_fwd_fp8(q8, k8, v8, q_descale, k_descale, v_descale, o, lse,
               _default_scale(d) if scale is None else scale, causal, stream)
    return o, lse


def attention_backward(q, k, v, o, do, lse, scale: float | None = None, causal: bool = False, workspace=None,
                       stream=None, deterministic: bool = False):
    """Allocates dQ, dK, dV (and the workspace unless given) with torch and runs
    fa_bwd (or fa_bwd_deterministic)."""
    B, H, N, d = _shape(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = torch.empty(max(1, fa_bwd_workspace_size(B, H, N, d)), dtype=torch.uint8, device=q.device)
    fn = fa_bwd_deterministic if deterministic else fa_bwd
    fn(q, k, v, o, do, lse, dq, dk, dv, _default_scale(d) if scale is None else scale, causal, workspace, stream)
    return dq, dk, dv


def attention_backward_fp8(q8, k8, v8, q_descale, k_descale, v_descale, o, do, lse, scale: float | None = None,
                           causal: bool = False, workspace=None, stream=None):
    """(dQ, dK, dV) bf16 of the e4m3 forward, allocating outputs and workspace with torch."""
    B, H, N, d = _shape(q8)
    dq, dk, dv = (torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device) for _ in range(3))
    if workspace is None:
        workspace = torch.empty(max(256, fa_bwd_fp8_workspace_size(B, H, N, d)), dtype=torch.uint8, device=q8.device)
    fa_bwd_fp8(q8, k8, v8, q_descale, k_descale, v_descale, o, do, lse, dq, dk, dv,
               _default_scale(d) if scale is None else scale, causal, workspace, stream)
    return dq, dk, dv


# ------------------------------------------------- serving over an 8-bit paged cache, and rotary positions
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
_E4M3 = (torch.uint8, torch.float8_e4m3fn)


def _launch(fn, device: int, stream, *args):
    """Calls fn(*args, stream) with GPU `device` current, on `stream` or that GPU's current stream."""
    if device == _current_device():
        st = fn(*args, _raw_stream(device) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device) if stream is None else stream.cuda_stream)
    if st != FA_OK:
        check(st)


# A decode step makes these calls once per layer and token, so the checks are written for few Python steps.
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _not_as(t, name, shape, dtypes, device):
    raise ValueError(f"{name}: expected contiguous {' or '.join(str(x) for x in dtypes)} {tuple(shape)} on cuda:{device}, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _check_as(t, name, shape, dtypes, device):
    if t.shape != shape or t.dtype not in dtypes or not t.is_contiguous() or t.get_device() != device:
        _not_as(t, name, shape, dtypes, device)


def _gpu_index(t):
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    return t.get_device()


def _empty(like, shape, stride, dtype, stream):
    """A tensor of the memory of the stream that the call runs on: freed, it is next used in that stream's order."""
    if stream is None:
        return like.new_empty_strided(shape, stride, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty_strided(shape, stride, dtype=dtype)


def _dims(t):
    if t.dim() != 4:
        raise ValueError("tensors must be [B, H, N, d]")
    return t.shape


_i32, _f32, _f64, _bf16 = torch.int32, torch.float32, torch.float64, torch.bfloat16
_I32, _F32, _F64, _BF16 = (_i32,), (_f32,), (_f64,), (_bf16,)


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_length: float = 0.0, low: float = 1.0, high: float | None = None, device="cuda"):
    """(inv_freq, attention factor) of rotary positions: inv_freq is an fp64 tensor [rot_dim / 2] on `device`,
    radians per position.  scaling is a key of ROPE_SCALINGS (see fa_rope_scaling in fa.h); `high` is 32 turns for
    "yarn" and 4 for "bands" unless given."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    out = (ctypes.c_double * max(1, rot_dim // 2))()
    att = ctypes.c_double()
    check(lib.fa_rope_frequencies(out, ctypes.byref(att), rot_dim, base, ROPE_SCALINGS[scaling], factor,
                                  original_length, low, high))
    return torch.tensor(list(out), dtype=torch.float64, device=device), att.value


def fa_rope(x, y, positions, inv_freq, factor: float = 1.0, interleaved: bool = False, transpose: bool = False,
            stream=None) -> None:
    """y <- x [B,H,N,d] bf16 with rotary positions on its first 2 * len(inv_freq) elements.  x and y may have any
    batch, head and token strides (d contiguous); y may be x.  positions: int32 [B,N], or None for 0..N-1."""
    dev = _gpu_index(x)
    if y.shape != x.shape or y.dtype is not torch.bfloat16 or y.get_device() != dev or y.dim() != 4 or y.stride(3) != 1:
        raise ValueError(f"y: expected bf16 {tuple(x.shape)} on cuda:{dev} with d contiguous, got {y.dtype} "
                         f"{tuple(y.shape)} on {y.device}")
    _rope(x, y, y.stride(), positions, inv_freq, factor, interleaved, transpose, stream, dev)


def _rope(x, y, y_stride, positions, inv_freq, factor, interleaved, transpose, stream, dev):
    B, H, N, d = _dims(x)
    xb, xh, xn, xd = x.stride()
    if x.dtype is not torch.bfloat16 or xd != 1:
        raise ValueError(f"x: expected bf16 with d contiguous, got {x.dtype} with strides {x.stride()}")
    if positions is not None:
        if (positions.shape != (B, N) or positions.dtype is not _i32 or not positions.is_contiguous()
                or positions.get_device() != dev):
            _not_as(positions, "positions", (B, N), _I32, dev)
        positions = positions.data_ptr()
    pairs = inv_freq.numel()
    if inv_freq.dim() != 1 or inv_freq.dtype is not _f64 or not inv_freq.is_contiguous() or inv_freq.get_device() != dev:
        _not_as(inv_freq, "inv_freq", (pairs,), _F64, dev)
    _launch(lib.fa_rope, dev, stream, x.data_ptr(), y.data_ptr(), positions, inv_freq.data_ptr(), factor, B, H, N, d,
            2 * pairs, 1 if interleaved else 0, 1 if transpose else 0, xb, xh, xn, y_stride[0], y_stride[1], y_stride[2])


def _rope_new(x, positions, inv_freq, factor, interleaved, transpose, stream):
    B, H, N, d = _dims(x)
    dev = _gpu_index(x)
    stride = (H * N * d, N * d, d, 1)
    y = _empty(x, (B, H, N, d), stride, None, stream)      # bf16, or refused below
    _rope(x, y, stride, positions, inv_freq, factor, interleaved, transpose, stream, dev)
    return y


def rope_forward(x, positions, inv_freq, interleaved: bool = False, factor: float = 1.0, stream=None):
    """Rotary positions on x, as a new contiguous tensor (of `stream`'s memory, as torch.cuda.stream would give it)."""
    return _rope_new(x, positions, inv_freq, factor, interleaved, False, stream)


def rope_backward(dy, positions, inv_freq, interleaved: bool = False, factor: float = 1.0, stream=None):
    """Gradient of rope_forward with respect to x, as a new contiguous tensor."""
    return _rope_new(dy, positions, inv_freq, factor, interleaved, True, stream)


def fa_page_tables(ctx_lens, new_lens, free_pages, free_head, block_table, slots, positions, seq_lens,
                   free_head_out, page_size: int, stream=None, held_pages=None) -> None:
    """Grows (new_lens >= 0) or finishes (new_lens < 0) the requests of a batch: takes pages from free_pages,
    writes block_table, slots, positions, seq_lens and free_head_out.  All int32; seq_lens may be ctx_lens and
    free_head_out may be free_head.  held_pages [B] (read and written) counts each request's pages; it is needed
    where ctx_lens is lowered across a page's border between calls, whose page would be lost otherwise."""
    dev = _gpu_index(ctx_lens)
    if slots.dim() != 2 or block_table.dim() != 2:
        raise ValueError("slots must be [B, N] and block_table [B, max_pages]")
    B, N = slots.shape
    max_pages = block_table.shape[1]
    n_free = free_pages.numel()
    # one look at what all have in common, then the shapes
    for t in (ctx_lens, new_lens, free_pages, free_head, block_table, slots, positions, seq_lens, free_head_out):
        if t.dtype is not _i32 or not t.is_contiguous() or t.get_device() != dev:
            _not_as(t, "every argument", t.shape, _I32, dev)
    if (ctx_lens.shape != (B,) or new_lens.shape != (B,) or free_pages.dim() != 1 or free_head.shape != (1,)
            or block_table.shape[0] != B or positions.shape != (B, N) or seq_lens.shape != (B,) or free_head_out.shape != (1,)):
        raise ValueError("expected ctx_lens, new_lens, seq_lens [B], free_pages [n_free], free_head, free_head_out [1], "
                         f"block_table [B, max_pages], slots, positions [B, N] with [B, N] = {[B, N]}")
    args = (ctx_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), free_head.data_ptr(), block_table.data_ptr(),
            slots.data_ptr(), positions.data_ptr(), seq_lens.data_ptr(), free_head_out.data_ptr())
    if held_pages is None:
        _launch(lib.fa_page_tables, dev, stream, *args, B, N, n_free, max_pages, page_size)
    else:
        _check_as(held_pages, "held_pages", (B,), _I32, dev)
        _launch(lib.fa_page_tables_held, dev, stream, *args, held_pages.data_ptr(), B, N, n_free, max_pages, page_size)


def _check_cache(k_cache, v_cache, k_scale, v_scale, Hkv, d, dev):
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, Hkv, page_size, d]")
    pages, heads, page, depth = shape = k_cache.shape
    if heads != Hkv or depth != d:
        raise ValueError(f"k_cache: expected [num_pages, {Hkv}, page_size, {d}], got {tuple(shape)}")
    if k_cache.dtype not in _E4M3 or not k_cache.is_contiguous() or k_cache.get_device() != dev:
        _not_as(k_cache, "k_cache", shape, _E4M3, dev)
    if v_cache.shape != shape or v_cache.dtype not in _E4M3 or not v_cache.is_contiguous() or v_cache.get_device() != dev:
        _not_as(v_cache, "v_cache", shape, _E4M3, dev)
    scales = (pages, Hkv)
    if k_scale.shape != scales or k_scale.dtype is not _f32 or not k_scale.is_contiguous() or k_scale.get_device() != dev:
        _not_as(k_scale, "k_scale", scales, _F32, dev)
    if v_scale.shape != scales or v_scale.dtype is not _f32 or not v_scale.is_contiguous() or v_scale.get_device() != dev:
        _not_as(v_scale, "v_scale", scales, _F32, dev)
    return pages, page


def fa_cache_append_fp8(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream=None) -> None:
    """Quantises k, v [B,Hkv,N,d] bf16 into the pages that slots [B,N] int32 names (negative: not written);
    k_cache, v_cache e4m3 [num_pages,Hkv,page_size,d], k_scale, v_scale fp32 [num_pages,Hkv]."""
    B, Hkv, N, d = shape = _dims(k)
    dev = _gpu_index(k)
    if k.dtype is not _bf16 or not k.is_contiguous():
        _not_as(k, "k", shape, _BF16, dev)
    if v.shape != shape or v.dtype is not _bf16 or not v.is_contiguous() or v.get_device() != dev:
        _not_as(v, "v", shape, _BF16, dev)
    if slots.shape != (B, N) or slots.dtype is not _i32 or not slots.is_contiguous() or slots.get_device() != dev:
        _not_as(slots, "slots", (B, N), _I32, dev)
    pages, page = _check_cache(k_cache, v_cache, k_scale, v_scale, Hkv, d, dev)
    _launch(lib.fa_cache_append_fp8, dev, stream, k.data_ptr(), v.data_ptr(), slots.data_ptr(), k_cache.data_ptr(),
               v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), B, Hkv, N, d, pages, page)


def fa_fwd_decode_paged_fp8_workspace_size(B: int, H: int, Hkv: int, Nq: int, d: int) -> int:
    n = int(lib.fa_fwd_decode_paged_fp8_workspace_size(B, H, Hkv, Nq, d))
    if n == ctypes.c_size_t(-1).value:
        raise FAError(1, "invalid or unsupported shape for fa_fwd_decode_paged_fp8_workspace_size")
    return n


def fa_fwd_decode_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, o, lse, scale: float,
                            causal: bool, workspace, stream=None) -> None:
    """O, LSE <- attention of q [B,H,Nq,d] (Nq <= 16) over the first seq_lens[b] tokens of each request's pages;
    block_table int32 [B,max_pages], seq_lens int32 [B], caches and scales as in fa_cache_append_fp8."""
    shape = _dims(q)
    dev = _gpu_index(q)
    _check_as(o, "o", shape, _BF16, dev)
    _check_as(lse, "lse", shape[:3], _F32, dev)
    _decode_paged(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, o, lse, scale, causal, workspace, stream, dev)


def _decode_paged(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, o, lse, scale, causal, workspace, stream,
                  dev):
    B, H, Nq, d = shape = q.shape
    if q.dtype is not _bf16 or not q.is_contiguous():
        _not_as(q, "q", shape, _BF16, dev)
    if k_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_cache must be [num_pages, Hkv, page_size, d] and block_table [B, max_pages]")
    Hkv = k_cache.shape[1]
    pages, page = _check_cache(k_cache, v_cache, k_scale, v_scale, Hkv, d, dev)
    max_pages = block_table.shape[1]
    if (block_table.shape[0] != B or block_table.dtype is not _i32 or not block_table.is_contiguous()
            or block_table.get_device() != dev):
        _not_as(block_table, "block_table", (B, max_pages), _I32, dev)
    if seq_lens.shape != (B,) or seq_lens.dtype is not _i32 or not seq_lens.is_contiguous() or seq_lens.get_device() != dev:
        _not_as(seq_lens, "seq_lens", (B,), _I32, dev)
    wptr, wbytes = 0, 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on cuda:{dev}")
        wptr, wbytes = workspace.data_ptr(), workspace.nbytes
    _launch(lib.fa_fwd_decode_paged_fp8, dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
            lse.data_ptr(), B, H, Hkv, Nq, d, pages, page, max_pages, scale, 1 if causal else 0, wptr, wbytes)


def attention_decode_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                               scale: float | None = None, causal: bool = False, workspace=None, stream=None):
    """Allocates O, LSE (and the workspace unless given) with torch, on `stream`, and runs fa_fwd_decode_paged_fp8."""
    B, H, Nq, d = _dims(q)
    dev = _gpu_index(q)
    o = _empty(q, (B, H, Nq, d), (H * Nq * d, Nq * d, d, 1), None, stream)      # bf16, or refused below
    lse = _empty(q, (B, H, Nq), (H * Nq, Nq, 1), _f32, stream)
    if workspace is None:
        n = fa_fwd_decode_paged_fp8_workspace_size(B, H, k_cache.shape[1], Nq, d)
        workspace = _empty(q, (max(16, n),), (1,), torch.uint8, stream)
    _decode_paged(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, o, lse,
                  _default_scale(d) if scale is None else scale, causal, workspace, stream, dev)
    return o, lse
