"""W4-G256 quantized matmul for B200 (sm_100a): Python binding.

Every function here marshals torch CUDA tensors into the C ABI of libw4.so
(``include/w4.h``) and raises ``W4Error`` on a non-OK status.  All arithmetic
runs in the library's CUDA kernels; torch only provides device memory and the
current stream.  There is no CPU path: without the built library, calls raise
``LibraryMissing``.

Entry points (same names as the C ABI):
    w4_pack(w)                              -> codes, d, m
    w4_pack_g32(w)                          -> codes, d, m   (groups of 32)
    w4_pack_codes(q)                        -> codes
    w4_unpack(codes, K)                     -> q
    w4_gemv(codes, d, m, x, out_dtype)      -> y
    w4_gemv_g32(codes, d, m, x, out_dtype)  -> y   (group-32 weights)
    w4a8_gemv(codes, d, m, qa, dx, bsum, out_dtype) -> y   (int8 activations, M <= 8)
    w4a8_gemv_bf16(codes, d, m, x, out_dtype) -> y   (x quantised inside, M <= 8)
    q8_quantize_act(x)                      -> qa, dx, bsum
    w4a8_mmq(codes, d, m, qa, dx, bsum, out_dtype) -> y
    w4a8_mmq_static(codes, d, m, qa, dx, bsum, out_dtype) -> y   (no workspace)
    w4a8_mmq_blockdots(codes, d, m, qa, dx, bsum, out_dtype) -> y, P   (test: int32 block products)
    w4a8_gemv_blockdots(codes, d, m, qa, dx, bsum, out_dtype) -> y, P  (test: int32 block products)
    w4a8_mmq_workspace_size(M, N, K)
    w4_check_device_error()
Microscaled 4-bit floating point (planes codes, scales, g; g is None for the
MX format and the fp32 tensor scale for NV):
    f4_tensor_scale(x)                      -> g
    f4_quantize(x, format, tensor_scale)    -> codes, scales, g
    f4_dequantize(codes, scales, g, out_dtype) -> y
    f4_embed(codes, scales, g, ids, scale, out_dtype) -> y   (rows of a packed table)
    f4_mm(codes, scales, g, qa, sa, ga, out_dtype) -> y      (both operands 4-bit, any M)
    f4_gemv(codes, scales, g, x, out_dtype) -> y             (bf16 activations, M <= 8)
    f4_gemv_workspace_size(M, N, K, format)
"""
from __future__ import annotations

from ._lib import (LibraryMissing, W4_F4_MX, W4_F4_NV, W4_IN_BF16, W4_IN_F16, W4_IN_F32, W4_OK,
                   W4_OUT_BF16, W4_OUT_F32, load, status_string)

__all__ = [
    "W4Error", "LibraryMissing", "w4_pack", "w4_pack_g32", "w4_pack_codes", "w4_unpack",
    "w4_gemv", "w4_gemv_g32", "w4a8_gemv",
    "w4a8_gemv_bf16",
    "q8_quantize_act", "w4a8_mmq", "w4a8_mmq_static", "w4a8_mmq_workspace_size",
    "w4a8_mmq_blockdots", "w4a8_gemv_blockdots",
    "f4_tensor_scale", "f4_quantize", "f4_dequantize", "f4_embed", "f4_mm", "f4_gemv",
    "f4_gemv_workspace_size",
    "w4_check_device_error",
    "w4_abi_version", "lib",
]

GROUP = 256
GROUP32 = 32
BLOCK = 32


class W4Error(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = int(code)
        msg = status_string(code)
        if code == 6:  # W4_ERR_CUDA
            msg += f" (cudaError {load().w4_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")


def lib():
    """The loaded ctypes library (raw C ABI)."""
    return load()


def _torch():
    import torch
    return torch


def _check(code: int, what: str):
    if code != W4_OK:
        raise W4Error(code, what)


def _stream(stream=None) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t) -> int:
    return t.data_ptr()


def _div(n: int, unit: int):
    """n / unit when exact, else None (any extent: the library then rejects n)."""
    return n // unit if n % unit == 0 else None


def _need(t, dtype, name: str, shape):
    """Check a tensor argument before its pointer crosses the C ABI, which
    sees only pointers and sizes: type, dtype, exact shape (None = any extent)
    and contiguity.  A plane with the wrong extent would otherwise be read or
    written out of bounds.  Placement is checked by _on_device, once every
    argument's shape has been."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(e is not None and e != s for e, s in zip(shape, t.shape)):
        want = "[" + ", ".join("*" if e is None else str(e) for e in shape) + "]"
        raise ValueError(f"{name} must have shape {want}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_device(**tensors):
    """Every tensor must be a CUDA tensor on the current device, where the
    library launches its kernels."""
    torch = _torch()
    for name, t in tensors.items():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    current = torch.cuda.current_device()
    for name, t in tensors.items():
        if t.device.index != current:
            raise ValueError(f"{name} is on {t.device}, not the current device cuda:{current}")


def _as_u16(t):
    torch = _torch()
    if t.dtype in (torch.bfloat16, torch.float16):
        return t.view(torch.int16)
    return t


def w4_abi_version() -> int:
    return int(load().w4_abi_version())


def w4_check_device_error() -> None:
    """Synchronise and raise if a kernel reported a timed-out wait."""
    _check(load().w4_check_device_error(), "w4_check_device_error")


def _pack(fn: str, group: int, w, codes, d, m, stream):
    torch = _torch()
    _need(w, torch.float32, "w", (None, None))
    N, K = w.shape
    if codes is None:
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    _need(codes, torch.uint8, "codes", (N, _div(K, 2)))
    if d is None:
        d = torch.empty((N, K // group), dtype=torch.float16, device=w.device)
    _need(d, torch.float16, "d", (N, _div(K, group)))
    if m is None:
        m = torch.empty((N, K // group), dtype=torch.float16, device=w.device)
    _need(m, torch.float16, "m", (N, _div(K, group)))
    _on_device(w=w, codes=codes, d=d, m=m)
    _check(getattr(load(), fn)(_ptr(w), N, K, _ptr(codes), _ptr(d), _ptr(m), _stream(stream)),
           fn)
    return codes, d, m


def w4_pack(w, codes=None, d=None, m=None, stream=None):
    """Quantise fp32 W[N,K] (K % 256 == 0) to W4-G256 planes.
    Returns (codes uint8[N,K/2], d fp16[N,K/256], m fp16[N,K/256])."""
    return _pack("w4_pack", GROUP, w, codes, d, m, stream)


def w4_pack_g32(w, codes=None, d=None, m=None, stream=None):
    """Quantise fp32 W[N,K] (K % 32 == 0) to group-32 planes (one d, m per
    32 weights).  Returns (codes uint8[N,K/2], d fp16[N,K/32], m fp16[N,K/32])."""
    return _pack("w4_pack_g32", GROUP32, w, codes, d, m, stream)


def w4_pack_codes(q, codes=None, stream=None):
    """One code per byte q uint8[N,K] -> packed codes uint8[N,K/2]."""
    torch = _torch()
    _need(q, torch.uint8, "q", (None, None))
    N, K = q.shape
    if codes is None:
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=q.device)
    _need(codes, torch.uint8, "codes", (N, _div(K, 2)))
    _on_device(q=q, codes=codes)
    _check(load().w4_pack_codes(_ptr(q), N, K, _ptr(codes), _stream(stream)), "w4_pack_codes")
    return codes


def w4_unpack(codes, K: int, q=None, stream=None):
    """Packed codes uint8[N,K/2] -> one code per byte uint8[N,K]."""
    torch = _torch()
    _need(codes, torch.uint8, "codes", (None, _div(K, 2)))
    if K % 2:
        raise ValueError("codes must have K/2 columns")
    N = codes.shape[0]
    if q is None:
        q = torch.empty((N, K), dtype=torch.uint8, device=codes.device)
    _need(q, torch.uint8, "q", (N, K))
    _on_device(codes=codes, q=q)
    _check(load().w4_unpack(_ptr(codes), N, K, _ptr(q), _stream(stream)), "w4_unpack")
    return q


def _out_code(out_dtype, y=None) -> int:
    """Output code from out_dtype; with out_dtype None, y's dtype, else bf16."""
    torch = _torch()
    if out_dtype is None:
        out_dtype = y.dtype if isinstance(y, torch.Tensor) else torch.bfloat16
    if out_dtype in (torch.float32, "f32", "fp32", W4_OUT_F32):
        return W4_OUT_F32
    if out_dtype in (torch.bfloat16, "bf16", W4_OUT_BF16):
        return W4_OUT_BF16
    raise ValueError(f"unsupported out_dtype {out_dtype}")


def _output(y, M: int, N: int, oc: int, like):
    """The caller's y checked against [M,N] and the output type, or a new one."""
    torch = _torch()
    dtype = torch.float32 if oc == W4_OUT_F32 else torch.bfloat16
    if y is None:
        y = torch.empty((M, N), dtype=dtype, device=like.device)
    _need(y, dtype, "y", (M, N))
    return y


def _weights(codes, d, m, K: int, group: int = GROUP) -> int:
    """Check the weight planes (d, m per `group` weights) for reduction
    length K; returns N."""
    torch = _torch()
    _need(codes, torch.uint8, "codes", (None, _div(K, 2)))
    N = codes.shape[0]
    _need(d, torch.float16, "d", (N, _div(K, group)))
    _need(m, torch.float16, "m", (N, _div(K, group)))
    return N


def _int8_acts(qa, dx, bsum):
    """Check int8 activation blocks (the output of q8_quantize_act); returns M, K."""
    torch = _torch()
    _need(qa, torch.int8, "qa", (None, None))
    M, K = qa.shape
    _need(dx, torch.float32, "dx", (M, _div(K, BLOCK)))
    _need(bsum, torch.int32, "bsum", (M, _div(K, BLOCK)))
    return M, K


def w4_gemv(codes, d, m, x, out_dtype=None, y=None, stream=None):
    """y[M,N] = x[M,K] @ dequant(W)^T for 1 <= M <= 8; x is bf16.
    out_dtype: torch.bfloat16 (default) or torch.float32; with a caller y and
    no out_dtype, y's dtype."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", (None, None))
    M, K = x.shape
    N = _weights(codes, d, m, K)
    oc = _out_code(out_dtype, y)
    y = _output(y, M, N, oc, x)
    _on_device(codes=codes, d=d, m=m, x=x, y=y)
    _check(load().w4_gemv(_ptr(codes), _ptr(d), _ptr(m), N, K, _ptr(x), M, _ptr(y), oc,
                          _stream(stream)), "w4_gemv")
    return y


def w4_gemv_g32(codes, d, m, x, out_dtype=None, y=None, stream=None):
    """w4_gemv for group-32 weights (w4_pack_g32 planes: d, m fp16[N,K/32]);
    y[M,N] = x[M,K] @ dequant(W)^T for 1 <= M <= 8, K % 32 == 0."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", (None, None))
    M, K = x.shape
    N = _weights(codes, d, m, K, GROUP32)
    oc = _out_code(out_dtype, y)
    y = _output(y, M, N, oc, x)
    _on_device(codes=codes, d=d, m=m, x=x, y=y)
    _check(load().w4_gemv_g32(_ptr(codes), _ptr(d), _ptr(m), N, K, _ptr(x), M, _ptr(y), oc,
                              _stream(stream)), "w4_gemv_g32")
    return y


def w4a8_gemv(codes, d, m, qa, dx, bsum, out_dtype=None, y=None, stream=None):
    """y[M,N] for 1 <= M <= 8 from W4-G256 weights and int8 activation blocks
    (the output of q8_quantize_act): exact int32 block dot products, scales in fp32."""
    M, K = _int8_acts(qa, dx, bsum)
    N = _weights(codes, d, m, K)
    oc = _out_code(out_dtype, y)
    y = _output(y, M, N, oc, qa)
    _on_device(codes=codes, d=d, m=m, qa=qa, dx=dx, bsum=bsum, y=y)
    _check(load().w4a8_gemv(_ptr(codes), _ptr(d), _ptr(m), N, K, _ptr(qa), _ptr(dx), _ptr(bsum),
                            M, _ptr(y), oc, _stream(stream)), "w4a8_gemv")
    return y


def w4a8_gemv_bf16(codes, d, m, x, out_dtype=None, y=None, stream=None):
    """w4a8_gemv with the quantiser folded in: bf16 x[M,K] (1 <= M <= 8) is
    quantised to int8 blocks inside the kernel; bit-identical to
    q8_quantize_act followed by w4a8_gemv."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", (None, None))
    M, K = x.shape
    N = _weights(codes, d, m, K)
    oc = _out_code(out_dtype, y)
    y = _output(y, M, N, oc, x)
    _on_device(codes=codes, d=d, m=m, x=x, y=y)
    _check(load().w4a8_gemv_bf16(_ptr(codes), _ptr(d), _ptr(m), N, K, _ptr(x), M, _ptr(y), oc,
                                 _stream(stream)), "w4a8_gemv_bf16")
    return y


def q8_quantize_act(x, qa=None, dx=None, bsum=None, stream=None):
    """bf16 x[M,K] (K % 32 == 0) -> (qa int8[M,K], dx fp32[M,K/32], bsum int32[M,K/32])."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", (None, None))
    M, K = x.shape
    if qa is None:
        qa = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if dx is None:
        dx = torch.empty((M, K // BLOCK), dtype=torch.float32, device=x.device)
    if bsum is None:
        bsum = torch.empty((M, K // BLOCK), dtype=torch.int32, device=x.device)
    _need(qa, torch.int8, "qa", (M, K))
    _need(dx, torch.float32, "dx", (M, _div(K, BLOCK)))
    _need(bsum, torch.int32, "bsum", (M, _div(K, BLOCK)))
    _on_device(x=x, qa=qa, dx=dx, bsum=bsum)
    _check(load().q8_quantize_act(_ptr(x), M, K, _ptr(qa), _ptr(dx), _ptr(bsum),
                                  _stream(stream)), "q8_quantize_act")
    return qa, dx, bsum


def w4a8_mmq_workspace_size(M: int, N: int, K: int) -> int:
    return int(load().w4a8_mmq_workspace_size(M, N, K))


def w4a8_mmq(codes, d, m, qa, dx, bsum, out_dtype=None, y=None, workspace=None, stream=None):
    """y[M,N] from W4-G256 weights and int8 activation blocks (tensor cores).
    workspace: optional uint8 1-D device tensor of at least
    w4a8_mmq_workspace_size(M, N, K) bytes (allocated here when omitted)."""
    torch = _torch()
    M, K = _int8_acts(qa, dx, bsum)
    N = _weights(codes, d, m, K)
    oc = _out_code(out_dtype, y)
    y = _output(y, M, N, oc, qa)
    placed = dict(codes=codes, d=d, m=m, qa=qa, dx=dx, bsum=bsum, y=y)
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace", (None,))
        placed["workspace"] = workspace
    _on_device(**placed)
    if workspace is None:
        ws_need = w4a8_mmq_workspace_size(M, N, K)
        if ws_need > 0:
            workspace = torch.empty(ws_need, dtype=torch.uint8, device=qa.device)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(load().w4a8_mmq(_ptr(codes), _ptr(d), _ptr(m), N, K, _ptr(qa), _ptr(dx), _ptr(bsum),
                           M, _ptr(y), oc, ws_ptr, ws_bytes, _stream(stream)), "w4a8_mmq")
    return y


def w4a8_mmq_static(codes, d, m, qa, dx, bsum, out_dtype=None, y=None, stream=None):
    """The W4A8 product without a workspace, for callers that cannot allocate
    device memory: the split-K scratch is the library's static device array
    (shared by every call on the device; overlapping calls must be serialised).
    Raises W4Error (W4_ERR_WORKSPACE) for shapes whose scratch need exceeds it.
    The C entry point allocates nothing; this wrapper allocates only the output
    (through torch) when `y` is omitted, so a caller that cannot allocate
    passes its own `y`."""
    M, K = _int8_acts(qa, dx, bsum)
    N = _weights(codes, d, m, K)
    oc = _out_code(out_dtype, y)
    y = _output(y, M, N, oc, qa)
    _on_device(codes=codes, d=d, m=m, qa=qa, dx=dx, bsum=bsum, y=y)
    _check(load().w4a8_mmq_static(_ptr(codes), _ptr(d), _ptr(m), N, K, _ptr(qa), _ptr(dx),
                                  _ptr(bsum), M, _ptr(y), oc, _stream(stream)), "w4a8_mmq_static")
    return y


def w4a8_mmq_blockdots(codes, d, m, qa, dx, bsum, out_dtype=None, y=None, stream=None):
    """w4a8_mmq that also returns the exact int32 block products
    P[M, N, K/32] read back from the kernel's tensor-memory accumulators (for
    tests of the integer core; much slower than w4a8_mmq).  Returns (y, P)."""
    torch = _torch()
    M, K = _int8_acts(qa, dx, bsum)
    N = _weights(codes, d, m, K)
    oc = _out_code(out_dtype, y)
    y = _output(y, M, N, oc, qa)
    _on_device(codes=codes, d=d, m=m, qa=qa, dx=dx, bsum=bsum, y=y)
    P = torch.empty((M, N, K // BLOCK), dtype=torch.int32, device=qa.device)
    ws_need = w4a8_mmq_workspace_size(M, N, K)
    ws = torch.empty(max(ws_need, 1), dtype=torch.uint8, device=qa.device) if ws_need else None
    _check(load().w4a8_mmq_blockdots(_ptr(codes), _ptr(d), _ptr(m), N, K, _ptr(qa), _ptr(dx),
                                     _ptr(bsum), M, _ptr(y), oc, _ptr(P),
                                     P.numel() * 4, _ptr(ws) if ws is not None else None,
                                     ws_need, _stream(stream)), "w4a8_mmq_blockdots")
    return y, P


def w4a8_gemv_blockdots(codes, d, m, qa, dx, bsum, out_dtype=None, y=None, stream=None):
    """w4a8_gemv (M <= 8) that also returns the exact int32 block products
    P[M, N, K/32] its integer core formed (for tests).  Returns (y, P)."""
    torch = _torch()
    M, K = _int8_acts(qa, dx, bsum)
    N = _weights(codes, d, m, K)
    oc = _out_code(out_dtype, y)
    y = _output(y, M, N, oc, qa)
    _on_device(codes=codes, d=d, m=m, qa=qa, dx=dx, bsum=bsum, y=y)
    P = torch.empty((M, N, K // BLOCK), dtype=torch.int32, device=qa.device)
    _check(load().w4a8_gemv_blockdots(_ptr(codes), _ptr(d), _ptr(m), N, K, _ptr(qa), _ptr(dx),
                                      _ptr(bsum), M, _ptr(y), oc, _ptr(P), P.numel() * 4,
                                      _stream(stream)), "w4a8_gemv_blockdots")
    return y, P



# ---------------------------------------------------------------------------
# microscaled 4-bit floating point
# ---------------------------------------------------------------------------

F4_FORMATS = {"mx": W4_F4_MX, "nv": W4_F4_NV}
F4_BLOCK = {W4_F4_MX: 32, W4_F4_NV: 16}


def _f4_format(format) -> int:
    if format in F4_FORMATS:
        return F4_FORMATS[format]
    raise ValueError(f"unknown format {format!r}, expected one of {sorted(F4_FORMATS)}")


def _in_code(x, name: str) -> int:
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype = x.dtype
    if dtype is torch.bfloat16:
        return W4_IN_BF16
    if dtype is torch.float32:
        return W4_IN_F32
    if dtype is torch.float16:
        return W4_IN_F16
    raise TypeError(f"{name} must be bfloat16, float16 or float32, got {dtype}")


# The small calls of these operators take a few microseconds on the GPU.  Plain
# calls (no y, workspace or stream of the caller's) with arguments that are right
# are therefore made by _f4call, an extension that checks, allocates and calls
# without the interpreter; it returns None for any other call, which then takes
# the way below: checks with a short path, and _need and _on_device to say what
# is wrong.  Without the extension every call does.
_ext = None


def _calls():
    """The extension, bound to the loaded library; False if it is not built, or
    not for this torch."""
    global _ext
    if _ext is None:
        import ctypes
        from .build import calls_tag
        torch, lib = _torch(), load()
        try:
            from . import _f4call as ext
        except ImportError:
            _ext = False
            return False
        if getattr(ext, "built_for", None) != calls_tag(torch.__version__):
            import warnings
            warnings.warn("_f4call.so was built for another torch or Python: run `python -m "
                          "w4_quant_matmul_b200.build` (calls of the f4 functions take the "
                          "slower way through ctypes)")
            _ext = False
            return False
        names = ("f4_tensor_scale", "f4_quantize", "f4_dequantize", "f4_embed", "f4_mm", "f4_gemv",
                 "f4_gemv_workspace_size")
        ext.init(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names),
                 torch.bfloat16, torch.float32)
        _ext = ext
    return _ext


def _is(t, dtype, shape) -> bool:
    """A plain contiguous tensor of this dtype and shape."""
    return (type(t) is _torch().Tensor and t.dtype is dtype and t.shape == shape
            and t.is_contiguous())


def _need2d(t, dtype, name: str):
    """_need for a matrix of any extents."""
    if not (type(t) is _torch().Tensor and t.dtype is dtype and t.dim() == 2
            and t.is_contiguous()):
        _need(t, dtype, name, (None, None))


def _run_on(stream, names, *tensors):
    """Check that all tensors (None: absent) are on the current device; the
    stream of the call as (torch stream or None for the current one, handle)."""
    torch = _torch()
    here = tensors[0].get_device()  # -1 on the CPU
    for t in tensors:
        if t is not None and t.get_device() != here:
            here = -1
            break
    if here < 0 or here != torch.cuda.current_device():
        _on_device(**{n: t for n, t in zip(names, tensors) if t is not None})
    if stream is None:
        # the handle behind torch.cuda.current_stream(), without building the object
        return None, torch._C._cuda_getCurrentRawStream(here)
    if stream.device != tensors[0].device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {tensors[0].device}")
    return stream, stream.cuda_stream


def _new(shape, dtype, like, stream):
    """An uninitialised tensor that belongs to the stream the call runs on: the
    allocator then hands its memory out again only in that stream's order."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _f4_scale_shape(R: int, K: int, format: int):
    """Shape of the scale plane: row tiles, tiles along K, bytes of a tile (the
    extent along K is open when K breaks the format)."""
    return (-(-R // 128), -(-K // (4 * F4_BLOCK[format])) if K % 32 == 0 else None, 512)


def _f4_planes(codes, scales, g, names, K=None):
    """Check the planes of one 4-bit matrix; returns rows, K, format."""
    torch = _torch()
    T, u8 = torch.Tensor, torch.uint8
    format, word = (W4_F4_MX, 128) if g is None else (W4_F4_NV, 64)
    if (type(codes) is T and codes.dtype is u8 and codes.dim() == 2 and codes.is_contiguous()
            and type(scales) is T and scales.dtype is u8 and scales.is_contiguous()):
        R, half = codes.shape
        k = 2 * half
        if (k % 32 == 0 and (K is None or K == k)
                and scales.shape == ((R + 127) // 128, (k + word - 1) // word, 512)
                and (g is None or _is(g, torch.float32, (1,)))):
            return R, k, format
    cn, sn, gn = names
    _need(codes, u8, cn, (None, None if K is None else _div(K, 2)))
    R = codes.shape[0]
    K = codes.shape[1] * 2 if K is None else K
    _need(scales, u8, sn, _f4_scale_shape(R, K, format))
    if g is not None:
        _need(g, torch.float32, gn, (1,))
    return R, K, format


def _f4_out(out_dtype, y, M: int, N: int):
    """Output code and dtype; the caller's y checked against [M,N]."""
    torch = _torch()
    if out_dtype is torch.bfloat16 or (out_dtype is None and y is None):
        oc, dtype = W4_OUT_BF16, torch.bfloat16
    else:
        oc = _out_code(out_dtype, y)
        dtype = torch.float32 if oc == W4_OUT_F32 else torch.bfloat16
    if y is not None and not _is(y, dtype, (M, N)):
        _need(y, dtype, "y", (M, N))
    return oc, dtype


def _opt(t):
    return None if t is None else t.data_ptr()


def f4_tensor_scale(x, g=None, stream=None):
    """Tensor scale of the NV format, max(amax / 2688, 2^-100) over the finite
    elements of x[R,K] (bf16, fp16 or fp32), as an fp32 tensor [1]."""
    torch = _torch()
    ic = _in_code(x, "x")
    _need2d(x, x.dtype, "x")
    if g is not None:
        _need(g, torch.float32, "g", (1,))
    st, handle = _run_on(stream, ("x", "g"), x, g)
    if g is None:
        g = _new((1,), torch.float32, x, st)
    _check(load().f4_tensor_scale(x.data_ptr(), ic, x.shape[0], x.shape[1], g.data_ptr(), handle),
           "f4_tensor_scale")
    return g


def f4_quantize(x, format="mx", tensor_scale=None, codes=None, scales=None, stream=None):
    """x[R,K] (bf16, fp16 or fp32; K % 32 == 0) -> 4-bit planes (codes
    uint8[R,K/2], scales uint8[ceil(R/128), ceil(K/(4*block)), 512], g).
    format: "mx" (blocks of 32, power-of-two scales; g is None) or "nv" (blocks
    of 16, e4m3 scales, g fp32[1]: `tensor_scale`, or found from x when
    omitted)."""
    torch = _torch()
    fc = _f4_format(format)
    if codes is None and scales is None and stream is None:
        out = (_ext or _calls()) and _ext.quantize(x, fc, tensor_scale)
        if out:
            return out
    ic = _in_code(x, "x")
    _need2d(x, x.dtype, "x")
    R, K = x.shape
    g = tensor_scale
    if g is not None:
        if fc == W4_F4_MX:
            raise ValueError("tensor_scale belongs to the nv format")
        if not _is(g, torch.float32, (1,)):
            _need(g, torch.float32, "tensor_scale", (1,))
    shape = _f4_scale_shape(R, K, fc)
    if codes is not None:
        _need(codes, torch.uint8, "codes", (R, _div(K, 2)))
    if scales is not None:
        _need(scales, torch.uint8, "scales", shape)
    st, handle = _run_on(stream, ("x", "tensor_scale", "codes", "scales"), x, g, codes, scales)
    if codes is None:
        codes = _new((R, K // 2), torch.uint8, x, st)
    if scales is None:
        scales = _new((shape[0], shape[1] or 0, 512), torch.uint8, x, st)
    if fc == W4_F4_NV and g is None:
        g = _new((1,), torch.float32, x, st)
        _check(load().f4_tensor_scale(x.data_ptr(), ic, R, K, g.data_ptr(), handle),
               "f4_tensor_scale")
    _check(load().f4_quantize(x.data_ptr(), ic, R, K, fc, _opt(g), codes.data_ptr(),
                              scales.data_ptr(), handle), "f4_quantize")
    return codes, scales, g


def f4_dequantize(codes, scales, g, out_dtype=None, y=None, stream=None):
    """The values y[R,K] that 4-bit planes stand for, bf16 (default) or fp32."""
    if y is None and stream is None and (_ext or _calls()):
        out = _ext.dequantize(codes, scales, g, out_dtype)
        if out is not None:
            return out
    R, K, fc = _f4_planes(codes, scales, g, ("codes", "scales", "g"))
    oc, dtype = _f4_out(out_dtype, y, R, K)
    st, handle = _run_on(stream, ("codes", "scales", "g", "y"), codes, scales, g, y)
    if y is None:
        y = _new((R, K), dtype, codes, st)
    _check(load().f4_dequantize(codes.data_ptr(), scales.data_ptr(), _opt(g), R, K, fc,
                                y.data_ptr(), oc, handle), "f4_dequantize")
    return y


def f4_embed(codes, scales, g, ids, scale=1.0, out_dtype=None, y=None, stream=None):
    """Embedding lookup: y[t] = scale * row ids[t] of the 4-bit table, for
    ids int64[T]; an id outside the table (padding) gives a row of zeros."""
    if y is None and stream is None and (_ext or _calls()):
        out = _ext.embed(codes, scales, g, ids, scale, out_dtype)
        if out is not None:
            return out
    torch = _torch()
    V, K, fc = _f4_planes(codes, scales, g, ("codes", "scales", "g"))
    if not (type(ids) is torch.Tensor and ids.dtype is torch.int64 and ids.dim() == 1
            and ids.is_contiguous()):
        _need(ids, torch.int64, "ids", (None,))
    T = ids.shape[0]
    oc, dtype = _f4_out(out_dtype, y, T, K)
    st, handle = _run_on(stream, ("codes", "scales", "g", "ids", "y"), codes, scales, g, ids, y)
    if y is None:
        y = _new((T, K), dtype, codes, st)
    _check(load().f4_embed(codes.data_ptr(), scales.data_ptr(), _opt(g), V, K, fc, ids.data_ptr(),
                           T, float(scale), y.data_ptr(), oc, handle), "f4_embed")
    return y


def f4_mm(codes, scales, g, qa, sa, ga, out_dtype=None, y=None, stream=None):
    """y[M,N] = A W^T from 4-bit weight planes (codes, scales, g) of W[N,K] and
    4-bit activation planes (qa, sa, ga) of A[M,K], both of one format
    (f4_quantize), on the block-scaled tensor cores."""
    if y is None and stream is None and (_ext or _calls()):
        out = _ext.mm(codes, scales, g, qa, sa, ga, out_dtype)
        if out is not None:
            return out
    N, K, fc = _f4_planes(codes, scales, g, ("codes", "scales", "g"))
    if (g is None) != (ga is None):
        raise ValueError("g and ga must both be given (nv) or both be None (mx)")
    M, _, _ = _f4_planes(qa, sa, ga, ("qa", "sa", "ga"), K)
    oc, dtype = _f4_out(out_dtype, y, M, N)
    st, handle = _run_on(stream, ("codes", "scales", "g", "qa", "sa", "ga", "y"),
                         codes, scales, g, qa, sa, ga, y)
    if y is None:
        y = _new((M, N), dtype, codes, st)
    _check(load().f4_mm(codes.data_ptr(), scales.data_ptr(), _opt(g), N, K, fc, qa.data_ptr(),
                        sa.data_ptr(), _opt(ga), M, y.data_ptr(), oc, handle), "f4_mm")
    return y


def f4_gemv_workspace_size(M: int, N: int, K: int, format="mx") -> int:
    """Bytes of workspace that f4_gemv needs on the current device; 0 where it needs
    none."""
    return int(load().f4_gemv_workspace_size(M, N, K, _f4_format(format)))


def f4_gemv(codes, scales, g, x, out_dtype=None, y=None, workspace=None, stream=None):
    """y[M,N] = x[M,K] W^T for 1 <= M <= 8 from 4-bit weight planes and bf16
    activations.  x is not quantised to 4 bits, but held in fixed point block by
    block (32 k for MX, 16 for NV): to 2^-22 of the block's largest magnitude, so that
    elements above 2^-14 of it are exact (NV: a block below 2^-17 of the token's
    largest is held as if it were of that size).  The weight planes are read before
    the kernel launched just before on the stream has ended: a kernel that writes them
    must not be that one if it lets its successor start early (programmatic dependent
    launch; f4_quantize and copies do not).  workspace:
    optional uint8 1-D device tensor of at least f4_gemv_workspace_size(M, N, K,
    format) bytes (allocated here when omitted); calls that can overlap on the GPU
    need one each."""
    if y is None and workspace is None and stream is None and (_ext or _calls()):
        out = _ext.gemv(codes, scales, g, x, out_dtype)
        if out is not None:
            return out
    torch = _torch()
    _need2d(x, torch.bfloat16, "x")
    M, K = x.shape
    N, _, fc = _f4_planes(codes, scales, g, ("codes", "scales", "g"), K)
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace", (None,))
    oc, dtype = _f4_out(out_dtype, y, M, N)
    st, handle = _run_on(stream, ("codes", "scales", "g", "x", "y", "workspace"),
                         codes, scales, g, x, y, workspace)
    if y is None:
        y = _new((M, N), dtype, codes, st)
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = workspace.numel()
    elif M > 1:  # a single token never needs any
        ws_bytes = load().f4_gemv_workspace_size(M, N, K, fc)
        if ws_bytes:
            workspace = _new((ws_bytes,), torch.uint8, x, st)
    _check(load().f4_gemv(codes.data_ptr(), scales.data_ptr(), _opt(g), N, K, fc, x.data_ptr(), M,
                          y.data_ptr(), oc, _opt(workspace), ws_bytes, handle), "f4_gemv")
    return y
