"""ctypes binding of libfq (the C ABI in include/fq.h): argument marshalling only.

Every function here checks tensor shapes/dtypes/devices, passes ``data_ptr()`` values and the
current CUDA stream to the C entry point of the same name, and raises FQError on a non-OK
status.  All computation happens in the CUDA kernels of libfq.so; there is no fallback: if the
library is missing, importing a compute function raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfq.so")

FQ_F16 = 0
FQ_F32 = 1
FQ_BF16 = 2
FQ_INDEX_EXACT = 0
FQ_INDEX_TOPC = 1
FQ_INDEX_TENSOR = 2
FQ_RESCALE_PLAIN = 0
FQ_RESCALE_MSE = 1
FQ_RESCALE_UNBIASED = 2

_c_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_i = ctypes.c_int

_SIGS = {
    "fq_abi_version": (_i, []),
    "fq_status_string": (ctypes.c_char_p, [_i]),
    "fq_padded_dim": (_i, [_i, _i]),
    "fq_payload_bytes": (_sz, [_i, _i, _i]),
    "fq_encode": (_i, [_vp, _i, _c_i64, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fq_decode": (_i, [_vp, _vp, _c_i64, _i, _i, _i, _vp, _vp, _vp, _i, _vp]),
    "fq_attn_workspace_bytes": (_sz, [_i, _i, _i, _c_i64, _i, _i]),
    "fq_attn_decode": (_i, [_vp, _i, _i, _i, _c_i64, _i,
                            _vp, _vp, _i, _i, _vp, _vp,
                            _vp, _vp, _i, _i, _vp, _vp,
                            ctypes.c_float, _vp, _vp, _sz, _vp]),
    "fq_build_search_index": (_i, [_vp, _i, _i, _i, _i, _i, _i, _vp, _sz,
                                   ctypes.POINTER(_sz)]),
    "fq_decode_gather": (_i, [_vp, _vp, _c_i64, _vp, _c_i64, _i, _i, _i, _vp, _vp, _vp, _i,
                              _vp]),
    "fq_attn_decode_lengths": (_i, [_vp, _i, _i, _i, _c_i64, _i, _vp,
                                    _vp, _vp, _i, _i, _vp, _vp,
                                    _vp, _vp, _i, _i, _vp, _vp,
                                    ctypes.c_float, _vp, _vp, _sz, _vp]),
    "fq_attn_decode_append": (_i, [_vp, _vp, _vp, _i, _i, _i, _c_i64, _i, _vp,
                                   _vp, _vp, _i, _i, _vp, _vp,
                                   _vp, _vp, _i, _i, _vp, _vp,
                                   ctypes.c_float, _vp, _vp, _sz, _vp]),
    "fq_encode_rho": (_i, [_vp, _i, _c_i64, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fq_decode_rescaled": (_i, [_vp, _vp, _vp, _c_i64, _i, _i, _i, _vp, _vp, _i, _vp, _i, _vp]),
    "fq_encode_prod": (_i, [_vp, _i, _c_i64, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fq_decode_prod": (_i, [_vp, _vp, _vp, _vp, _c_i64, _i, _i, _vp, _vp, _vp, _vp, _i, _vp]),
    "fq_wait_status": (_i, [ctypes.POINTER(ctypes.c_uint), _i]),
    "fq_selftest_wait_timeout": (_i, [ctypes.c_uint32, _vp]),
    "fq_attn_decode_noalloc": (_i, [_vp, _i, _i, _i, _c_i64, _i,
                                    _vp, _vp, _i, _i, _vp, _vp,
                                    _vp, _vp, _i, _i, _vp, _vp,
                                    ctypes.c_float, _vp, _vp]),
    "fq_kv4_unit_bytes": (_sz, [_i, _i]),
    "fq_page_step": (_i, [_vp, _vp, _i, _vp, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp,
                          _vp]),
    "fq_kv4_write": (_i, [_vp, _vp, _i, _c_i64, _i, _i, _c_i64, _c_i64, _c_i64, _c_i64, _vp, _vp,
                          _c_i64, _i, _i, _vp, _vp, _vp]),
    "fq_kv4_attn_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "fq_kv4_attn": (_i, [_vp, _i, _c_i64, _i, _i, _c_i64, _c_i64, _vp, _i, _i, _vp, _c_i64, _i, _i,
                         _i, _vp, _i, _vp, _i, ctypes.c_float, _vp, _vp, _sz, _vp]),
}

FQ_ATTN_NOALLOC_SCRATCH_BYTES = 4 << 20

_lib = None


class FQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: status {status} ({status_string(status)})")


def lib() -> ctypes.CDLL:
    """The loaded libfq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m random_access_kv_fq_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_symbols() -> list[str]:
    return list(_SIGS)


def status_string(status: int) -> str:
    return lib().fq_status_string(int(status)).decode()


def _check(fn: str, st: int) -> None:
    if st != 0:
        raise FQError(fn, st)


def fq_padded_dim(d: int, k: int) -> int:
    return int(lib().fq_padded_dim(d, k))


def fq_payload_bytes(d: int, k: int, N: int) -> int:
    return int(lib().fq_payload_bytes(d, k, N))


def fq_attn_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, d: int, kV: int) -> int:
    return int(lib().fq_attn_workspace_bytes(B, Hq, Hkv, T, d, kV))


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return FQ_F16
    if t.dtype == torch.float32:
        return FQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def fq_encode(x, rot, codebook, k: int, N: int, codes=None, norms=None, search_index=None,
              stream=None):
    """Encode rows of x [n, d] (fp16/fp32, CUDA).  Returns (codes uint8 [n, P], norms int16
    [n] holding fp16 bit patterns; view them with .view(torch.float16))."""
    import torch
    assert x.dim() == 2 and x.is_cuda and x.is_contiguous()
    n, d = x.shape
    P = fq_payload_bytes(d, k, N)
    if codes is None:
        codes = torch.empty((n, max(P, 1)), dtype=torch.uint8, device=x.device)
    if norms is None:
        norms = torch.empty((n,), dtype=torch.int16, device=x.device)
    st = lib().fq_encode(_ptr(x), _dtype_code(x), n, d, k, N, _ptr(rot), _ptr(codebook),
                         _ptr(codes), _ptr(norms), _ptr(search_index), _stream(stream))
    _check("fq_encode", st)
    return codes, norms


def fq_decode(codes, norms, rot, codebook, d: int, k: int, N: int, out_dtype=None, y=None,
              stream=None):
    """Decode n records into y [n, d] (fp32 by default, or fp16)."""
    import torch
    n = codes.shape[0]
    if y is None:
        y = torch.empty((n, d), dtype=out_dtype or torch.float32, device=codes.device)
    st = lib().fq_decode(_ptr(codes), _ptr(norms), n, d, k, N, _ptr(rot), _ptr(codebook),
                         _ptr(y), _dtype_code(y), _stream(stream))
    _check("fq_decode", st)
    return y


def fq_attn_decode(q, k_codes, k_norms, kK: int, NK: int, rotK, cbK, v_codes, v_norms,
                   kV: int, NV: int, rotV, cbV, scale: Optional[float] = None, out=None,
                   workspace=None, stream=None):
    """One decode-attention step.  q [B, Hq, d] fp16; k/v codes [B, Hkv, T, P]; norms
    [B, Hkv, T] (fp16 bits).  Returns out [B, Hq, d] fp32."""
    import torch
    B, Hq, d = q.shape
    _, Hkv, T, _ = k_codes.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    need = fq_attn_workspace_bytes(B, Hq, Hkv, T, d, kV)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().fq_attn_decode(_ptr(q), B, Hq, Hkv, T, d,
                              _ptr(k_codes), _ptr(k_norms), kK, NK, _ptr(rotK), _ptr(cbK),
                              _ptr(v_codes), _ptr(v_norms), kV, NV, _ptr(rotV), _ptr(cbV),
                              float(scale), _ptr(out), _ptr(workspace), ws_bytes,
                              _stream(stream))
    _check("fq_attn_decode", st)
    return out


def fq_decode_gather(codes, norms, token_ids, rot, codebook, d: int, k: int, N: int,
                     out_dtype=None, y=None, stream=None):
    """Decode the records at token_ids (int64 CUDA tensor, any order, repeats allowed) of the
    plane (codes [n, P], norms [n]) into y [len(token_ids), d]."""
    import torch
    n_ids = token_ids.numel()
    if y is None:
        y = torch.empty((n_ids, d), dtype=out_dtype or torch.float32, device=token_ids.device)
    assert token_ids.dtype == torch.int64 and token_ids.is_contiguous()
    st = lib().fq_decode_gather(_ptr(codes), _ptr(norms), codes.shape[0], _ptr(token_ids), n_ids,
                                d, k, N, _ptr(rot), _ptr(codebook), _ptr(y), _dtype_code(y),
                                _stream(stream))
    _check("fq_decode_gather", st)
    return y


def _attn_ws(q, B, Hq, Hkv, T, d, kV, workspace):
    import torch
    need = fq_attn_workspace_bytes(B, Hq, Hkv, T, d, kV)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return workspace, ws_bytes


def fq_attn_decode_lengths(q, lengths, k_codes, k_norms, kK: int, NK: int, rotK, cbK, v_codes,
                           v_norms, kV: int, NV: int, rotV, cbV, scale: Optional[float] = None,
                           out=None, workspace=None, stream=None):
    """fq_attn_decode with per-sequence context lengths (int32 CUDA tensor [B])."""
    import torch
    B, Hq, d = q.shape
    _, Hkv, T, _ = k_codes.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    assert lengths.dtype == torch.int32 and lengths.numel() == B
    workspace, ws_bytes = _attn_ws(q, B, Hq, Hkv, T, d, kV, workspace)
    st = lib().fq_attn_decode_lengths(_ptr(q), B, Hq, Hkv, T, d, _ptr(lengths),
                                      _ptr(k_codes), _ptr(k_norms), kK, NK, _ptr(rotK), _ptr(cbK),
                                      _ptr(v_codes), _ptr(v_norms), kV, NV, _ptr(rotV), _ptr(cbV),
                                      float(scale), _ptr(out), _ptr(workspace), ws_bytes,
                                      _stream(stream))
    _check("fq_attn_decode_lengths", st)
    return out


def fq_attn_decode_append(q, k_new, v_new, lengths, k_codes, k_norms, kK: int, NK: int, rotK,
                          cbK, v_codes, v_norms, kV: int, NV: int, rotV, cbV,
                          scale: Optional[float] = None, out=None, workspace=None, stream=None):
    """One decode step that encodes its own key/value (fp16 [B, Hkv, d]) into slot lengths[b]
    of the caches (in place), attends over lengths[b] + 1 tokens and advances lengths."""
    import torch
    B, Hq, d = q.shape
    _, Hkv, T, _ = k_codes.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    assert lengths.dtype == torch.int32 and lengths.numel() == B
    assert k_new.shape == (B, Hkv, d) and v_new.shape == (B, Hkv, d)
    workspace, ws_bytes = _attn_ws(q, B, Hq, Hkv, T, d, kV, workspace)
    st = lib().fq_attn_decode_append(_ptr(q), _ptr(k_new), _ptr(v_new), B, Hq, Hkv, T, d,
                                     _ptr(lengths), _ptr(k_codes), _ptr(k_norms), kK, NK,
                                     _ptr(rotK), _ptr(cbK), _ptr(v_codes), _ptr(v_norms), kV, NV,
                                     _ptr(rotV), _ptr(cbV), float(scale), _ptr(out),
                                     _ptr(workspace), ws_bytes, _stream(stream))
    _check("fq_attn_decode_append", st)
    return out


def fq_attn_decode_noalloc(q, k_codes, k_norms, kK: int, NK: int, rotK, cbK, v_codes, v_norms,
                           kV: int, NV: int, rotV, cbV, scale: Optional[float] = None, out=None,
                           stream=None):
    """fq_attn_decode without a workspace argument: the library's fixed per-GPU scratch holds
    the partials (for callers that cannot allocate device memory)."""
    import torch
    B, Hq, d = q.shape
    _, Hkv, T, _ = k_codes.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    st = lib().fq_attn_decode_noalloc(_ptr(q), B, Hq, Hkv, T, d,
                                      _ptr(k_codes), _ptr(k_norms), kK, NK, _ptr(rotK), _ptr(cbK),
                                      _ptr(v_codes), _ptr(v_norms), kV, NV, _ptr(rotV), _ptr(cbV),
                                      float(scale), _ptr(out), _stream(stream))
    _check("fq_attn_decode_noalloc", st)
    return out


def fq_encode_rho(x, rot, codebook, k: int, N: int, search_index=None, stream=None):
    """fq_encode plus the rho plane of the target-aware rescale.  Returns (codes, norms, rho);
    norms and rho hold fp16 bit patterns."""
    import torch
    assert x.dim() == 2 and x.is_cuda and x.is_contiguous()
    n, d = x.shape
    P = fq_payload_bytes(d, k, N)
    codes = torch.empty((n, max(P, 1)), dtype=torch.uint8, device=x.device)
    norms = torch.empty((n,), dtype=torch.int16, device=x.device)
    rho = torch.empty((n,), dtype=torch.int16, device=x.device)
    st = lib().fq_encode_rho(_ptr(x), _dtype_code(x), n, d, k, N, _ptr(rot), _ptr(codebook),
                             _ptr(codes), _ptr(norms), _ptr(rho), _ptr(search_index),
                             _stream(stream))
    _check("fq_encode_rho", st)
    return codes, norms, rho


def fq_decode_rescaled(codes, norms, rho, rot, codebook, d: int, k: int, N: int, rule: int,
                       out_dtype=None, stream=None):
    import torch
    n = codes.shape[0]
    y = torch.empty((n, d), dtype=out_dtype or torch.float32, device=codes.device)
    st = lib().fq_decode_rescaled(_ptr(codes), _ptr(norms), _ptr(rho), n, d, k, N, _ptr(rot),
                                  _ptr(codebook), rule, _ptr(y), _dtype_code(y), _stream(stream))
    _check("fq_decode_rescaled", st)
    return y


def fq_encode_prod(x, rot, c1, qjl, stream=None):
    """TurboQuant_prod encode.  Returns (codes, signs, norms, gamma)."""
    import torch
    assert x.dim() == 2 and x.is_cuda and x.is_contiguous()
    n, d = x.shape
    N1 = c1.numel()
    P1 = fq_payload_bytes(d, 1, N1)
    codes = torch.empty((n, max(P1, 1)), dtype=torch.uint8, device=x.device)
    signs = torch.empty((n, (d + 7) // 8), dtype=torch.uint8, device=x.device)
    norms = torch.empty((n,), dtype=torch.int16, device=x.device)
    gamma = torch.empty((n,), dtype=torch.int16, device=x.device)
    st = lib().fq_encode_prod(_ptr(x), _dtype_code(x), n, d, N1, _ptr(rot), _ptr(c1), _ptr(qjl),
                              _ptr(codes), _ptr(signs), _ptr(norms), _ptr(gamma), _stream(stream))
    _check("fq_encode_prod", st)
    return codes, signs, norms, gamma


def fq_decode_prod(codes, signs, norms, gamma, rot, c1, qjl, d: int, out_dtype=None,
                   stream=None):
    import torch
    n = codes.shape[0]
    y = torch.empty((n, d), dtype=out_dtype or torch.float32, device=codes.device)
    st = lib().fq_decode_prod(_ptr(codes), _ptr(signs), _ptr(norms), _ptr(gamma), n, d,
                              c1.numel(), _ptr(rot), _ptr(c1), _ptr(qjl), _ptr(y), _dtype_code(y),
                              _stream(stream))
    _check("fq_decode_prod", st)
    return y


def fq_wait_status(clear: bool = False) -> int:
    """Number of CTAs whose bounded device-side waits gave up on the current device (waits for
    the device first).  0 means no launch since the last clear lost a wait."""
    n = ctypes.c_uint(0)
    st = lib().fq_wait_status(ctypes.byref(n), 1 if clear else 0)
    if st not in (0, 6):
        _check("fq_wait_status", st)
    return int(n.value)


def fq_build_search_index(codebook, d: int, k: int, N: int, kind: int, L: int,
                          c: int) -> np.ndarray:
    """Build the grid candidate index on the host; returns a uint8 numpy buffer to upload."""
    cb = np.ascontiguousarray(np.asarray(codebook, dtype=np.float32))
    need = _sz(0)
    st = lib().fq_build_search_index(cb.ctypes.data, d, k, N, kind, L, c, None, 0,
                                     ctypes.byref(need))
    if st not in (0, 4):
        _check("fq_build_search_index", st)
    buf = np.zeros(int(need.value), dtype=np.uint8)
    st = lib().fq_build_search_index(cb.ctypes.data, d, k, N, kind, L, c, buf.ctypes.data,
                                     buf.size, ctypes.byref(need))
    _check("fq_build_search_index", st)
    return buf


# ---- the 4-bit paged cache ---------------------------------------------------------------------

# These calls take microseconds of GPU time, so the checks below are kept to cheap attribute reads and
# the common case (the current device's current stream) goes straight through.  Sizes go to new_empty
# as numbers, not as a tuple: 1.4 us instead of 1.9 to 2.3.

class _Torch:
    """What the calls below need of torch, looked up once."""

    def __init__(self):
        import torch
        self.device, self.raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self.int32, self.uint8 = torch.int32, torch.uint8
        self.types = {torch.float16: FQ_F16, torch.float32: FQ_F32, torch.bfloat16: FQ_BF16}


_torch = None
_KV4_SIZES = {}  # arguments of the size functions -> bytes


def _t() -> _Torch:
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _kv4_size(fn, *args) -> int:
    n = _KV4_SIZES.get((fn, args))
    if n is None:
        if len(_KV4_SIZES) > 4096:
            _KV4_SIZES.clear()
        n = _KV4_SIZES[fn, args] = int(getattr(lib(), fn)(*args))
    return n


class _OnStream:
    """Makes a stream and its device current, so that what a call allocates belongs to the stream
    that uses it."""

    def __init__(self, device: int, stream):
        import torch
        if device < 0:
            raise ValueError("expected CUDA tensors")
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif isinstance(stream, int):
            # 0 is the legacy default stream, which torch knows as its default stream
            stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                      else torch.cuda.default_stream(device))
        if stream.device.index != device:
            raise ValueError(f"a stream of {stream.device} for tensors on device {device}")
        self._ctx = torch.cuda.stream(stream)

    def __enter__(self):
        self._ctx.__enter__()

    def __exit__(self, *exc):
        return self._ctx.__exit__(*exc)


def _same_device(device: int, *tensors) -> None:
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("tensors on different devices")


def _int32(name, t, shape):
    if t.dtype is not _torch.int32 or not t.is_contiguous():
        raise TypeError(f"{name}: a contiguous int32 tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _kv4_type(t) -> int:
    code = _torch.types.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _kv4_cache(cache, d: int, group: int):
    """(n_blocks, Hkv, page) of a cache tensor [n_blocks, Hkv, page / 16, unit bytes]."""
    if cache.dtype is not _torch.uint8 or not cache.is_contiguous():
        raise TypeError("cache: a contiguous uint8 tensor [n_blocks, Hkv, page / 16, unit bytes]")
    n_blocks, hkv, units, size = cache.shape
    unit = _kv4_size("fq_kv4_unit_bytes", d, group)
    if unit == 0:
        raise FQError("fq_kv4_unit_bytes", 2)
    if size != unit:
        raise ValueError(f"cache: units of {size} bytes, expected {unit}")
    return n_blocks, hkv, 16 * units


def fq_kv4_unit_bytes(d: int, group: int) -> int:
    return int(lib().fq_kv4_unit_bytes(d, group))


def fq_kv4_attn_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, max_q: int, max_blocks: int,
                                page: int) -> int:
    return int(lib().fq_kv4_attn_workspace_bytes(B, Hq, Hkv, d, max_q, max_blocks, page))


def fq_page_step(lens, new_lens, block_tables, free_list, free_count, page: int, n_slots: int,
                 lens_out=None, free_count_out=None, stream=None):
    """One step of a paged cache's book-keeping (int32 CUDA tensors): requests of lens [B] tokens
    add new_lens [B] (negative: end) and grow block_tables [B, max_blocks] from the stack
    free_list[:free_count]; tables and free list are updated in place, free_count too unless
    free_count_out is given.  Returns (lens_out [B], cu_new [B + 1], slots [n_slots], refused [1]);
    the rows of refused requests in this step's attention mean nothing."""
    tt = _t()
    dev = lens.get_device()
    _same_device(dev, new_lens, block_tables, free_list, free_count, lens_out, free_count_out)
    if stream is not None or dev < 0 or tt.device() != dev:
        with _OnStream(dev, stream):
            return fq_page_step(lens, new_lens, block_tables, free_list, free_count, page, n_slots,
                                lens_out, free_count_out)
    B, max_blocks = block_tables.shape
    n_blocks = free_list.numel()
    _int32("lens", lens, (B,))
    _int32("new_lens", new_lens, (B,))
    _int32("block_tables", block_tables, (B, max_blocks))
    _int32("free_list", free_list, (n_blocks,))
    _int32("free_count", free_count, (1,))
    if n_slots < 0:
        raise ValueError("n_slots: at least 0")
    count_in = count_out = free_count.data_ptr()
    if free_count_out is not None:
        _int32("free_count_out", free_count_out, (1,))
        count_out = free_count_out.data_ptr()
    # the outputs in one allocation
    if lens_out is None:
        slots, cu_new, lens_out, refused = lens.new_empty(n_slots + 2 * B + 2).unsafe_split_with_sizes(
            (n_slots, B + 1, B, 1))
    else:
        _int32("lens_out", lens_out, (B,))
        slots, cu_new, refused = lens.new_empty(n_slots + B + 2).unsafe_split_with_sizes(
            (n_slots, B + 1, 1))
    st = lib().fq_page_step(lens.data_ptr(), new_lens.data_ptr(), B, block_tables.data_ptr(),
                            max_blocks, page, free_list.data_ptr(), n_blocks, count_in,
                            lens_out.data_ptr(), count_out, cu_new.data_ptr(), slots.data_ptr(),
                            n_slots, refused.data_ptr(), tt.raw_stream(dev))
    if st:
        _check("fq_page_step", st)
    return lens_out, cu_new, slots, refused


def fq_kv4_write(k, v, slots, cache, group: int, values: bool = False, stream=None):
    """Quantise k and v [n, Hkv, d] (fp16, bf16 or fp32, last axis contiguous) to 4 bits and write
    them at slots [n] (int32; tokens with a slot outside the pool are skipped) of the cache
    [n_blocks, Hkv, page / 16, unit bytes].  With values=True returns the quantised values
    (k_values, v_values) [n, Hkv, d] in the inputs' type."""
    tt = _t()
    dev = k.get_device()
    if v.get_device() != dev or slots.get_device() != dev or cache.get_device() != dev:
        raise ValueError("tensors on different devices")
    if stream is not None or dev < 0 or tt.device() != dev:
        with _OnStream(dev, stream):
            return fq_kv4_write(k, v, slots, cache, group, values)
    if k.shape != v.shape or k.dtype is not v.dtype:
        raise ValueError("k and v: two tensors [n, Hkv, d] of one type")
    n, hkv, d = k.shape
    k0, k1, k2 = k.stride()
    v0, v1, v2 = v.stride()
    if n > 0 and (k2 != 1 or v2 != 1):
        raise ValueError("k and v: the last axis has to be contiguous")
    _int32("slots", slots, (n,))
    n_blocks, cache_hkv, page = _kv4_cache(cache, d, group)
    if cache_hkv != hkv:
        raise ValueError(f"cache of {cache_hkv} kv heads, keys of {hkv}")
    kind = _kv4_type(k)
    kv = vv = kp = vp = None
    if values:
        kv, vv = k.new_empty(n, hkv, d), k.new_empty(n, hkv, d)
        kp, vp = kv.data_ptr(), vv.data_ptr()
    st = lib().fq_kv4_write(k.data_ptr(), v.data_ptr(), kind, n, hkv, d, k0, k1, v0, v1,
                            slots.data_ptr(), cache.data_ptr(), n_blocks, page, group, kp, vp,
                            tt.raw_stream(dev))
    if st:
        _check("fq_kv4_write", st)
    return (kv, vv) if values else None


def fq_kv4_attn(q, cache, block_tables, kv_lens, group: int, cu_q=None, max_q: Optional[int] = None,
                window: int = 0, scale: Optional[float] = None, out=None, workspace=None,
                stream=None):
    """Causal attention of q [n_q, Hq, d] (fp16 or bf16, last axis contiguous) over the 4-bit cache
    [n_blocks, Hkv, page / 16, unit bytes] through block_tables [B, max_blocks] and kv_lens [B]
    (int32).  cu_q [B + 1] (int32) gives the sequences' rows of q, at most max_q each, which has to be
    given then; without it every sequence has one.  window > 0: only the last `window` tokens are
    seen.  Returns out [n_q, Hq, d] of q's type; rows that no sequence has are not written (of a new
    `out` they hold anything)."""
    if max_q is None:
        if cu_q is not None:
            raise ValueError("max_q: the most query tokens that cu_q gives a sequence")
        max_q = 1
    tt = _t()
    dev = q.get_device()
    _same_device(dev, cache, block_tables, kv_lens, cu_q, out, workspace)
    if stream is not None or dev < 0 or tt.device() != dev:
        with _OnStream(dev, stream):
            return fq_kv4_attn(q, cache, block_tables, kv_lens, group, cu_q, max_q, window, scale,
                               out, workspace)
    n_q, hq, d = q.shape
    q0, q1, q2 = q.stride()
    if n_q > 0 and q2 != 1:
        raise ValueError("q: the last axis has to be contiguous")
    n_blocks, hkv, page = _kv4_cache(cache, d, group)
    B, max_blocks = block_tables.shape
    _int32("block_tables", block_tables, (B, max_blocks))
    _int32("kv_lens", kv_lens, (B,))
    cu = None
    if cu_q is not None:
        _int32("cu_q", cu_q, (B + 1,))
        cu = cu_q.data_ptr()
    kind = _kv4_type(q)
    if out is None:
        out = q.new_empty(n_q, hq, d)
    elif out.shape != q.shape or out.dtype is not q.dtype or not out.is_contiguous():
        raise ValueError("out: a contiguous tensor of q's shape and type")
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():  # its elements would not be all that lies between its ends, nor need be there
            raise ValueError("workspace: a contiguous tensor")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        ws_bytes = _kv4_size("fq_kv4_attn_workspace_bytes", B, hq, hkv, d, max_q, max_blocks, page)
        if ws_bytes:
            workspace = cache.new_empty(ws_bytes)
            ws = workspace.data_ptr()
    st = lib().fq_kv4_attn(q.data_ptr(), kind, n_q, hq, d, q0, q1, cu, B, max_q, cache.data_ptr(),
                           n_blocks, hkv, page, group, block_tables.data_ptr(), max_blocks,
                           kv_lens.data_ptr(), window, d ** -0.5 if scale is None else scale,
                           out.data_ptr(), ws, ws_bytes, tt.raw_stream(dev))
    if st:
        _check("fq_kv4_attn", st)
    return out
