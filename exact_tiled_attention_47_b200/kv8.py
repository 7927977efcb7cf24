"""Paged cache held in 8 bits: the binding of ``fa_kv8_append`` and ``fa_kv8_attend``, and helpers.

A cache is four tensors, ``k_pages``/``v_pages`` [num_pages, Hkv, page_size, D] of codes
(torch.float8_e4m3fn or torch.int8) and ``k_scales``/``v_scales`` fp32 [num_pages, Hkv, page_size / 16];
a code stands for code * scale.  The functions named like the C entry points only marshal arguments;
the helpers check tensors, allocate outputs and raise on errors, as those of the package do.
"""
from __future__ import annotations

import contextlib
import functools

import exact_tiled_attention_47_b200 as fa

from . import _lib
from ._lib import load

_TORCH = _INT32 = _FLOAT32 = _CODES = _FLOATS = None


def _torch():
    """torch, imported on first use as everywhere in the package; sets the types that the checks compare with."""
    global _TORCH, _INT32, _FLOAT32, _CODES, _FLOATS
    if _TORCH is None:
        import torch
        _INT32, _FLOAT32 = torch.int32, torch.float32
        _CODES = {torch.float8_e4m3fn: fa.FA_E4M3, torch.int8: fa.FA_INT8}
        _FLOATS = {torch.bfloat16: fa.FA_BF16, torch.float16: fa.FA_FP16, torch.float32: fa.FA_FP32}
        _TORCH = torch
    return _TORCH


def _types():
    """{code dtype: its number}, {16-bit or output dtype: its number}."""
    _torch()
    return _CODES, _FLOATS


def fa_kv8_append(k, v, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, new_lens, B, Nt, Hkv, num_pages,
                  page_size, pages_per_seq, D, stream=None, in_dtype=None, kv_dtype=None) -> int:
    """Marshal to the C ``fa_kv8_append``; returns its status.  Dtypes default to those of k and k_pages."""
    codes, floats = _types()
    p = fa._ptr
    return load().fa_kv8_append(p(k), p(v), p(k_pages), p(v_pages), p(k_scales), p(v_scales), p(block_table), p(seqlens_k),
                                p(new_lens), int(B), int(Nt), int(Hkv), int(num_pages), int(page_size), int(pages_per_seq), int(D),
                                fa._stream(stream), floats.get(k.dtype, -1) if in_dtype is None else int(in_dtype),
                                codes.get(k_pages.dtype, -1) if kv_dtype is None else int(kv_dtype))


def fa_kv8_attend_workspace_bytes(B, Nq, Hq, Hkv, D) -> int:
    return int(load().fa_kv8_attend_workspace_bytes(int(B), int(Nq), int(Hq), int(Hkv), int(D)))


def fa_kv8_attend(q, k_pages, v_pages, k_scales, v_scales, block_table, o, lse, B, Nq, Hq, Hkv, num_pages, page_size,
                  pages_per_seq, D, scale, seqlens_k, workspace, workspace_bytes=None, stream=None, in_dtype=None, kv_dtype=None,
                  o_dtype=None) -> int:
    """Marshal to the C ``fa_kv8_attend``; returns its status.  Dtypes default to those of q, k_pages and o."""
    codes, floats = _types()
    p = fa._ptr
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return load().fa_kv8_attend(p(q), p(k_pages), p(v_pages), p(k_scales), p(v_scales), p(block_table), p(o), p(lse), int(B), int(Nq),
                                int(Hq), int(Hkv), int(num_pages), int(page_size), int(pages_per_seq), int(D), float(scale),
                                p(seqlens_k), p(workspace), int(workspace_bytes), fa._stream(stream),
                                floats.get(q.dtype, -1) if in_dtype is None else int(in_dtype),
                                codes.get(k_pages.dtype, -1) if kv_dtype is None else int(kv_dtype),
                                floats.get(o.dtype, -1) if o_dtype is None else int(o_dtype))


@contextlib.contextmanager
def _on(device, stream):
    with _TORCH.cuda.device(device), contextlib.nullcontext() if stream is None else _TORCH.cuda.stream(stream):
        yield


def place_of(device, stream):
    """(context, raw stream) of a helper's call on tensors of this device: entered (in_context), the context makes their
    device and the caller's stream current, so that what the helper allocates belongs to the stream its kernels run on;
    it is None where both already are.  Nothing is entered here: a helper may still return or refuse."""
    if stream is None and device.type == "cuda" and device.index == _torch().cuda.current_device():
        return None, _TORCH._C._cuda_getCurrentRawStream(device.index)
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    cuda = _TORCH.cuda
    if stream is None:
        return _on(device, None), cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        stream = cuda.ExternalStream(stream, device=device) if stream else cuda.default_stream(device)
    if stream.device != device:
        raise ValueError("the stream belongs to another device than the tensors")
    return _on(device, stream), stream.cuda_stream


def in_context(context, f, *args):
    """f(*args) inside a context of place_of()."""
    if context is None:
        return f(*args)
    with context:
        return f(*args)


def alike(t, dtype, shape, device):
    return t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()


def check_tensor(name, t, dtype, shape, device):
    """Raises ValueError unless t is a contiguous tensor of this dtype, shape and device."""
    if not alike(t, dtype, shape, device):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {list(shape)} on {device}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device} with strides {list(t.stride())}")


def _check_cache(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, Hkv, D, device):
    """(num_pages, Hkv, page_size, pages_per_seq, code type) of a cache; ValueError unless its tensors fit together."""
    _torch()
    dtype, shape, table = k_pages.dtype, k_pages.shape, block_table.shape
    code = _CODES.get(dtype)
    if code is None or len(shape) != 4:
        raise ValueError("k_pages: expected [num_pages, Hkv, page_size, D] of torch.float8_e4m3fn or torch.int8")
    num_pages, heads, page_size, dim = shape
    if (Hkv is not None and heads != Hkv) or dim != D:
        raise ValueError(f"k_pages {list(shape)} does not hold the given heads or head dimension")
    if len(table) != 2:
        raise ValueError("block_table: expected [B, pages_per_seq]")
    scales = (num_pages, heads, page_size // 16)
    if not (alike(k_pages, dtype, shape, device) and alike(v_pages, dtype, shape, device) and alike(k_scales, _FLOAT32, scales, device)
            and alike(v_scales, _FLOAT32, scales, device) and alike(block_table, _INT32, table, device) and table[0] == B
            and (seqlens_k is None or alike(seqlens_k, _INT32, (B,), device))):
        check_tensor("k_pages", k_pages, dtype, shape, device)
        check_tensor("v_pages", v_pages, dtype, shape, device)
        check_tensor("k_scales", k_scales, _FLOAT32, scales, device)
        check_tensor("v_scales", v_scales, _FLOAT32, scales, device)
        check_tensor("block_table", block_table, _INT32, (B, table[1]), device)
        check_tensor("seqlens_k", seqlens_k, _INT32, (B,), device)
    return num_pages, heads, page_size, table[1], code


def new_kv8_cache(num_pages, page_size, Hkv, D, dtype=None, device="cuda"):
    """(k_pages, v_pages, k_scales, v_scales) of an empty cache; dtype torch.float8_e4m3fn (default) or torch.int8."""
    import torch
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    if dtype not in _types()[0]:
        raise ValueError("dtype: torch.float8_e4m3fn or torch.int8")
    if page_size < 16 or page_size > 65536 or page_size & (page_size - 1):
        raise ValueError("page_size: a power of two from 16 to 65536")
    codes = [torch.zeros((num_pages, Hkv, page_size, D), dtype=torch.int8, device=device).view(dtype) for _ in range(2)]
    return (*codes, *(torch.zeros((num_pages, Hkv, page_size // 16), dtype=torch.float32, device=device) for _ in range(2)))


def append_kv8(k, v, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, new_lens=None, stream=None):
    """Quantise new rows k, v [B, Nt, Hkv, D] into the cache, in place.

    ``seqlens_k`` int32 [B]: the lengths with the new rows included; the first ``new_lens[b]`` (int32 [B]; None: all
    Nt) rows of item b become its last keys.  Rows in a strided k or v are copied together first.
    """
    B, Nt, Hkv, D = shape = k.shape
    dev, dtype = k.device, k.dtype
    num_pages, _, page_size, pps, code = _check_cache(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, Hkv, D, dev)
    if seqlens_k is None:
        raise ValueError("seqlens_k: an int32 tensor [B], the lengths with the new rows included")
    if new_lens is not None:
        check_tensor("new_lens", new_lens, _INT32, (B,), dev)
    if v.dtype is not dtype or v.shape != shape or v.device != dev:
        raise ValueError("k and v must be alike")
    context, raw = place_of(dev, stream)
    if context is not None or not (k.is_contiguous() and v.is_contiguous()):
        with context or contextlib.nullcontext():
            k, v = k.contiguous(), v.contiguous()
            st = fa_kv8_append(k, v, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, new_lens, B, Nt, Hkv, num_pages,
                               page_size, pps, D, raw)
    else:
        st = (_lib._lib or load()).fa_kv8_append(
            k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
            block_table.data_ptr(), seqlens_k.data_ptr(), None if new_lens is None else new_lens.data_ptr(), B, Nt, Hkv, num_pages,
            page_size, pps, D, raw, _FLOATS.get(dtype, -1), code)
    if st != fa.FA_OK:
        raise fa.FAError(st, "fa_kv8_append")


@functools.lru_cache(maxsize=256)
def _workspace_bytes(*sizes):
    return max(1, fa_kv8_attend_workspace_bytes(*sizes))


def attend_kv8(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k=None, scale=None, out_dtype=None, workspace=None,
               stream=None):
    """O [B,Nq,Hq,D], LSE [B,Hq,Nq] of the newest Nq tokens q of each sequence over its 8-bit cache.

    ``block_table`` int32 [B, pages_per_seq]; ``seqlens_k`` int32 [B] (keys of each sequence, those of the Nq tokens
    included) or None (every table entry in use).  Query i of item b sees keys up to seqlens_k[b] - Nq + i.
    """
    B, Nq, Hq, D = q.shape
    dev, dtype = q.device, q.dtype
    num_pages, Hkv, page_size, pps, code = _check_cache(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, None, D, dev)
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError("workspace: expected a contiguous tensor on the device of q")
    context, raw = place_of(dev, stream)

    def call():
        rq = q if q.is_contiguous() else q.contiguous()
        if workspace is None:
            size = _workspace_bytes(B, Nq, Hq, Hkv, D)
            ws = rq.new_empty(size, dtype=_TORCH.uint8)
        else:
            ws, size = workspace, workspace.nbytes
        o = _TORCH.empty_like(rq) if out_dtype is None else _TORCH.empty_like(rq, dtype=out_dtype)
        lse = rq.new_empty((B, Hq, Nq), dtype=_FLOAT32)
        return (_lib._lib or load()).fa_kv8_attend(
            rq.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block_table.data_ptr(),
            o.data_ptr(), lse.data_ptr(), B, Nq, Hq, Hkv, num_pages, page_size, pps, D, D ** -0.5 if scale is None else scale,
            None if seqlens_k is None else seqlens_k.data_ptr(), ws.data_ptr(), size, raw, _FLOATS.get(dtype, -1), code,
            _FLOATS.get(o.dtype, -1)), o, lse

    st, o, lse = call() if context is None else in_context(context, call)
    if st != fa.FA_OK:
        raise fa.FAError(st, "fa_kv8_attend")
    return o, lse
