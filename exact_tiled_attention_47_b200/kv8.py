"""Paged cache held in 8 bits: the binding of ``fa_kv8_append`` and ``fa_kv8_attend``, and helpers.

A cache is four tensors, ``k_pages``/``v_pages`` [num_pages, Hkv, page_size, D] of codes
(torch.float8_e4m3fn or torch.int8) and ``k_scales``/``v_scales`` fp32 [num_pages, Hkv, page_size / 16];
a code stands for code * scale.  The functions named like the C entry points only marshal arguments;
the helpers check tensors, allocate outputs and raise on errors, as those of the package do.
"""
from __future__ import annotations

import contextlib
import functools
import math

import exact_tiled_attention_47_b200 as fa

from . import _lib
from ._lib import load

_CODES = None
_FLOATS = None


def _types():
    """{code dtype: its number}, {16-bit or output dtype: its number} (torch is imported on first use)."""
    global _CODES, _FLOATS
    if _CODES is None:
        import torch
        _CODES = {torch.float8_e4m3fn: fa.FA_E4M3, torch.int8: fa.FA_INT8}
        _FLOATS = {torch.bfloat16: fa.FA_BF16, torch.float16: fa.FA_FP16, torch.float32: fa.FA_FP32}
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


def enter(device, stream):
    """(context, raw stream) of a helper's call on tensors of this device: the context makes their device and
    the caller's stream current, so that what the helper allocates belongs to the stream its kernels run on;
    it is None where both already are."""
    import torch
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if stream is None and device.index == torch.cuda.current_device():
        return None, torch._C._cuda_getCurrentRawStream(device.index)
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(device))
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError("the stream belongs to another device than the tensors")
        stack.enter_context(torch.cuda.stream(stream))
    return stack, torch.cuda.current_stream(device).cuda_stream


def in_context(context, f, *args):
    """f(*args) inside a context of enter()."""
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
    import torch
    code = _types()[0].get(k_pages.dtype)
    shape = k_pages.shape
    if code is None or len(shape) != 4:
        raise ValueError("k_pages: expected [num_pages, Hkv, page_size, D] of torch.float8_e4m3fn or torch.int8")
    num_pages, heads, page_size, dim = shape
    if (Hkv is not None and heads != Hkv) or dim != D:
        raise ValueError(f"k_pages {list(shape)} does not hold the given heads or head dimension")
    scales = (num_pages, heads, page_size // 16)
    check_tensor("k_pages", k_pages, k_pages.dtype, shape, device)
    check_tensor("v_pages", v_pages, k_pages.dtype, shape, device)
    check_tensor("k_scales", k_scales, torch.float32, scales, device)
    check_tensor("v_scales", v_scales, torch.float32, scales, device)
    if block_table.dim() != 2:
        raise ValueError("block_table: expected [B, pages_per_seq]")
    pages_per_seq = block_table.shape[1]
    check_tensor("block_table", block_table, torch.int32, (B, pages_per_seq), device)
    if seqlens_k is not None:
        check_tensor("seqlens_k", seqlens_k, torch.int32, (B,), device)
    return num_pages, heads, page_size, pages_per_seq, code


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
    import torch
    B, Nt, Hkv, D = k.shape
    dev = k.device
    num_pages, _, page_size, pps, code = _check_cache(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, Hkv, D, dev)
    if new_lens is not None:
        check_tensor("new_lens", new_lens, torch.int32, (B,), dev)
    if v.dtype is not k.dtype or v.shape != k.shape or v.device != dev:
        raise ValueError("k and v must be alike")
    context, raw = enter(dev, stream)

    def call():
        rk, rv = (k, v) if k.is_contiguous() and v.is_contiguous() else (k.contiguous(), v.contiguous())
        return (_lib._lib or load()).fa_kv8_append(
            rk.data_ptr(), rv.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
            block_table.data_ptr(), seqlens_k.data_ptr(), None if new_lens is None else new_lens.data_ptr(), B, Nt, Hkv, num_pages,
            page_size, pps, D, raw, _types()[1].get(k.dtype, -1), code)

    st = in_context(context, call)
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
    import torch
    B, Nq, Hq, D = q.shape
    dev = q.device
    num_pages, Hkv, page_size, pps, code = _check_cache(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, None, D, dev)
    floats = _types()[1]
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError("workspace: expected a contiguous tensor on the device of q")
    context, raw = enter(dev, stream)

    def call():
        rq = q if q.is_contiguous() else q.contiguous()
        ws = torch.empty(_workspace_bytes(B, Nq, Hq, Hkv, D), device=dev, dtype=torch.uint8) if workspace is None else workspace
        o = torch.empty_like(rq, dtype=out_dtype)
        lse = torch.empty((B, Hq, Nq), device=dev, dtype=torch.float32)
        st = (_lib._lib or load()).fa_kv8_attend(
            rq.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block_table.data_ptr(),
            o.data_ptr(), lse.data_ptr(), B, Nq, Hq, Hkv, num_pages, page_size, pps, D, 1.0 / math.sqrt(D) if scale is None else scale,
            None if seqlens_k is None else seqlens_k.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), raw,
            floats.get(q.dtype, -1), code, floats.get(o.dtype, -1))
        return st, o, lse

    st, o, lse = in_context(context, call)
    if st != fa.FA_OK:
        raise fa.FAError(st, "fa_kv8_attend")
    return o, lse
