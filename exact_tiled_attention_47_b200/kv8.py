"""Paged cache held in 8 bits: the binding of ``fa_kv8_append`` and ``fa_kv8_attend``, and helpers.

A cache is four tensors, ``k_pages``/``v_pages`` [num_pages, Hkv, page_size, D] of codes
(torch.float8_e4m3fn or torch.int8) and ``k_scales``/``v_scales`` fp32 [num_pages, Hkv, page_size / 16];
a code stands for code * scale.  The functions named like the C entry points only marshal arguments;
the helpers check tensors, allocate outputs and raise on errors, as those of the package do.
"""
from __future__ import annotations

import math

import exact_tiled_attention_47_b200 as fa

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


class on_stream:
    """The device of the tensors and the caller's stream (a torch stream, a handle, or None for the
    current one) made current, so that what a helper allocates belongs to the stream its kernels run on."""

    __slots__ = ("stack",)

    def __init__(self, device, stream):
        import torch
        self.stack = []
        if device.type != "cuda":
            raise ValueError("tensors must be on a CUDA device")
        if device.index != torch.cuda.current_device():
            self.stack.append(torch.cuda.device(device))
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
            if stream.device != device:
                raise ValueError("the stream belongs to another device than the tensors")
            self.stack.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.stack:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.stack):
            c.__exit__(*exc)


def check_tensor(name, t, dtype, shape, device):
    """Raises ValueError unless t is a contiguous tensor of this dtype, shape and device."""
    if t.dtype is not dtype or tuple(t.shape) != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {list(shape)} on {device}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device} with strides {list(t.stride())}")


def _check_cache(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, Hkv, D, device):
    import torch
    if k_pages.dim() != 4 or k_pages.dtype not in _types()[0]:
        raise ValueError("k_pages: expected [num_pages, Hkv, page_size, D] of torch.float8_e4m3fn or torch.int8")
    num_pages, heads, page_size, dim = k_pages.shape
    if Hkv is not None and heads != Hkv or dim != D:
        raise ValueError(f"k_pages {list(k_pages.shape)} does not hold the given heads or head dimension")
    check_tensor("k_pages", k_pages, k_pages.dtype, (num_pages, heads, page_size, dim), device)
    check_tensor("v_pages", v_pages, k_pages.dtype, (num_pages, heads, page_size, dim), device)
    scales = (num_pages, heads, page_size // 16)
    check_tensor("k_scales", k_scales, torch.float32, scales, device)
    check_tensor("v_scales", v_scales, torch.float32, scales, device)
    if block_table.dim() != 2:
        raise ValueError("block_table: expected [B, pages_per_seq]")
    check_tensor("block_table", block_table, torch.int32, (B, block_table.shape[1]), device)
    if seqlens_k is not None:
        check_tensor("seqlens_k", seqlens_k, torch.int32, (B,), device)
    return num_pages, heads, page_size


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
    num_pages, _, page_size = _check_cache(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, Hkv, D, dev)
    if new_lens is not None:
        check_tensor("new_lens", new_lens, torch.int32, (B,), dev)
    if v.dtype is not k.dtype or v.shape != k.shape or v.device != dev:
        raise ValueError("k and v must be alike")
    with on_stream(dev, stream):
        k, v = k.contiguous(), v.contiguous()
        st = fa_kv8_append(k, v, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, new_lens, B, Nt, Hkv, num_pages, page_size,
                           block_table.shape[1], D)
    if st != fa.FA_OK:
        raise fa.FAError(st, "fa_kv8_append")


def attend_kv8(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k=None, scale=None, out_dtype=None, workspace=None,
               stream=None):
    """O [B,Nq,Hq,D], LSE [B,Hq,Nq] of the newest Nq tokens q of each sequence over its 8-bit cache.

    ``block_table`` int32 [B, pages_per_seq]; ``seqlens_k`` int32 [B] (keys of each sequence, those of the Nq tokens
    included) or None (every table entry in use).  Query i of item b sees keys up to seqlens_k[b] - Nq + i.
    """
    import torch
    B, Nq, Hq, D = q.shape
    dev = q.device
    num_pages, Hkv, page_size = _check_cache(k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, B, None, D, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with on_stream(dev, stream):
        q = q.contiguous()
        if workspace is None:
            workspace = torch.empty(max(1, fa_kv8_attend_workspace_bytes(B, Nq, Hq, Hkv, D)), device=dev, dtype=torch.uint8)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace: expected a contiguous tensor on the device of q")
        o = torch.empty((B, Nq, Hq, D), device=dev, dtype=q.dtype if out_dtype is None else out_dtype)
        lse = torch.empty((B, Hq, Nq), device=dev, dtype=torch.float32)
        st = fa_kv8_attend(q, k_pages, v_pages, k_scales, v_scales, block_table, o, lse, B, Nq, Hq, Hkv, num_pages, page_size,
                           block_table.shape[1], D, scale, seqlens_k, workspace)
    if st != fa.FA_OK:
        raise fa.FAError(st, "fa_kv8_attend")
    return o, lse
