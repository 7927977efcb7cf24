"""Pages of a cache: the binding of ``fa_pages_*``, and helpers.

State, on the device: ``block_table`` int32 [S, pages_per_seq], ``seqlens`` int32 [S] and ``refcount`` int32
[num_pages] (zeros to begin with).  ``pools`` are the cache's tensors, whatever they hold, with the page as
their first dimension (K, V and scales of all layers).  The functions named like the C entry points only
marshal arguments; the helpers check tensors, allocate workspaces and raise on errors.  Faults that the
device finds (a slot named twice, no free pages) are read with ``fa_device_status``.
"""
from __future__ import annotations

import ctypes

import exact_tiled_attention_47_b200 as fa

from ._lib import load
from .kv8 import check_tensor, on_stream


def _pointers(pools):
    return (ctypes.c_void_p * len(pools))(*[fa._ptr(t) for t in pools])


def _sizes(page_bytes):
    return (ctypes.c_size_t * len(page_bytes))(*page_bytes)


def _bytes_of(workspace, workspace_bytes):
    return workspace.numel() * workspace.element_size() if workspace_bytes is None else int(workspace_bytes)


def fa_pages_workspace_bytes(n, S, num_pages) -> int:
    return int(load().fa_pages_workspace_bytes(int(n), int(S), int(num_pages)))


def fa_pages_extend(block_table, seqlens, refcount, slots, add, n, S, pages_per_seq, num_pages, page_size, workspace,
                    workspace_bytes=None, stream=None) -> int:
    """Marshal to the C ``fa_pages_extend``; returns its status."""
    p = fa._ptr
    return load().fa_pages_extend(p(block_table), p(seqlens), p(refcount), p(slots), p(add), int(n), int(S), int(pages_per_seq),
                                  int(num_pages), int(page_size), p(workspace), _bytes_of(workspace, workspace_bytes), fa._stream(stream))


def fa_pages_fork(block_table, seqlens, refcount, src, dst, n, S, pages_per_seq, num_pages, page_size, pools, page_bytes, workspace,
                  workspace_bytes=None, stream=None) -> int:
    """Marshal to the C ``fa_pages_fork`` (pools: tensors or addresses; page_bytes: ints); returns its status."""
    p = fa._ptr
    return load().fa_pages_fork(p(block_table), p(seqlens), p(refcount), p(src), p(dst), int(n), int(S), int(pages_per_seq),
                                int(num_pages), int(page_size), _pointers(pools), _sizes(page_bytes), len(pools), p(workspace),
                                _bytes_of(workspace, workspace_bytes), fa._stream(stream))


def fa_pages_free(block_table, seqlens, refcount, slots, n, S, pages_per_seq, num_pages, page_size, stream=None) -> int:
    """Marshal to the C ``fa_pages_free``; returns its status."""
    p = fa._ptr
    return load().fa_pages_free(p(block_table), p(seqlens), p(refcount), p(slots), int(n), int(S), int(pages_per_seq), int(num_pages),
                                int(page_size), fa._stream(stream))


def fa_pages_compact(block_table, seqlens, refcount, block_table_out, refcount_out, remap, n_live, S, pages_per_seq, num_pages,
                     page_size, pools, page_bytes, workspace, workspace_bytes=None, stream=None) -> int:
    """Marshal to the C ``fa_pages_compact``; returns its status."""
    p = fa._ptr
    return load().fa_pages_compact(p(block_table), p(seqlens), p(refcount), p(block_table_out), p(refcount_out), p(remap), p(n_live),
                                   int(S), int(pages_per_seq), int(num_pages), int(page_size), _pointers(pools), _sizes(page_bytes),
                                   len(pools), p(workspace), _bytes_of(workspace, workspace_bytes), fa._stream(stream))


def fa_pages_copy(src_pools, dst_pools, page_bytes, src, dst, n, src_num_pages, dst_num_pages, workspace, workspace_bytes=None,
                  stream=None) -> int:
    """Marshal to the C ``fa_pages_copy``; returns its status."""
    p = fa._ptr
    if len(src_pools) != len(dst_pools) or len(src_pools) != len(page_bytes):
        return fa.FA_ERR_SHAPE
    return load().fa_pages_copy(_pointers(src_pools), _pointers(dst_pools), _sizes(page_bytes), len(src_pools), p(src), p(dst), int(n),
                                int(src_num_pages), int(dst_num_pages), p(workspace), _bytes_of(workspace, workspace_bytes),
                                fa._stream(stream))


# ------------------------------------------------------------------------------------------------
# helpers


def _check_state(block_table, seqlens, refcount):
    import torch
    if block_table.dim() != 2 or refcount.dim() != 1:
        raise ValueError("expected block_table [S, pages_per_seq] and refcount [num_pages]")
    S, pages_per_seq = block_table.shape
    dev = block_table.device
    check_tensor("block_table", block_table, torch.int32, (S, pages_per_seq), dev)
    check_tensor("seqlens", seqlens, torch.int32, (S,), dev)
    check_tensor("refcount", refcount, torch.int32, (refcount.numel(),), dev)
    return S, pages_per_seq, refcount.numel(), dev


def _check_list(name, t, n, dev):
    import torch
    check_tensor(name, t, torch.int32, (t.numel() if n is None else n,), dev)
    return t.numel()


def _page_bytes(pools, num_pages, dev):
    """Bytes of a page in each pool."""
    out = []
    for t in pools:
        if t.dim() < 1 or t.shape[0] != num_pages or t.device != dev or not t.is_contiguous():
            raise ValueError(f"pools: expected contiguous tensors of {num_pages} pages on {dev}, got {list(t.shape)} on {t.device}")
        out.append(t.numel() // num_pages * t.element_size())
    return out


def _workspace(workspace, n, S, num_pages, dev):
    import torch
    if workspace is None:
        return torch.empty(max(1, fa_pages_workspace_bytes(n, S, num_pages)), device=dev, dtype=torch.uint8)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor on the device of the state")
    return workspace


def _raise(st, where):
    if st != fa.FA_OK:
        raise fa.FAError(st, where)


def extend_pages(block_table, seqlens, refcount, page_size, add, slots=None, workspace=None, stream=None):
    """Lengthen slots (int32 [n]; None: the first n) by ``add`` (int32 [n]) keys each, with the pages that takes."""
    S, pps, num_pages, dev = _check_state(block_table, seqlens, refcount)
    n = _check_list("add", add, None, dev)
    if slots is not None:
        _check_list("slots", slots, n, dev)
    if n == 0:
        return
    with on_stream(dev, stream):
        ws = _workspace(workspace, n, S, num_pages, dev)
        st = fa_pages_extend(block_table, seqlens, refcount, slots, add, n, S, pps, num_pages, page_size, ws)
    _raise(st, "fa_pages_extend")


def fork_pages(block_table, seqlens, refcount, page_size, src, dst, pools, workspace=None, stream=None):
    """Make each empty slot dst[i] a copy of slot src[i]: full pages shared, a last partial page copied in every pool."""
    S, pps, num_pages, dev = _check_state(block_table, seqlens, refcount)
    n = _check_list("src", src, None, dev)
    _check_list("dst", dst, n, dev)
    sizes = _page_bytes(pools, num_pages, dev)
    if n == 0:
        return
    with on_stream(dev, stream):
        ws = _workspace(workspace, n, S, num_pages, dev)
        st = fa_pages_fork(block_table, seqlens, refcount, src, dst, n, S, pps, num_pages, page_size, pools, sizes, ws)
    _raise(st, "fa_pages_fork")


def free_pages(block_table, seqlens, refcount, page_size, slots, stream=None):
    """Empty slots (int32 [n]) and give back the pages that nobody else holds."""
    S, pps, num_pages, dev = _check_state(block_table, seqlens, refcount)
    n = _check_list("slots", slots, None, dev)
    if n == 0:
        return
    with on_stream(dev, stream):
        st = fa_pages_free(block_table, seqlens, refcount, slots, n, S, pps, num_pages, page_size)
    _raise(st, "fa_pages_free")


def compact_pages(block_table, seqlens, refcount, page_size, pools, in_place=False, workspace=None, stream=None):
    """Move the live pages of every pool to the front; returns (block_table, refcount, remap, n_live) of the new places.

    ``in_place``: the given block_table and refcount are updated and returned; else new tensors are.  ``remap`` int32
    [num_pages]: the new place of each live page, -1 for free ones; ``n_live`` int32 [1].
    """
    import torch
    S, pps, num_pages, dev = _check_state(block_table, seqlens, refcount)
    sizes = _page_bytes(pools, num_pages, dev)
    with on_stream(dev, stream):
        table_out, ref_out = (block_table, refcount) if in_place else (torch.empty_like(block_table), torch.empty_like(refcount))
        remap, n_live = torch.empty_like(refcount), torch.empty(1, device=dev, dtype=torch.int32)
        ws = _workspace(workspace, 1, S, num_pages, dev)
        st = fa_pages_compact(block_table, seqlens, refcount, table_out, ref_out, remap, n_live, S, pps, num_pages, page_size, pools, sizes, ws)
    _raise(st, "fa_pages_compact")
    return table_out, ref_out, remap, n_live


def copy_pages(src_pools, dst_pools, src, dst, workspace=None, stream=None):
    """Copy page src[i] (int32 [n]) of each source pool to page dst[i] of the destination pool at the same place."""
    if not src_pools or len(src_pools) != len(dst_pools):
        raise ValueError("expected as many source pools as destination pools, at least one")
    dev = src_pools[0].device
    n = _check_list("src", src, None, dev)
    _check_list("dst", dst, n, dev)
    a, b = src_pools[0].shape[0], dst_pools[0].shape[0]
    sizes = _page_bytes(src_pools, a, dev)
    if sizes != _page_bytes(dst_pools, b, dev):
        raise ValueError("source and destination pools have pages of unlike sizes")
    if n == 0:
        return
    with on_stream(dev, stream):
        ws = _workspace(workspace, n, 1, max(a, b), dev)
        st = fa_pages_copy(src_pools, dst_pools, sizes, src, dst, n, a, b, ws)
    _raise(st, "fa_pages_copy")
