"""Pages of a cache: the binding of ``fa_pages_*``, and helpers.

State, on the device: ``block_table`` int32 [S, pages_per_seq], ``seqlens`` int32 [S] and ``refcount`` int32
[num_pages] (zeros to begin with).  ``pools`` are the cache's tensors, whatever they hold, with the page as
their first dimension (K, V and scales of all layers).  The functions named like the C entry points only
marshal arguments; the helpers check tensors, allocate workspaces and raise on errors.  Faults that the
device finds (a slot named twice, no free pages) are read with ``fa_device_status``.
"""
from __future__ import annotations

import ctypes
import functools

import exact_tiled_attention_47_b200 as fa

from . import _lib, kv8
from ._lib import load
from .kv8 import alike, check_tensor, in_context, place_of


def _pointers(pools):
    return (ctypes.c_void_p * len(pools))(*[t if isinstance(t, int) else t.data_ptr() for t in pools])


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
    shape, count, dev = block_table.shape, refcount.shape, block_table.device
    if len(shape) != 2 or len(count) != 1:
        raise ValueError("expected block_table [S, pages_per_seq] and refcount [num_pages]")
    int32 = kv8._torch().int32
    if not (alike(block_table, int32, shape, dev) and alike(seqlens, int32, shape[:1], dev) and alike(refcount, int32, count, dev)):
        check_tensor("block_table", block_table, int32, shape, dev)
        check_tensor("seqlens", seqlens, int32, shape[:1], dev)
        check_tensor("refcount", refcount, int32, count, dev)
    return shape[0], shape[1], count[0], dev


def _check_list(name, t, n, dev):
    check_tensor(name, t, kv8._torch().int32, (t.numel() if n is None else n,), dev)
    return t.numel()


def _page_bytes(pools, num_pages, dev):
    """Bytes of a page in each pool."""
    out = []
    for t in pools:
        if t.dim() < 1 or t.shape[0] != num_pages or t.device != dev or not t.is_contiguous():
            raise ValueError(f"pools: expected contiguous tensors of {num_pages} pages on {dev}, got {list(t.shape)} on {t.device}")
        out.append(t.nbytes // num_pages)
    return out


@functools.lru_cache(maxsize=256)
def _workspace_bytes(*sizes):
    return max(1, fa_pages_workspace_bytes(*sizes))


def _check_workspace(workspace, dev):
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError("workspace: expected a contiguous tensor on the device of the state")


def _workspace(workspace, n, S, num_pages, dev):
    """(tensor, bytes), allocated on the current stream where the caller gave none."""
    if workspace is None:
        need = _workspace_bytes(n, S, num_pages)
        return kv8._TORCH.empty(need, device=dev, dtype=kv8._TORCH.uint8), need
    return workspace, workspace.nbytes


def _raise(st, where):
    if st != fa.FA_OK:
        raise fa.FAError(st, where)


def extend_pages(block_table, seqlens, refcount, page_size, add, slots=None, workspace=None, stream=None):
    """Lengthen slots (int32 [n]; None: the first n) by ``add`` (int32 [n], not negative) keys each, with the pages that takes.

    To take keys back (rejected drafts), keep ``seqlens`` as what the slots hold and pass ``append_kv8`` and ``attend_kv8``
    valid lengths of their own; or lower ``seqlens`` inside a slot's last page.  Lowered past a page's border, pages are lost.
    """
    S, pps, num_pages, dev = _check_state(block_table, seqlens, refcount)
    n = _check_list("add", add, None, dev)
    if slots is not None:
        _check_list("slots", slots, n, dev)
    _check_workspace(workspace, dev)
    context, raw = place_of(dev, stream)
    if n == 0:
        return

    def call():
        ws, size = _workspace(workspace, n, S, num_pages, dev)
        return (_lib._lib or load()).fa_pages_extend(
            block_table.data_ptr(), seqlens.data_ptr(), refcount.data_ptr(), None if slots is None else slots.data_ptr(), add.data_ptr(), n,
            S, pps, num_pages, page_size, ws.data_ptr(), size, raw)

    _raise(in_context(context, call), "fa_pages_extend")


def fork_pages(block_table, seqlens, refcount, page_size, src, dst, pools, workspace=None, stream=None):
    """Make each empty slot dst[i] a copy of slot src[i]: full pages shared, a last partial page copied in every pool."""
    S, pps, num_pages, dev = _check_state(block_table, seqlens, refcount)
    n = _check_list("src", src, None, dev)
    _check_list("dst", dst, n, dev)
    sizes = _page_bytes(pools, num_pages, dev)
    _check_workspace(workspace, dev)
    context, raw = place_of(dev, stream)
    if n == 0:
        return

    def call():
        ws, size = _workspace(workspace, n, S, num_pages, dev)
        return (_lib._lib or load()).fa_pages_fork(
            block_table.data_ptr(), seqlens.data_ptr(), refcount.data_ptr(), src.data_ptr(), dst.data_ptr(), n, S, pps, num_pages, page_size,
            _pointers(pools), _sizes(sizes), len(sizes), ws.data_ptr(), size, raw)

    _raise(in_context(context, call), "fa_pages_fork")


def free_pages(block_table, seqlens, refcount, page_size, slots, stream=None):
    """Empty slots (int32 [n]) and give back the pages that nobody else holds."""
    S, pps, num_pages, dev = _check_state(block_table, seqlens, refcount)
    n = _check_list("slots", slots, None, dev)
    context, raw = place_of(dev, stream)
    if n == 0:
        return

    def call():
        return (_lib._lib or load()).fa_pages_free(block_table.data_ptr(), seqlens.data_ptr(), refcount.data_ptr(), slots.data_ptr(), n, S, pps,
                                                   num_pages, page_size, raw)

    _raise(in_context(context, call), "fa_pages_free")


def compact_pages(block_table, seqlens, refcount, page_size, pools, in_place=False, workspace=None, stream=None):
    """Move the live pages of every pool to the front; returns (block_table, refcount, remap, n_live) of the new places.

    ``in_place``: the given block_table and refcount are updated and returned; else new tensors are.  ``remap`` int32
    [num_pages]: the new place of each live page, -1 for free ones; ``n_live`` int32 [1].
    """
    S, pps, num_pages, dev = _check_state(block_table, seqlens, refcount)
    sizes = _page_bytes(pools, num_pages, dev)
    _check_workspace(workspace, dev)
    context, raw = place_of(dev, stream)

    def call():
        like = kv8._TORCH.empty_like
        table_out, ref_out = (block_table, refcount) if in_place else (like(block_table), like(refcount))
        remap, n_live = like(refcount), refcount.new_empty(1)
        ws, size = _workspace(workspace, 1, S, num_pages, dev)
        st = (_lib._lib or load()).fa_pages_compact(
            block_table.data_ptr(), seqlens.data_ptr(), refcount.data_ptr(), table_out.data_ptr(), ref_out.data_ptr(), remap.data_ptr(),
            n_live.data_ptr(), S, pps, num_pages, page_size, _pointers(pools), _sizes(sizes), len(sizes), ws.data_ptr(), size, raw)
        return st, (table_out, ref_out, remap, n_live)

    st, out = in_context(context, call)
    _raise(st, "fa_pages_compact")
    return out


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
    _check_workspace(workspace, dev)
    context, raw = place_of(dev, stream)
    if n == 0:
        return

    def call():
        ws, size = _workspace(workspace, n, 1, max(a, b), dev)
        return (_lib._lib or load()).fa_pages_copy(_pointers(src_pools), _pointers(dst_pools), _sizes(sizes), len(sizes), src.data_ptr(),
                                                   dst.data_ptr(), n, a, b, ws.data_ptr(), size, raw)

    _raise(in_context(context, call), "fa_pages_copy")
