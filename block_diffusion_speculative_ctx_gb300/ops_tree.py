"""Serving operators for trees of drafted tokens and for pages that several sequences hold, over
torch tensors: argument checks and marshalling, as in ops.py.

    tree_masks      ancestor masks, depths and positions of trees from their nodes' parents
    tree_attention  attention of trees over a paged cache, behind a shared prefix or none
    tree_accept     greedy acceptance of verified trees
    kv_compact      the accepted nodes' keys and values to their places
    kv_fork         sequences that continue others on shared pages
    kv_release      the pages of ended sequences back to the free list

One step of a batch: ``tree_masks`` once, ``tree_attention`` in each layer of the verify pass,
``tree_accept`` on its argmax, ``kv_compact`` on the caches of all layers."""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional

import torch

from . import load
from . import ops as _ops
from .ops import (_F32T, _I32, _I32T, _I64, _P, OPS_MAX_BATCH, PAGE_TOKENS, _attend, _bad, _call, _device,
                  dflash_shared_prefix_args)

TREE_MAX_NODES = 1024


class dflash_tree_masks_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("batch", "rows", "words", "base_pos")] + [("ld_mask", _I64)]
                + [(n, _P) for n in ("parents", "q_start", "kv_lens", "masks", "depth", "row_pos", "status")])


class dflash_tree_attention_args(ctypes.Structure):
    _fields_ = [("attn", dflash_shared_prefix_args), ("masks", _P), ("ld_mask", _I64), ("words", _I32), ("reserved", _I32)]


class dflash_tree_accept_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("batch", "rows", "width", "reserved")]
                + [(n, _P) for n in ("parents", "tokens", "posterior", "q_start", "path", "accepted", "bonus", "status")])


class dflash_kv_compact_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "batch", "layers", "n_pages", "n_kv_heads", "head_dim", "width", "width_table")]
                + [(n, _I64) for n in ("ld_layer", "ld_table")]
                + [(n, _P) for n in ("k_cache", "v_cache", "table", "kv_lens", "q_start", "path", "accepted", "kv_out",
                                     "status")])


class dflash_kv_fork_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "batch", "children", "width", "n_free", "scratch_page", "layers", "n_pages",
                                     "n_kv_heads", "head_dim")]
                + [(n, _I64) for n in ("ld_layer", "ld_table", "ld_out")]
                + [(n, _P) for n in ("k_cache", "v_cache", "parents", "kv_lens", "table", "free_pages", "used", "refs",
                                     "table_out", "lens_out", "used_out", "status")])


class dflash_kv_release_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("batch", "n", "width", "n_free", "n_pages", "reserved")] + [("ld_table", _I64)]
                + [(n, _P) for n in ("seqs", "kv_lens", "table", "free_pages", "used", "refs", "used_out", "status",
                                     "keep_lens")])


# (packed forms of the structs, as in ops.py)
_MASKS, _TREE = struct.Struct("4iq7Q"), struct.Struct("10ifi3q11QQq2i")
_ACCEPT, _COMPACT = struct.Struct("4i8Q"), struct.Struct("8i2q9Q")
_FORK, _RELEASE = struct.Struct("10i3q12Q"), struct.Struct("6iq9Q")


class TreeMasks(NamedTuple):
    masks: torch.Tensor
    depth: torch.Tensor
    row_pos: Optional[torch.Tensor]
    status: torch.Tensor


class TreeAccept(NamedTuple):
    path: torch.Tensor
    accepted: torch.Tensor
    bonus: torch.Tensor
    status: torch.Tensor


class KVCompact(NamedTuple):
    kv_lens: torch.Tensor
    status: torch.Tensor


class KVFork(NamedTuple):
    table: torch.Tensor
    kv_lens: torch.Tensor
    used: torch.Tensor
    status: torch.Tensor


class KVRelease(NamedTuple):
    used: torch.Tensor
    status: torch.Tensor


def _batch(name, t, extra=0):
    n = t.numel() - extra
    if not 1 <= n <= OPS_MAX_BATCH:
        _bad(f"{name} must hold {1 + extra} to {OPS_MAX_BATCH + extra} entries")
    return n


def tree_masks(parents, q_start, *, kv_lens=None, base_pos: int = 0, words: Optional[int] = None, masks=None, depth=None,
               row_pos=None, status=None) -> TreeMasks:
    """Masks, depths and positions of trees (``dflash_tree_masks``).

    parents: int32 [rows], each node's parent by its number in the tree (before the node's own; -1: a root);
    q_start: int32 [batch + 1], the trees' rows.  ``masks``: int32 [rows, words], bit i set for node i of the
    row's tree that is the row's node or an ancestor; ``words`` defaults to those of ``masks``, or to as many as
    the rows of the whole batch need: give the widest tree's ceil(m / 32).  ``depth``: int32 [rows].  With
    kv_lens (int32 [batch], own keys, the tree's among them) ``row_pos`` is base_pos + kv_lens - m + depth.
    Missing outputs are allocated (0 in rows of no tree).  ``status``: int32 [batch] on the device, 0 or a sum of
    1 (a parent not before its child), 2 (too many nodes), 4 (bad q_start), 8 (a length whose positions are below 0
    or beyond int32: row_pos is -1, masks and depth are as they should be)."""
    dev = _device(parents)
    rows, batch = parents.numel(), _batch("q_start", q_start, 1)
    if masks is None:
        if words is None:
            words = max(1, -(-min(rows, TREE_MAX_NODES) // 32))
        masks = torch.zeros((rows, words), dtype=_I32T, device=parents.device)
    elif words is None:
        words = masks.shape[-1]
    ld = max(_ops._mat("masks", masks, _I32T, rows, words, dev), words)
    if depth is None:
        depth = torch.zeros(rows, dtype=_I32T, device=parents.device)
    if status is None:
        status = torch.empty(batch, dtype=_I32T, device=parents.device)
    p_par, p_start, p_depth, p_status = _ops._ints(dev, "parents", parents, rows, "q_start", q_start, batch + 1, "depth", depth,
                                                   rows, "status", status, batch)
    p_kv = p_pos = 0
    if kv_lens is not None:
        if row_pos is None:
            row_pos = torch.zeros(rows, dtype=_I32T, device=parents.device)
        p_kv, p_pos = _ops._ints(dev, "kv_lens", kv_lens, batch, "row_pos", row_pos, rows)
    elif row_pos is not None:
        _bad("row_pos needs kv_lens")
    _call(load().dflash_tree_masks, _MASKS.pack,
          (batch, rows, words, base_pos, ld, p_par, p_start, p_kv, masks.data_ptr(), p_depth, p_pos, p_status), dev)
    _ops._written(masks, depth, row_pos, status)
    return TreeMasks(masks, depth, row_pos, status)


def tree_attention(q, k_cache, v_cache, table, kv_lens, q_start, masks, *, prefix_pages=None, prefix_len: int = 0,
                   scale: Optional[float] = None, out=None, lse=None, workspace=None, weight_pairs: bool = False):
    """Attention of trees of drafted tokens over a paged cache (``dflash_tree_attention``).

    As ``shared_prefix_attention`` (types, layouts, workspace of ``shared_prefix_workspace`` bytes, rows outside
    q_start), but of the sequence's own kv_lens keys row r sees the committed ones, those before its m last,
    and of these m the nodes whose bit is set in masks[r] (int32 [rows, words], as ``tree_masks`` makes them, or
    any others).  A row that sees nothing gives 0 and an lse of -inf.  Returns (out, lse).
    bf16 calls round each softmax weight once to bf16 for the product with v (rms 2.1e-3 .. 2.4e-3 of the output from 64
    bits); ``weight_pairs`` holds it as a bf16 pair, which leaves the output's own rounding (1.7e-3) and takes 5 % longer
    where a call is short and up to 30 % where it is bound by the softmax."""
    dev = _device(q, q, k_cache, v_cache, out, lse)
    if q.dim() != 3 or k_cache.dim() != 4:
        _bad("q must be [rows, H, hd] and the caches [pages, H_kv, 64, hd]")
    rows, h, hd = q.shape
    dtype = q.dtype
    dt, _, pages, hkv, kv_hd, _ = _ops._caches(k_cache, v_cache, dev)
    if k_cache.dtype is not dtype or kv_hd != hd:
        _bad(f"k_cache and v_cache must be {dtype} [pages, H_kv, {PAGE_TOKENS}, {hd}]")
    batch = _batch("kv_lens", kv_lens)
    if out is None:
        out = torch.zeros((rows, h, hd), dtype=dtype, device=q.device)
    if lse is None:
        lse = torch.zeros((rows, h), dtype=_F32T, device=q.device)
    p_kv, p_start, p_lse = _ops._flats(dev, "kv_lens", kv_lens, _I32T, batch, "q_start", q_start, _I32T, batch + 1,
                                       "lse", lse, _F32T, rows * h)
    p_pre = 0
    if prefix_pages is not None:
        n_pre = prefix_pages.numel()
        p_pre = _ops._flat("prefix_pages", prefix_pages, _I32T, n_pre, dev)
        if n_pre * PAGE_TOKENS < prefix_len:
            _bad(f"prefix_pages holds {n_pre} pages, too few for {prefix_len} tokens")
    elif prefix_len != 0:
        _bad("prefix_pages is needed for a prefix")
    ld_table = _ops._mat("table", table, _I32T, batch, None, dev)
    ld_mask = _ops._mat("masks", masks, _I32T, rows, None, dev)
    words = masks.shape[1]
    ld_q = _ops._rows3("q", q, dtype, rows, h, hd, dev)
    ld_out = _ops._rows3("out", out, dtype, rows, h, hd, dev)
    args = (dt, h, hkv, hd, batch, rows, pages, prefix_len, table.shape[1], 0, hd ** -0.5 if scale is None else scale,
            1 if weight_pairs else 0, ld_q, ld_out, ld_table, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), p_pre,
            table.data_ptr(), p_kv, p_start, out.data_ptr(), p_lse)
    _attend(load().dflash_tree_attention, _TREE.pack, args, (masks.data_ptr(), max(ld_mask, words), words, 0),
            (dt, h, hkv, hd, batch, rows), workspace, dev, q.device)
    _ops._written(out, lse)
    return out, lse


def tree_accept(parents, tokens, posterior, q_start, *, width: Optional[int] = None, path=None, accepted=None, bonus=None,
                status=None) -> TreeAccept:
    """Greedy acceptance of verified trees (``dflash_tree_accept``).

    parents, tokens, posterior: int32 [rows], a node's parent in its tree, its drafted token and the target's
    choice behind it; q_start: int32 [batch + 1].  ``path``: int32 [batch, width], the nodes kept from the root
    on (-1 behind them; at most ``width``); ``accepted``: int32 [batch], the drafts among them (-1 for a sequence
    without rows); ``bonus``: int32 [batch], the target's choice behind the last.  ``status``: int32 [batch], 1,
    2 or 4 as ``tree_masks``: a bad tree has accepted = bonus = -1 and a path of -1."""
    dev = _device(parents)
    rows, batch = parents.numel(), _batch("q_start", q_start, 1)
    if path is None:
        if width is None:
            _bad("width is needed when no path is given")
        path = torch.empty((batch, width), dtype=_I32T, device=parents.device)
    elif path.dim() != 2 or (width is not None and path.shape[1] != width):
        _bad("path must be [batch, width]")
    width = path.shape[1]
    if accepted is None:
        accepted = torch.empty(batch, dtype=_I32T, device=parents.device)
    if bonus is None:
        bonus = torch.empty(batch, dtype=_I32T, device=parents.device)
    if status is None:
        status = torch.empty(batch, dtype=_I32T, device=parents.device)
    _call(load().dflash_tree_accept, _ACCEPT.pack,
          (batch, rows, width, 0,
           *_ops._ints(dev, "parents", parents, rows, "tokens", tokens, rows, "posterior", posterior, rows, "q_start", q_start,
                       batch + 1, "path", path, batch * width, "accepted", accepted, batch, "bonus", bonus, batch, "status",
                       status, batch)), dev)
    _ops._written(path, accepted, bonus, status)
    return TreeAccept(path, accepted, bonus, status)


def kv_compact(k_cache, v_cache, table, kv_lens, q_start, path, accepted, *, kv_out=None, status=None) -> KVCompact:
    """The accepted nodes of trees to their places in the caches of all layers (``dflash_kv_compact``).

    k_cache, v_cache: [pages, H_kv, 64, hd] or [layers, pages, H_kv, 64, hd] (fp32 or bf16), changed in place;
    table: int32 [batch, width]; kv_lens: int32 [batch], own keys, the tree's among them; q_start: int32
    [batch + 1]; path, accepted: as ``tree_accept`` gives them.  The lengths behind it are in ``kv_lens`` of the
    result (``kv_out``, not kv_lens itself).  An ``accepted`` of -1, as a tree gets that ``tree_accept`` refused, keeps no
    node, the root neither: its length is the one before the step, and status is 0 (``tree_accept``'s is not).  ``status``: int32 [batch], 0 or a sum of 1 (a path that does not rise
    within the tree), 4 (bad q_start), 8 (bad length), 16 (bad page): nothing of the sequence has moved."""
    dev = _device(kv_lens, k_cache, v_cache)
    batch = _batch("kv_lens", kv_lens)
    dt, layers, pages, hkv, hd, ld_layer = _ops._caches(k_cache, v_cache, dev)
    ld_table = _ops._mat("table", table, _I32T, batch, None, dev)
    if path.dim() != 2:
        _bad("path must be [batch, width]")
    width = path.shape[1]
    if kv_out is None:
        kv_out = torch.empty(batch, dtype=_I32T, device=kv_lens.device)
    if status is None:
        status = torch.empty(batch, dtype=_I32T, device=kv_lens.device)
    _call(load().dflash_kv_compact, _COMPACT.pack,
          (dt, batch, layers, pages, hkv, hd, width, table.shape[1], ld_layer, ld_table, k_cache.data_ptr(), v_cache.data_ptr(),
           table.data_ptr(),
           *_ops._ints(dev, "kv_lens", kv_lens, batch, "q_start", q_start, batch + 1, "path", path, batch * width, "accepted",
                       accepted, batch, "kv_out", kv_out, batch, "status", status, batch)), dev)
    _ops._written(k_cache, v_cache, kv_out, status)
    return KVCompact(kv_out, status)


def kv_fork(parents, kv_lens, table, free_pages, used, refs, k_cache, v_cache, *, scratch_page: int = 0, table_out=None,
            lens_out=None, used_out=None, status=None) -> KVFork:
    """Sequences that continue others on shared pages (``dflash_kv_fork``).

    parents: int32 [children], the sequence that each continues; kv_lens, table: int32 [batch] and [batch, width];
    free_pages, used: the free list of ``kv_tables``; refs: int32 [pages], each page's holders beyond the first,
    changed in place; k_cache, v_cache: as ``kv_compact`` takes them.  A child shares its parent's full pages; the
    one that ends inside is copied to a page of its own.  Missing outputs are allocated; ``used_out=used`` works in
    place, and ``table_out`` may be further rows of table's matrix.  ``status`` stays on the device: 0, or a sum of
    1 (pool short), 2 (table too narrow), 8 (a bad length or parent), and 16 (a bad page, which is left out)."""
    dev = _device(parents, k_cache, v_cache)
    n, batch = _batch("parents", parents), _batch("kv_lens", kv_lens)
    dt, layers, pages, hkv, hd, ld_layer = _ops._caches(k_cache, v_cache, dev)
    ld_table, width = _ops._mat("table", table, _I32T, batch, None, dev), table.shape[1]
    if table_out is None:
        table_out = torch.empty((n, width), dtype=_I32T, device=table.device)
    if lens_out is None:
        lens_out = torch.empty(n, dtype=_I32T, device=table.device)
    if used_out is None:
        used_out = torch.empty(1, dtype=_I32T, device=table.device)
    if status is None:
        status = torch.empty(1, dtype=_I32T, device=table.device)
    n_free = free_pages.numel()
    p_par, p_kv, p_free, p_used, p_refs, p_lens, p_uo, p_status = _ops._ints(
        dev, "parents", parents, n, "kv_lens", kv_lens, batch, "free_pages", free_pages, n_free, "used", used, 1, "refs", refs,
        pages, "lens_out", lens_out, n, "used_out", used_out, 1, "status", status, 1)
    # (an empty list still has to be told from none at all)
    _call(load().dflash_kv_fork, _FORK.pack,
          (dt, batch, n, width, n_free, scratch_page, layers, pages, hkv, hd, ld_layer, ld_table,
           _ops._mat("table_out", table_out, _I32T, n, width, dev), k_cache.data_ptr(), v_cache.data_ptr(),
           p_par, p_kv, table.data_ptr(), p_free or p_status, p_used, p_refs, table_out.data_ptr(), p_lens, p_uo, p_status), dev)
    _ops._written(refs, k_cache, v_cache, table_out, lens_out, used_out, status)
    return KVFork(table_out, lens_out, used_out, status)


def kv_release(seqs, kv_lens, table, free_pages, used, refs, *, keep_lens=None, used_out=None, status=None) -> KVRelease:
    """The pages of ended or shortened sequences back to the free list (``dflash_kv_release``).

    seqs: int32 [n], the sequences that end; kv_lens, table: int32 [batch] and [batch, width]; free_pages, used, refs:
    as ``kv_fork``, free_pages and refs changed in place.  A page returns when its last holder leaves.  A sequence ends
    once: the counts do not tell free pages from held ones, and a later call that names it again puts its pages into
    the list twice.  With keep_lens (int32 [batch]) the sequences live on with so many tokens and give back the pages
    behind them: after a step of trees, kv_lens are the lengths with the trees and keep_lens ``kv_compact``'s.
    ``used_out=used`` works in place.  ``status`` stays on the device: 0, or a sum of 1 (more pages return than were
    taken), 2 (table too narrow), 8 (a bad length, used or sequence, or one named twice), 16 (a bad page), 32 (a page
    returned by more sequences of this call than hold it), 64 (a cut ends inside a page that others hold, which the next
    token would be written to: fork the sequence at the shorter length instead, and end it): nothing has changed."""
    dev = _device(seqs)
    n, batch = _batch("seqs", seqs), _batch("kv_lens", kv_lens)
    ld_table = _ops._mat("table", table, _I32T, batch, None, dev)
    if used_out is None:
        used_out = torch.empty(1, dtype=_I32T, device=table.device)
    if status is None:
        status = torch.empty(1, dtype=_I32T, device=table.device)
    n_free, pages = free_pages.numel(), refs.numel()
    p_seqs, p_kv, p_free, p_used, p_refs, p_uo, p_status = _ops._ints(
        dev, "seqs", seqs, n, "kv_lens", kv_lens, batch, "free_pages", free_pages, n_free, "used", used, 1, "refs", refs, pages,
        "used_out", used_out, 1, "status", status, 1)
    _call(load().dflash_kv_release, _RELEASE.pack,
          (batch, n, table.shape[1], n_free, pages, 0, ld_table, p_seqs, p_kv, table.data_ptr(), p_free or p_status, p_used,
           p_refs, p_uo, p_status, 0 if keep_lens is None else _ops._flat("keep_lens", keep_lens, _I32T, batch, dev)), dev)
    _ops._written(free_pages, refs, used_out, status)
    return KVRelease(used_out, status)
