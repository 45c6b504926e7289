"""Serving operators over torch tensors: argument checks and marshalling for the
stateless calls of the C ABI (include/dflash.h, "serving operators").

    kv_tables                page tables and slot maps of a batch from its request lengths
    shared_prefix_attention  attention of a batch whose sequences share a prefix
    process_logits           penalties for repeated tokens, biases and grammar masks on logits

Every call queues its kernels on torch's current stream of the tensors' device and
returns without synchronising.  None has a gradient: tensors that require one, outputs
among them, are refused while autograd is recording, and so are tensors with a
forward-mode tangent.  Outputs of the caller's count as written in place (their versions
rise)."""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
import threading
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad as _forward_ad

from . import build as _build_mod
from . import DFLASH_DTYPE_BF16, DFLASH_DTYPE_F32, DFLASH_OK, DFlashError, dflash_last_error, load

_P, _I32, _I64, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
OPS_MAX_BATCH = 2048
PAGE_TOKENS = 64
_DTYPES = {torch.float32: DFLASH_DTYPE_F32, torch.bfloat16: DFLASH_DTYPE_BF16}


class dflash_kv_tables_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("batch", "width", "rows", "n_free", "base_pos", "scratch_page")]
                + [(n, _I64) for n in ("ld_table", "ld_out")]
                + [(n, _P) for n in ("kv_lens", "new_lens", "table", "free_pages", "used", "table_out", "used_out",
                                     "q_start", "row_seq", "row_pos", "slots", "status")])


class dflash_shared_prefix_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "n_heads", "n_kv_heads", "head_dim", "batch", "rows", "n_pages",
                                     "prefix_len", "width", "causal")]
                + [("scale", _F), ("reserved", _I32)]
                + [(n, _I64) for n in ("ld_q", "ld_out", "ld_table")]
                + [(n, _P) for n in ("q", "k_cache", "v_cache", "prefix_pages", "table", "kv_lens", "q_start", "out",
                                     "lse", "workspace")]
                + [("workspace_bytes", ctypes.c_size_t)])


class dflash_logits_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "batch", "rows_per_seq", "vocab", "hist_width", "bias_width", "n_masks",
                                     "reserved")]
                + [(n, _I64) for n in ("ld_logits", "ld_out", "ld_hist", "ld_mask")]
                + [(n, _P) for n in ("logits", "out", "history", "hist_lens", "prompt_lens", "drafts", "repetition",
                                     "presence", "frequency", "bias_ids", "bias_values", "masks", "mask_index")])


class KVTables(NamedTuple):
    table: Optional[torch.Tensor]
    used: Optional[torch.Tensor]
    q_start: torch.Tensor
    row_seq: torch.Tensor
    row_pos: torch.Tensor
    slots: torch.Tensor
    status: torch.Tensor


# Every call packs its argument struct with one of these (a fraction of a ctypes.Structure's cost: the
# small calls are as long as their host side) and passes the bytes.
_TABLES, _ATTN, _LOGITS = struct.Struct("6i2q12Q"), struct.Struct("10ifi3q11Q"), struct.Struct("8i4q13Q")
_I32T, _I64T, _F32T = torch.int32, torch.int64, torch.float32
_U8T = torch.uint8
_WORKSPACE = {}  # bytes by (dtype, H, H_kv, hd, batch, rows)
# Workspaces of calls on a device's default stream, one a device: (bytes, address, tensor).  That stream is never
# captured and lives as long as the device; on any other stream each call allocates its own.  An allocation beside a call
# costs 5 us of the 17 that a small one takes.  A call queues two kernels, the second of which reads what the first left in
# the workspace, and the C call runs without the interpreter's lock: so a call that uses a kept workspace holds _KEPT_LOCK
# from looking it up until both are queued (the stream then runs the calls one after the other, whichever threads made
# them).  Re-entrant, for a call out of a signal handler or a finalizer.  Kept up to KEPT_MAX bytes (32 verify blocks of 16 rows
# of 32 heads take 92 MB): calls that need more run for hundreds of microseconds and allocate theirs.
KEPT_MAX = 256 << 20
_KEPT = {}
_KEPT_LOCK = threading.RLock()
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device


def _bad(msg):
    raise ValueError(msg)


def _device(first, *floats):
    """Index of the one CUDA device of the call; floating tensors that record a gradient are refused."""
    dev = first.get_device()
    if dev < 0:
        _bad("the operators run on CUDA tensors only")
    if torch.is_grad_enabled():
        for t in floats:
            if t is not None and t.requires_grad:
                _bad("a tensor requires a gradient, which these operators do not have")
    if _forward_ad._current_level >= 0:
        for t in floats:
            if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
                _bad("a tensor carries a forward-mode tangent, which these operators do not have")
    return dev


def _flat(name, t, dtype, n, dev):
    """Address of a contiguous tensor of n elements on the device."""
    if t.dtype is not dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        _bad(f"{name} must be a contiguous {dtype} tensor of {n} elements on cuda:{dev}, "
             f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _mat(name, t, dtype, rows, cols, dev):
    """Row stride, in elements, of a row-major matrix on the device (cols None: any)."""
    if t.dtype is not dtype or t.dim() != 2 or t.get_device() != dev:
        _bad(f"{name} must be a {dtype} matrix on cuda:{dev}, not {t.dtype} {tuple(t.shape)} on {t.device}")
    n, m = t.shape
    if n != rows or (cols is not None and m != cols):
        _bad(f"{name} must be [{rows}, {'any' if cols is None else cols}], not [{n}, {m}]")
    if t.is_contiguous():
        return m
    ld, inner = t.stride()
    if n <= 1 or m == 0:
        ld = m
    if (inner != 1 and m > 1) or ld < m:
        _bad(f"{name} must be row-major")
    return ld


def _rows3(name, t, dtype, rows, heads, hd, dev):
    """Row stride of a [rows, heads, hd] tensor whose rows are contiguous."""
    if t.dtype is not dtype or t.shape != (rows, heads, hd) or t.get_device() != dev:
        _bad(f"{name} must be a {dtype} [{rows}, {heads}, {hd}] on cuda:{dev}, "
             f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return heads * hd
    ld, between, inner = t.stride()
    if inner != 1 or (heads > 1 and between != hd):
        _bad(f"{name}: the heads of a row must be contiguous")
    return ld if rows > 1 else heads * hd


def _written(*tensors):
    """The tensors (or None) have been written to: their versions rise."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


_PYTHON_CHECKS = (_flat, _mat, _rows3)
_PYTHON_WRITTEN = _written


def _use_extension():
    """The same three checks (and _written) from csrc/tensor_args.cpp, where it has been built (a small call's host side is
    shorter by a third)."""
    global _flat, _mat, _rows3, _written
    path = _build_mod.tensor_args_path()
    if path is None or not os.path.exists(path):
        return
    try:
        spec = importlib.util.spec_from_loader("_tensor_args", importlib.machinery.ExtensionFileLoader("_tensor_args", path))
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        _flat, _mat, _rows3, _written = m.flat, m.mat, m.rows3, m.written
    except (ImportError, AttributeError):  # (AttributeError: built from an older source)
        return


_use_extension()


def _call(fn, pack, values, dev):
    try:
        args = pack(*values)
    except struct.error as e:
        raise ValueError(f"an integer argument is out of its range or no integer: {e}") from None
    if _current_device() == dev:
        st = fn(args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(args, _raw_stream(dev))
    if st != DFLASH_OK:
        raise DFlashError(st, dflash_last_error(None))


def kv_tables(kv_lens, new_lens, table, free_pages=None, used=None, *, rows: Optional[int] = None, scratch_page: int = 0,
              base_pos: int = 0, table_out=None, used_out=None, q_start=None, row_seq=None, row_pos=None, slots=None,
              status=None) -> KVTables:
    """Page tables and slot maps of a batch (``dflash_kv_tables``).

    kv_lens, new_lens: int32 [batch], tokens cached and tokens to append.  table: int32 [batch, width],
    the pages held.  free_pages: int32 list of free pages of which the first ``used[0]`` are taken
    (None: the table already backs every new token and no page is taken).  rows: capacity of the row
    maps (default: that of ``row_seq`` / ``row_pos`` / ``slots``).  Missing outputs are allocated;
    ``table_out=table`` and ``used_out=used`` work in place.  ``status`` stays on the device: 0, or a
    sum of 1 (pool short), 2 (table too narrow), 4 (more new rows than ``rows``), 8 (negative length)."""
    dev = _device(kv_lens)
    batch = kv_lens.numel()
    if not 1 <= batch <= OPS_MAX_BATCH:
        _bad(f"kv_lens must hold 1 to {OPS_MAX_BATCH} lengths")
    p_kv, p_new = _flat("kv_lens", kv_lens, _I32T, batch, dev), _flat("new_lens", new_lens, _I32T, batch, dev)
    ld = ld_out = _mat("table", table, _I32T, batch, None, dev)
    width = table.shape[1]
    if rows is None:
        for t in (row_seq, row_pos, slots):
            if t is not None:
                rows = t.numel()
        if rows is None:
            _bad("rows is needed when no row map is given")
    elif rows < 0:
        _bad("rows must not be negative")
    if q_start is None:
        q_start = torch.empty(batch + 1, dtype=_I32T, device=kv_lens.device)
    if row_seq is None:
        row_seq = torch.empty(rows, dtype=_I32T, device=kv_lens.device)
    if row_pos is None:
        row_pos = torch.empty(rows, dtype=_I32T, device=kv_lens.device)
    if slots is None:
        slots = torch.empty(rows, dtype=_I64T, device=kv_lens.device)
    if status is None:
        status = torch.empty(1, dtype=_I32T, device=kv_lens.device)
    p_status = _flat("status", status, _I32T, 1, dev)
    n_free = p_free = p_used = p_out = p_uo = 0
    if free_pages is not None:
        if used is None:
            _bad("free_pages needs used")
        n_free = free_pages.numel()
        # (an empty list still has to be told from none at all)
        p_free = _flat("free_pages", free_pages, _I32T, n_free, dev) or p_status
        p_used = _flat("used", used, _I32T, 1, dev)
        if table_out is None:
            table_out = torch.empty((batch, width), dtype=_I32T, device=kv_lens.device)
        if used_out is None:
            used_out = torch.empty(1, dtype=_I32T, device=kv_lens.device)
        p_uo = _flat("used_out", used_out, _I32T, 1, dev)
    elif used is not None or used_out is not None:
        _bad("used and used_out need free_pages")
    if table_out is not None:
        ld_out = _mat("table_out", table_out, _I32T, batch, width, dev)
        p_out = table_out.data_ptr()
    _call(load().dflash_kv_tables,
          _TABLES.pack, (batch, width, rows, n_free, base_pos, scratch_page, ld, ld_out, p_kv, p_new, table.data_ptr(), p_free,
                       p_used, p_out, p_uo, _flat("q_start", q_start, _I32T, batch + 1, dev),
                       _flat("row_seq", row_seq, _I32T, rows, dev), _flat("row_pos", row_pos, _I32T, rows, dev),
                       _flat("slots", slots, _I64T, rows, dev), p_status), dev)
    _written(table_out, used_out, q_start, row_seq, row_pos, slots, status)
    return KVTables(table_out, used_out, q_start, row_seq, row_pos, slots, status)


def shared_prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len: int, table, kv_lens, q_start, *,
                            causal: bool = True, scale: Optional[float] = None, out=None, lse=None,
                            workspace=None, weight_pairs: bool = False):
    """Attention of a batch whose sequences share a prefix (``dflash_shared_prefix_attention``).

    q: [rows, H, hd] (fp32 or bf16); k_cache, v_cache: [pages, H_kv, 64, hd]; prefix_pages: int32, the
    prefix's pages (None for an empty prefix); table: int32 [batch, width], each sequence's own pages;
    kv_lens: int32 [batch], its own keys; q_start: int32 [batch + 1], its rows.  ``scale`` defaults to
    hd ** -0.5.  Returns (out, lse); rows outside q_start keep what ``out`` and ``lse`` held (0 where they
    are allocated here).  ``workspace``: uint8, at least ``shared_prefix_workspace`` bytes; calls that may
    run at the same time need one each.  None: allocated for the call, or on a device's default stream the
    largest one of up to 256 MB needed there so far, which is kept.  ``weight_pairs``: bf16 calls hold each
    softmax weight as a bf16 pair (16 bits) instead of one bf16 (8 bits) for the product with v."""
    if q.dim() != 3 or k_cache.dim() != 4:
        _bad("q must be [rows, H, hd] and the caches [pages, H_kv, 64, hd]")
    dev = _device(q, q, k_cache, v_cache, out, lse)
    rows, h, hd = q.shape
    kv_shape = k_cache.shape
    pages, hkv, page_tokens, kv_hd = kv_shape
    dtype = q.dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        _bad(f"q must be float32 or bfloat16, not {dtype}")
    n_kv = pages * hkv * PAGE_TOKENS * hd
    if page_tokens != PAGE_TOKENS or kv_hd != hd or v_cache.shape != kv_shape:
        _bad(f"k_cache and v_cache must be [pages, H_kv, {PAGE_TOKENS}, {hd}]")
    p_k, p_v = _flat("k_cache", k_cache, dtype, n_kv, dev), _flat("v_cache", v_cache, dtype, n_kv, dev)
    batch = kv_lens.numel()
    if not 1 <= batch <= OPS_MAX_BATCH:
        _bad(f"kv_lens must hold 1 to {OPS_MAX_BATCH} lengths")
    p_kv, p_start = _flat("kv_lens", kv_lens, _I32T, batch, dev), _flat("q_start", q_start, _I32T, batch + 1, dev)
    p_pre = 0
    if prefix_pages is not None:
        n_pre = prefix_pages.numel()
        p_pre = _flat("prefix_pages", prefix_pages, _I32T, n_pre, dev)
        if n_pre * PAGE_TOKENS < prefix_len:
            _bad(f"prefix_pages holds {n_pre} pages, too few for {prefix_len} tokens")
    elif prefix_len != 0:
        _bad("prefix_pages is needed for a prefix")
    ld_table = _mat("table", table, _I32T, batch, None, dev)
    ld_q = _rows3("q", q, dtype, rows, h, hd, dev)
    if out is None:
        out = torch.zeros((rows, h, hd), dtype=dtype, device=q.device)
    ld_out = _rows3("out", out, dtype, rows, h, hd, dev)
    if lse is None:
        lse = torch.zeros((rows, h), dtype=_F32T, device=q.device)
    fn = load().dflash_shared_prefix_attention
    args = (dt, h, hkv, hd, batch, rows, pages, prefix_len, table.shape[1], bool(causal), hd ** -0.5 if scale is None else scale,
            1 if weight_pairs else 0,
            ld_q, ld_out, ld_table, q.data_ptr(), p_k, p_v, p_pre, table.data_ptr(), p_kv, p_start, out.data_ptr(),
            _flat("lse", lse, _F32T, rows * h, dev))
    if workspace is not None:
        n_ws = workspace.numel() * workspace.element_size()
        _call(fn, _ATTN.pack, (*args, _flat("workspace", workspace, workspace.dtype, workspace.numel(), dev), n_ws), dev)
    else:
        sizes = (dt, h, hkv, hd, batch, rows)
        n_ws = _WORKSPACE.get(sizes)
        if n_ws is None:
            if len(_WORKSPACE) > 4096:
                _WORKSPACE.clear()
            n_ws = _WORKSPACE[sizes] = load().dflash_shared_prefix_workspace(*sizes)
        if n_ws > KEPT_MAX or _raw_stream(dev) != 0:
            workspace = torch.empty(n_ws, dtype=_U8T, device=q.device)
            _call(fn, _ATTN.pack, (*args, workspace.data_ptr(), n_ws), dev)
        else:
            with _KEPT_LOCK:
                kept = _KEPT.get(dev)
                if kept is None or kept[0] < n_ws:
                    workspace = torch.empty(n_ws, dtype=_U8T, device=q.device)
                    kept = _KEPT[dev] = (n_ws, workspace.data_ptr(), workspace)
                _call(fn, _ATTN.pack, (*args, kept[1], n_ws), dev)
    _written(out, lse)
    return out, lse


def shared_prefix_workspace(q, k_cache, batch: int) -> int:
    """Bytes of workspace that a call of ``shared_prefix_attention`` with these tensors needs."""
    return load().dflash_shared_prefix_workspace(_DTYPES[q.dtype], q.shape[1], k_cache.shape[1], q.shape[2], batch,
                                                 q.shape[0])


def process_logits(logits, *, rows_per_seq: int = 1, history=None, hist_lens=None, prompt_lens=None, drafts=None,
                   repetition=None, presence=None, frequency=None, bias_ids=None, bias_values=None, masks=None,
                   mask_index=None, out=None):
    """Penalties, biases and grammar masks on logits (``dflash_process_logits``).

    logits: [batch * rows_per_seq, vocab] (fp32 or bf16), rows sequence-major.  history: int32
    [batch, width] token ids with hist_lens and prompt_lens [batch]; drafts: int32
    [batch, rows_per_seq - 1], the tokens between a sequence's rows; repetition, presence, frequency:
    fp32 [batch]; bias_ids / bias_values: [batch, n] (id -1: unused; the last entry of an id counts);
    masks: int32 bit sets [n_masks, >= ceil(vocab / 32)] with mask_index int32 [rows] (-1: none).
    Returns ``out`` (allocated when None; ``out=logits`` works in place)."""
    if logits.dim() != 2:
        _bad("logits must be [rows, vocab]")
    dev = _device(logits, logits, repetition, presence, frequency, bias_values, out)
    n, vocab = logits.shape
    dtype = logits.dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        _bad(f"logits must be float32 or bfloat16, not {dtype}")
    if not 1 <= rows_per_seq <= 32 or n % rows_per_seq:
        _bad("rows_per_seq must be in [1, 32] and divide the rows")
    batch = n // rows_per_seq
    if not 1 <= batch <= OPS_MAX_BATCH:
        _bad(f"1 to {OPS_MAX_BATCH} sequences")
    if out is None:
        out = torch.empty((n, vocab), dtype=dtype, device=logits.device)
    ld, ld_out = _mat("logits", logits, dtype, n, vocab, dev), _mat("out", out, dtype, n, vocab, dev)
    hist_width = bias_width = n_masks = ld_hist = ld_mask = 0
    p_hist = p_len = p_prompt = p_draft = p_rep = p_pres = p_freq = p_ids = p_val = p_mask = p_idx = 0
    if history is not None:
        if hist_lens is None or prompt_lens is None:
            _bad("history needs hist_lens and prompt_lens")
        ld_hist = _mat("history", history, _I32T, batch, None, dev)
        hist_width = history.shape[1]
        p_len, p_prompt = _flat("hist_lens", hist_lens, _I32T, batch, dev), _flat("prompt_lens", prompt_lens, _I32T, batch, dev)
        p_hist = history.data_ptr() or p_len  # (an empty history still has to be told from none at all)
        if repetition is not None:
            p_rep = _flat("repetition", repetition, _F32T, batch, dev)
        if presence is not None:
            p_pres = _flat("presence", presence, _F32T, batch, dev)
        if frequency is not None:
            p_freq = _flat("frequency", frequency, _F32T, batch, dev)
        if drafts is not None:
            if rows_per_seq == 1:
                _bad("drafts need more than one row a sequence")
            p_draft = _flat("drafts", drafts, _I32T, batch * (rows_per_seq - 1), dev)
    elif any(t is not None for t in (hist_lens, prompt_lens, drafts, repetition, presence, frequency)):
        _bad("penalties and drafts need a history")
    if bias_ids is not None:
        if bias_values is None:
            _bad("bias_ids needs bias_values")
        bias_width = bias_ids.numel() // batch
        p_ids = _flat("bias_ids", bias_ids, _I32T, batch * bias_width, dev)
        p_val = _flat("bias_values", bias_values, _F32T, batch * bias_width, dev)
    elif bias_values is not None:
        _bad("bias_values needs bias_ids")
    if masks is not None:
        if mask_index is None:
            _bad("masks need mask_index")
        n_masks = masks.shape[0]
        ld_mask = _mat("masks", masks, _I32T, n_masks, None, dev)
        if masks.shape[1] * 32 < vocab:
            _bad("a mask must hold a bit for every token")
        ld_mask = max(ld_mask, masks.shape[1])
        p_mask, p_idx = masks.data_ptr(), _flat("mask_index", mask_index, _I32T, n, dev)
    elif mask_index is not None:
        _bad("mask_index needs masks")
    _call(load().dflash_process_logits,
          _LOGITS.pack, (dt, batch, rows_per_seq, vocab, hist_width, bias_width, n_masks, 0, ld, ld_out, ld_hist, ld_mask,
                       logits.data_ptr(), out.data_ptr(), p_hist, p_len, p_prompt, p_draft, p_rep, p_pres, p_freq,
                       p_ids if bias_width else 0, p_val, p_mask if n_masks else 0, p_idx), dev)
    _written(out)
    return out
