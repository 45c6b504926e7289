"""Serving operators over torch tensors: argument checks and marshalling for the
stateless calls of the C ABI (include/dflash.h, "serving operators").

    kv_tables                page tables and slot maps of a batch from its request lengths
    shared_prefix_attention  attention of a batch whose sequences share a prefix
    process_logits           penalties for repeated tokens, biases and grammar masks on logits

Every call queues its kernels on torch's current stream of the tensors' device and
returns without synchronising.  None has a gradient: tensors that require one are
refused while autograd is recording."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

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


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _same_device(first, tensors):
    """The one CUDA device of the call; gradients are refused."""
    dev = first.device
    _need(dev.type == "cuda", "the operators run on CUDA tensors only")
    grad = torch.is_grad_enabled()
    for name, t in tensors:
        if t is None:
            continue
        _need(t.device == dev, f"{name} is on {t.device}, not on {dev}")
        _need(not (grad and t.requires_grad), f"{name} requires a gradient, which this operator has not")
    return dev


def _vec(name, t, dtype, n):
    _need(t.dtype == dtype and t.dim() == 1 and t.shape[0] == n and t.is_contiguous(),
          f"{name} must be a contiguous {dtype} tensor of {n}")


def _mat(name, t, dtype, rows, cols=None):
    """A row-major matrix (any row stride); its row stride in elements."""
    _need(t.dtype == dtype and t.dim() == 2 and t.shape[0] == rows and (cols is None or t.shape[1] == cols),
          f"{name} must be a {dtype} matrix of {rows} rows" + ("" if cols is None else f" and {cols} columns"))
    if t.shape[1] <= 1 or t.shape[0] == 0:
        return max(t.stride(0), t.shape[1]) if rows > 1 else t.shape[1]
    _need(t.stride(1) == 1 and (rows <= 1 or t.stride(0) >= t.shape[1]), f"{name} must be row-major")
    return t.stride(0) if rows > 1 else t.shape[1]


def _call(fn, args, dev):
    stream = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev.index:
        st = fn(ctypes.byref(args), stream)
    else:
        with torch.cuda.device(dev):
            st = fn(ctypes.byref(args), stream)
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
    batch = kv_lens.shape[0] if kv_lens.dim() == 1 else 0
    _need(1 <= batch <= OPS_MAX_BATCH, f"kv_lens must be a vector of 1 to {OPS_MAX_BATCH} lengths")
    dev = _same_device(kv_lens, (("new_lens", new_lens), ("table", table), ("free_pages", free_pages), ("used", used),
                                 ("table_out", table_out), ("used_out", used_out), ("q_start", q_start),
                                 ("row_seq", row_seq), ("row_pos", row_pos), ("slots", slots), ("status", status)))
    i32 = torch.int32
    _vec("kv_lens", kv_lens, i32, batch)
    _vec("new_lens", new_lens, i32, batch)
    ld = _mat("table", table, i32, batch)
    width = table.shape[1]
    for t in (row_seq, row_pos, slots):
        if t is not None:
            _need(rows is None or rows == t.shape[0], "row_seq, row_pos and slots must have `rows` entries")
            rows = t.shape[0]
    _need(rows is not None and rows >= 0, "rows is needed when no row map is given")
    new = lambda n, dt=i32: torch.empty(n, dtype=dt, device=dev)  # noqa: E731
    q_start = new(batch + 1) if q_start is None else q_start
    row_seq = new(rows) if row_seq is None else row_seq
    row_pos = new(rows) if row_pos is None else row_pos
    slots = new(rows, torch.int64) if slots is None else slots
    status = new(1) if status is None else status
    for name, t, dt, n in (("q_start", q_start, i32, batch + 1), ("row_seq", row_seq, i32, rows),
                           ("row_pos", row_pos, i32, rows), ("slots", slots, torch.int64, rows),
                           ("status", status, i32, 1)):
        _vec(name, t, dt, n)
    ld_out, n_free = ld, 0
    if free_pages is not None:
        n_free = free_pages.shape[0] if free_pages.dim() == 1 else -1
        _need(used is not None, "free_pages needs used")
        _vec("free_pages", free_pages, i32, n_free)
        _vec("used", used, i32, 1)
        table_out = torch.empty((batch, width), dtype=i32, device=dev) if table_out is None else table_out
        used_out = new(1) if used_out is None else used_out
        _vec("used_out", used_out, i32, 1)
    else:
        _need(used is None and used_out is None, "used and used_out need free_pages")
    if table_out is not None:
        ld_out = _mat("table_out", table_out, i32, batch, width)
    # an empty free list still has to be told from none at all
    free = None if free_pages is None else (free_pages.data_ptr() or status.data_ptr())
    args = dflash_kv_tables_args(batch, width, rows, n_free, base_pos, scratch_page, ld, ld_out, kv_lens.data_ptr(),
                                 new_lens.data_ptr(), _ptr(table), free, _ptr(used), _ptr(table_out), _ptr(used_out),
                                 q_start.data_ptr(), _ptr(row_seq), _ptr(row_pos), _ptr(slots), status.data_ptr())
    _call(load().dflash_kv_tables, args, dev)
    return KVTables(table_out, used_out, q_start, row_seq, row_pos, slots, status)


def _rows3(name, t, rows, heads, hd):
    """Row stride of a [rows, heads, hd] tensor whose rows are contiguous."""
    _need(t.dim() == 3 and tuple(t.shape) == (rows, heads, hd), f"{name} must be [{rows}, {heads}, {hd}]")
    if rows == 0:
        return heads * hd
    _need(t.stride(2) == 1 and (heads == 1 or t.stride(1) == hd), f"{name}: the heads of a row must be contiguous")
    return t.stride(0) if rows > 1 else heads * hd


def shared_prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len: int, table, kv_lens, q_start, *,
                            causal: bool = True, scale: Optional[float] = None, out=None, lse=None,
                            workspace=None):
    """Attention of a batch whose sequences share a prefix (``dflash_shared_prefix_attention``).

    q: [rows, H, hd] (fp32 or bf16); k_cache, v_cache: [pages, H_kv, 64, hd]; prefix_pages: int32, the
    prefix's pages (None for an empty prefix); table: int32 [batch, width], each sequence's own pages;
    kv_lens: int32 [batch], its own keys; q_start: int32 [batch + 1], its rows.  ``scale`` defaults to
    hd ** -0.5.  Returns (out, lse); rows outside q_start keep what ``out`` and ``lse`` held (0 where they
    are allocated here)."""
    _need(q.dim() == 3 and k_cache.dim() == 4, "q must be [rows, H, hd] and the caches [pages, H_kv, 64, hd]")
    rows, h, hd = q.shape
    pages, hkv = k_cache.shape[0], k_cache.shape[1]
    dev = _same_device(q, (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("prefix_pages", prefix_pages),
                           ("table", table), ("kv_lens", kv_lens), ("q_start", q_start), ("out", out), ("lse", lse),
                           ("workspace", workspace)))
    dt = _DTYPES.get(q.dtype)
    _need(dt is not None, f"q must be float32 or bfloat16, not {q.dtype}")
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(c.dtype == q.dtype and tuple(c.shape) == (pages, hkv, PAGE_TOKENS, hd) and c.is_contiguous(),
              f"{name} must be a contiguous {q.dtype} [pages, H_kv, {PAGE_TOKENS}, {hd}]")
    batch = kv_lens.shape[0] if kv_lens.dim() == 1 else 0
    _need(1 <= batch <= OPS_MAX_BATCH, f"kv_lens must be a vector of 1 to {OPS_MAX_BATCH} lengths")
    _vec("kv_lens", kv_lens, torch.int32, batch)
    _vec("q_start", q_start, torch.int32, batch + 1)
    prefix_len = int(prefix_len)
    n_pre = (prefix_len + PAGE_TOKENS - 1) // PAGE_TOKENS
    if prefix_pages is not None:
        _need(prefix_pages.dtype == torch.int32 and prefix_pages.dim() == 1 and prefix_pages.is_contiguous()
              and prefix_pages.shape[0] >= n_pre, f"prefix_pages must be a contiguous int32 tensor of at least {n_pre}")
    else:
        _need(prefix_len == 0, "prefix_pages is needed for a prefix")
    ld_table = _mat("table", table, torch.int32, batch)
    ld_q = _rows3("q", q, rows, h, hd)
    out = torch.zeros((rows, h, hd), dtype=q.dtype, device=dev) if out is None else out
    _need(out.dtype == q.dtype, f"out must be {q.dtype}")
    ld_out = _rows3("out", out, rows, h, hd)
    lse = torch.zeros((rows, h), dtype=torch.float32, device=dev) if lse is None else lse
    _need(lse.dtype == torch.float32 and tuple(lse.shape) == (rows, h) and lse.is_contiguous(),
          f"lse must be a contiguous float32 [{rows}, {h}]")
    lib = load()
    if workspace is None:
        workspace = torch.empty(lib.dflash_shared_prefix_workspace(dt, h, hkv, hd, batch, rows), dtype=torch.uint8,
                                device=dev)
    _need(workspace.is_contiguous(), "workspace must be contiguous")
    args = dflash_shared_prefix_args(dt, h, hkv, hd, batch, rows, pages, prefix_len, table.shape[1], bool(causal),
                                     hd ** -0.5 if scale is None else scale, 0, ld_q, ld_out, ld_table, q.data_ptr(),
                                     k_cache.data_ptr(), v_cache.data_ptr(), _ptr(prefix_pages), table.data_ptr(),
                                     kv_lens.data_ptr(), q_start.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                     workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _call(lib.dflash_shared_prefix_attention, args, dev)
    return out, lse


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
    _need(logits.dim() == 2, "logits must be [rows, vocab]")
    n, vocab = logits.shape
    _need(1 <= rows_per_seq <= 32 and n % rows_per_seq == 0, "rows_per_seq must be in [1, 32] and divide the rows")
    batch = n // rows_per_seq
    _need(1 <= batch <= OPS_MAX_BATCH, f"1 to {OPS_MAX_BATCH} sequences")
    dev = _same_device(logits, (("logits", logits), ("history", history), ("hist_lens", hist_lens),
                                ("prompt_lens", prompt_lens), ("drafts", drafts), ("repetition", repetition),
                                ("presence", presence), ("frequency", frequency), ("bias_ids", bias_ids),
                                ("bias_values", bias_values), ("masks", masks), ("mask_index", mask_index),
                                ("out", out)))
    dt = _DTYPES.get(logits.dtype)
    _need(dt is not None, f"logits must be float32 or bfloat16, not {logits.dtype}")
    out = torch.empty((n, vocab), dtype=logits.dtype, device=dev) if out is None else out
    ld = _mat("logits", logits, logits.dtype, n)
    ld_out = _mat("out", out, logits.dtype, n, vocab)
    i32, f32 = torch.int32, torch.float32
    hist_width = bias_width = n_masks = ld_hist = ld_mask = 0
    if history is not None:
        _need(hist_lens is not None and prompt_lens is not None, "history needs hist_lens and prompt_lens")
        ld_hist = _mat("history", history, i32, batch)
        hist_width = history.shape[1]
        _vec("hist_lens", hist_lens, i32, batch)
        _vec("prompt_lens", prompt_lens, i32, batch)
        for name, t in (("repetition", repetition), ("presence", presence), ("frequency", frequency)):
            if t is not None:
                _vec(name, t, f32, batch)
        if drafts is not None:
            _need(rows_per_seq > 1, "drafts need more than one row a sequence")
            _mat("drafts", drafts, i32, batch, rows_per_seq - 1)
            _need(drafts.is_contiguous(), "drafts must be contiguous")
    else:
        _need(hist_lens is None and prompt_lens is None and drafts is None and repetition is None and presence is None
              and frequency is None, "penalties and drafts need a history")
    if bias_ids is not None:
        _need(bias_values is not None, "bias_ids needs bias_values")
        bias_width = bias_ids.shape[1] if bias_ids.dim() == 2 else 0
        _mat("bias_ids", bias_ids, i32, batch, bias_width)
        _mat("bias_values", bias_values, f32, batch, bias_width)
        _need(bias_ids.is_contiguous() and bias_values.is_contiguous(), "bias_ids and bias_values must be contiguous")
    else:
        _need(bias_values is None, "bias_values needs bias_ids")
    if masks is not None:
        _need(mask_index is not None, "masks need mask_index")
        n_masks = masks.shape[0]
        ld_mask = _mat("masks", masks, i32, n_masks)
        _need(masks.shape[1] * 32 >= vocab, "a mask must hold a bit for every token")
        _vec("mask_index", mask_index, i32, n)
    else:
        _need(mask_index is None, "mask_index needs masks")
    # an empty list (no column, no mask) leaves its group out
    args = dflash_logits_args(dt, batch, rows_per_seq, vocab, hist_width, bias_width, n_masks, 0, ld, ld_out, ld_hist,
                              ld_mask, logits.data_ptr(), out.data_ptr(),
                              None if history is None else (history.data_ptr() or hist_lens.data_ptr()), _ptr(hist_lens),
                              _ptr(prompt_lens), _ptr(drafts), _ptr(repetition), _ptr(presence), _ptr(frequency),
                              _ptr(bias_ids) if bias_width else None, _ptr(bias_values),
                              _ptr(masks) if n_masks else None, _ptr(mask_index))
    _call(load().dflash_process_logits, args, dev)
    return out
