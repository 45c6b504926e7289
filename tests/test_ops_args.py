"""Refusals of the serving operators, host side (no GPU): every bad argument is E_INVAL with a reason,
and the ctypes mirrors of the argument structs have the header's layout."""
import ctypes
import os
import subprocess

import pytest

import block_diffusion_speculative_ctx_gb300 as dfl
from block_diffusion_speculative_ctx_gb300 import build as dbuild

ops = pytest.importorskip("block_diffusion_speculative_ctx_gb300.ops")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return dfl.load()


def test_struct_layouts_match_the_header(tmp_path):
    prog = tmp_path / "sz.c"
    structs = (ops.dflash_kv_tables_args, ops.dflash_shared_prefix_args, ops.dflash_logits_args)
    names = [f"sizeof({s.__name__})" for s in structs]
    names += [f"offsetof({s.__name__}, {f[0]})" for s in structs for f in s._fields_]
    prog.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"dflash.h\"\nint main(void) {\n"
                    + "".join(f'  printf("%zu\\n", (size_t){n});\n' for n in names) + "  return 0;\n}\n")
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = [ctypes.sizeof(s) for s in structs] + [getattr(s, f[0]).offset for s in structs for f in s._fields_]
    assert got == want
    # the packed form that the calls pass
    assert [ops._TABLES.size, ops._ATTN.size, ops._LOGITS.size] == want[:3]


P = 4096  # stands for a device pointer (never read: every call here is refused)


def tables(**kw):
    d = dict(batch=2, width=4, rows=8, n_free=4, base_pos=0, scratch_page=0, ld_table=4, ld_out=4, kv_lens=P, new_lens=P,
             table=P, free_pages=P, used=P, table_out=2 * P, used_out=P, q_start=P, row_seq=P, row_pos=P, slots=P, status=P)
    d.update(kw)
    return ops.dflash_kv_tables_args(**d)


def attn(**kw):
    d = dict(dtype=1, n_heads=8, n_kv_heads=2, head_dim=128, batch=2, rows=4, n_pages=16, prefix_len=100, width=2, causal=1,
             scale=0.1, reserved=0, ld_q=1024, ld_out=1024, ld_table=2, q=P, k_cache=P, v_cache=P, prefix_pages=P, table=P,
             kv_lens=P, q_start=P, out=P, lse=P, workspace=P, workspace_bytes=1 << 40)
    d.update(kw)
    return ops.dflash_shared_prefix_args(**d)


def rules(**kw):
    d = dict(dtype=0, batch=2, rows_per_seq=4, vocab=1000, hist_width=8, bias_width=3, n_masks=2, reserved=0, ld_logits=1000,
             ld_out=1000, ld_hist=8, ld_mask=32, logits=P, out=P, history=P, hist_lens=P, prompt_lens=P, drafts=P,
             repetition=P, presence=P, frequency=P, bias_ids=P, bias_values=P, masks=P, mask_index=P)
    d.update(kw)
    return ops.dflash_logits_args(**d)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=2049), dict(width=-1), dict(rows=-1), dict(rows=1 << 30), dict(n_free=-1), dict(width=1 << 25),
    dict(base_pos=-1), dict(kv_lens=None), dict(new_lens=None), dict(q_start=None), dict(status=None), dict(table=None),
    dict(ld_table=3), dict(ld_out=3), dict(used=None), dict(used_out=None), dict(table_out=None),
    dict(table_out=P, ld_out=5)])
def test_kv_tables_refuses(lib, kw):
    assert lib.dflash_kv_tables(ctypes.byref(tables(**kw)), None) == dfl.DFLASH_E_INVAL
    assert "kv_tables" in dfl.dflash_last_error(None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(head_dim=96), dict(n_heads=9), dict(n_kv_heads=0), dict(n_heads=130, ld_q=130 * 128, ld_out=130 * 128),
    dict(n_heads=2048, n_kv_heads=2048, ld_q=1 << 18, ld_out=1 << 18), dict(batch=0), dict(batch=2049), dict(rows=-1),
    dict(rows=(1 << 20) + 1), dict(n_pages=0), dict(n_pages=1 << 24), dict(prefix_len=-1), dict(width=-1), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(k_cache=None), dict(v_cache=None),
    dict(kv_lens=None), dict(q_start=None), dict(table=None), dict(prefix_pages=None), dict(out=None), dict(workspace=None),
    dict(q=P + 8), dict(k_cache=P + 2), dict(v_cache=P + 4), dict(out=P + 8), dict(workspace=P + 1), dict(ld_q=1016),
    dict(ld_q=1028), dict(ld_out=1000), dict(ld_table=1), dict(workspace_bytes=0)])
def test_shared_prefix_attention_refuses(lib, kw):
    assert lib.dflash_shared_prefix_attention(ctypes.byref(attn(**kw)), None) == dfl.DFLASH_E_INVAL
    assert "shared_prefix_attention" in dfl.dflash_last_error(None)


def test_shared_prefix_workspace_sizes(lib):
    f = lib.dflash_shared_prefix_workspace
    assert f(1, 32, 8, 128, 32, 512) > 0
    assert f(1, 32, 8, 128, 32, 513) >= f(1, 32, 8, 128, 32, 512)
    # what a larger call needs is enough for a smaller one
    for dtype in (0, 1):
        for h, hkv, hd in ((4, 2, 64), (32, 8, 128), (7, 7, 64), (64, 1, 128), (24, 8, 64)):
            grid = [[f(dtype, h, hkv, hd, b, r) for r in (1, 2, 7, 8, 9, 31, 33, 64, 257, 2048, 4096)] for b in (1, 2, 8, 33, 64, 1024)]
            assert all(x > 0 for row in grid for x in row)
            assert all(row == sorted(row) for row in grid)
            assert all(list(col) == sorted(col) for col in zip(*grid))


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(batch=0), dict(batch=2049), dict(rows_per_seq=0), dict(rows_per_seq=33), dict(vocab=0),
    dict(logits=None), dict(out=None), dict(logits=P + 2), dict(ld_logits=999), dict(ld_out=999), dict(ld_out=1004),
    dict(hist_lens=None), dict(prompt_lens=None), dict(ld_hist=7), dict(history=None), dict(bias_values=None),
    dict(mask_index=None), dict(ld_mask=31), dict(hist_width=(1 << 29) + 1, ld_hist=1 << 30), dict(bias_width=(1 << 29) + 1)])
def test_process_logits_refuses(lib, kw):
    assert lib.dflash_process_logits(ctypes.byref(rules(**kw)), None) == dfl.DFLASH_E_INVAL
    assert "process_logits" in dfl.dflash_last_error(None)


def test_null_args(lib):
    assert lib.dflash_kv_tables(None, None) == dfl.DFLASH_E_INVAL
    assert lib.dflash_shared_prefix_attention(None, None) == dfl.DFLASH_E_INVAL
    assert lib.dflash_process_logits(None, None) == dfl.DFLASH_E_INVAL


def test_the_bindings_refuse_cpu_tensors():
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dfl.kv_tables(i, i, i[:, None], rows=4)
    with pytest.raises(ValueError, match="CUDA"):
        dfl.process_logits(torch.zeros(2, 8))
    c = torch.zeros(1, 1, 64, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dfl.shared_prefix_attention(torch.zeros(1, 1, 64), c, c, None, 0, i[:1, None], i[:1], i)


def test_the_checks_in_python_and_in_the_extension_agree(lib):
    """The same addresses and strides, and refusals of the same tensors, wherever both forms are there."""
    import torch
    if ops._flat is ops._PYTHON_CHECKS[0]:
        ops._use_extension()
    if ops._flat is ops._PYTHON_CHECKS[0]:
        pytest.skip("the extension has not been built")
    i, x = torch.arange(24, dtype=torch.int32), torch.zeros(4, 6, 8)
    m = i.view(4, 6)
    calls = [(0, ("a", t, d, n, dev)) for t in (i, m, i[::2], i[:0], i[3:4], m[:, :2], m.t()) for d in (torch.int32, torch.int64)
             for n in (t.numel(), 24) for dev in (-1, 0)]
    calls += [(1, ("a", t, torch.int32, r, c, -1)) for t in (m, m[:, 1:4], m[::2], m.t(), m[:1, :3], m[:0], m[:, :0], m[:, ::2], i,
                                                             m[:1].expand(4, 6)) for r in (4, 2, 6, 1, 0) for c in (None, 6, 3)]
    calls += [(2, ("a", t, torch.float32, *s, -1)) for t in (x, x[::2], x[:, :3], x[:, :, :4], x.transpose(0, 1), x[:1], x[:, :1], x[:0], x[:, :, :0], m)
              for s in ((0, 6, 8), (4, 6, 0), (4, 6, 8), (2, 6, 8), (4, 3, 8), (4, 6, 4), (6, 4, 8), (1, 6, 8), (4, 1, 8))]
    refused = 0
    for which, a in calls:
        got = []
        for f in (ops._PYTHON_CHECKS[which], (ops._flat, ops._mat, ops._rows3)[which]):
            try:
                got.append(f(*a))
            except ValueError as e:
                got.append(ValueError)
                assert str(e).startswith("a")
        assert got[0] == got[1], (which, a, got)
        refused += got[0] is ValueError
    assert 0 < refused < len(calls)


def test_calls_on_a_kept_workspace_queue_one_at_a_time(monkeypatch):
    """A call queues two kernels with the workspace between them: two host threads on the default stream must not be
    inside the C call with the same workspace at once.  (The C call is a stand-in: no GPU.)"""
    import threading
    import time

    import torch
    inside, lock, overlaps, calls = {}, threading.Lock(), [], []

    def call(fn, pack, values, dev):
        ws, size = values[-2:]
        with lock:
            overlaps.append(inside.get(ws, 0))
            inside[ws] = inside.get(ws, 0) + 1
            calls.append((ws, size))
        time.sleep(0.002)  # (gives up the interpreter's lock, as the foreign call does)
        with lock:
            inside[ws] -= 1

    monkeypatch.setattr(ops, "_call", call)
    monkeypatch.setattr(ops, "_device", lambda *a: 0)
    monkeypatch.setattr(ops, "_flat", lambda name, t, *a: t.data_ptr())
    monkeypatch.setattr(ops, "_mat", lambda *a: 4)
    monkeypatch.setattr(ops, "_rows3", lambda *a: 256)
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(ops, "_KEPT", {})
    c = torch.zeros(2, 2, 64, 64)

    def work(rows):
        i = torch.zeros(rows + 1, dtype=torch.int32)
        for _ in range(20):
            ops.shared_prefix_attention(torch.zeros(rows, 4, 64), c, c, None, 0, i[:rows, None], i[:rows], i)

    threads = [threading.Thread(target=work, args=(r,)) for r in (1, 3, 40)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(calls) == 60 and not any(overlaps)
    assert len({n for _, n in calls}) == 3


def test_session_masks_refuse_other_index_types():
    """A mask index of another type or with gaps would be read as other numbers."""
    import torch
    from types import SimpleNamespace
    calls = []
    sess = dfl.Session.__new__(dfl.Session)
    sess.w, sess.ctx = SimpleNamespace(vocab=70), None
    sess.lib = SimpleNamespace(dflash_set_token_masks=lambda ctx, n, masks, rows, index: calls.append((n, rows)) or 0)
    masks = torch.zeros(2, 3, dtype=torch.int32)
    index = torch.zeros(8, dtype=torch.int32)
    for bad in (index.long(), index.float(), index[::2]):
        with pytest.raises(ValueError, match="mask_index"):
            sess.set_token_masks(masks, bad)
    for bad in (masks.long(), masks[:, :2], masks.t().contiguous().t(), masks[0]):
        with pytest.raises(ValueError, match="masks"):
            sess.set_token_masks(bad, index)
    assert not calls
    sess.set_token_masks(masks, index)
    sess.set_token_masks(masks.numpy(), [0, 1, -1])
    assert calls == [(2, 8), (2, 3)]


def test_no_workspace_is_kept_beyond_its_limit(monkeypatch):
    """A large call on the default stream allocates for itself; what is kept stays within the limit.  (No GPU: the foreign
    call is a stand-in.)"""
    import torch
    calls = []
    monkeypatch.setattr(ops, "_call", lambda fn, pack, values, dev: calls.append(values[-2:]))
    monkeypatch.setattr(ops, "_device", lambda *a: 0)
    monkeypatch.setattr(ops, "_flat", lambda name, t, *a: t.data_ptr())
    monkeypatch.setattr(ops, "_mat", lambda *a: 4)
    monkeypatch.setattr(ops, "_rows3", lambda *a: 256)
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(ops, "_KEPT", {})
    c = torch.zeros(2, 2, 64, 64)
    for rows in (1, 150000, 8, 150000, 1):
        i = torch.zeros(2, dtype=torch.int32)
        ops.shared_prefix_attention(torch.zeros(rows, 4, 64), c, c, None, 0, i[:1, None], i[:1], i)
    assert [n > ops.KEPT_MAX for _, n in calls] == [False, True, False, True, False]
    assert calls[2][0] == calls[4][0] == ops._KEPT[0][1] and ops._KEPT[0][0] == calls[2][1] <= ops.KEPT_MAX


def test_versions_of_written_tensors_rise(lib):
    """In either form of the binding's helper, views of a tensor included; inference tensors have no version."""
    import torch
    forms = [ops._PYTHON_WRITTEN]
    if ops._written is ops._PYTHON_WRITTEN:
        ops._use_extension()
    if ops._written is not ops._PYTHON_WRITTEN:
        forms.append(ops._written)
    for f in forms:
        t, i = torch.zeros(4, 4), torch.zeros(3, dtype=torch.int32)
        f(t, None, i)
        assert t._version == 1 and i._version == 1
        f(t[1:])
        assert t._version == 2
        with torch.inference_mode():
            z = torch.zeros(2)
        f(z)


def test_gradients_are_refused_in_both_modes():
    import torch
    from torch.autograd import forward_ad
    from types import SimpleNamespace
    first = SimpleNamespace(get_device=lambda: 0)
    x = torch.zeros(3)
    assert ops._device(first, x, None) == 0
    with pytest.raises(ValueError, match="gradient"):
        ops._device(first, x, x.clone().requires_grad_())
    with torch.no_grad():
        ops._device(first, x.clone().requires_grad_())
    with forward_ad.dual_level():
        ops._device(first, x, None)
        dual = forward_ad.make_dual(x.clone(), torch.ones(3))
        with pytest.raises(ValueError, match="tangent"):
            ops._device(first, x, dual)
        with torch.no_grad():
            with pytest.raises(ValueError, match="tangent"):
                ops._device(first, dual)


@pytest.mark.parametrize("flags", [2, 3, -1, 1 << 30])
def test_unknown_attention_flags_are_refused(lib, flags):
    assert lib.dflash_shared_prefix_attention(ctypes.byref(attn(reserved=flags)), None) == dfl.DFLASH_E_INVAL
    assert "flags" in dfl.dflash_last_error(None)
