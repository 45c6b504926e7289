"""Refusals of the operators of trees, shared pages and log probabilities, host side (no GPU); their argument structs have the
header's layout; and their oracles agree with simpler statements of the same things."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import block_diffusion_speculative_ctx_gb300 as dfl
from block_diffusion_speculative_ctx_gb300 import build as dbuild
from oracle import serving, trees

torch = pytest.importorskip("torch")
ops = pytest.importorskip("block_diffusion_speculative_ctx_gb300.ops")
ot = pytest.importorskip("block_diffusion_speculative_ctx_gb300.ops_tree")
ol = pytest.importorskip("block_diffusion_speculative_ctx_gb300.ops_logprobs")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096  # stands for a device pointer (never read: every call here is refused)


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return dfl.load()


def test_struct_layouts_match_the_header(tmp_path):
    structs = (ot.dflash_tree_masks_args, ot.dflash_tree_attention_args, ot.dflash_tree_accept_args, ot.dflash_kv_compact_args,
               ot.dflash_kv_fork_args, ot.dflash_kv_release_args, ol.dflash_logprobs_args, ol.dflash_logprobs_grad_args)
    names = [f"sizeof({s.__name__})" for s in structs]
    names += [f"offsetof({s.__name__}, {f[0]})" for s in structs for f in s._fields_]
    prog, exe = tmp_path / "sz.c", tmp_path / "sz"
    prog.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"dflash.h\"\nint main(void) {\n"
                    + "".join(f'  printf("%zu\\n", (size_t){n});\n' for n in names) + "  return 0;\n}\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(s) for s in structs] + [getattr(s, f[0]).offset for s in structs for f in s._fields_]
    packs = (ot._MASKS, ot._TREE, ot._ACCEPT, ot._COMPACT, ot._FORK, ot._RELEASE, ol._LOGPROBS, ol._GRAD)
    assert [p.size for p in packs] == got[:len(structs)]


def masks(**kw):
    return ot.dflash_tree_masks_args(**dict(dict(batch=2, rows=8, words=1, base_pos=0, ld_mask=1, parents=P, q_start=P, kv_lens=P, masks=P,
                                                 depth=P, row_pos=P, status=P), **kw))


def attention(attn=None, **kw):
    a = dict(dtype=1, n_heads=8, n_kv_heads=2, head_dim=128, batch=2, rows=4, n_pages=16, prefix_len=100, width=2, causal=1,
             scale=0.1, reserved=0, ld_q=1024, ld_out=1024, ld_table=2, q=P, k_cache=P, v_cache=P, prefix_pages=P, table=P,
             kv_lens=P, q_start=P, out=P, lse=P, workspace=P, workspace_bytes=1 << 40)
    return ot.dflash_tree_attention_args(**dict(dict(attn=ops.dflash_shared_prefix_args(**dict(a, **(attn or {}))), masks=P, ld_mask=2, words=2,
                                                     reserved=0), **kw))


def accept(**kw):
    return ot.dflash_tree_accept_args(**dict(dict(batch=2, rows=8, width=4, reserved=0, parents=P, tokens=P, posterior=P, q_start=P, path=P,
                                                  accepted=P, bonus=P, status=P), **kw))


def compact(**kw):
    return ot.dflash_kv_compact_args(**dict(dict(dtype=1, batch=2, layers=3, n_pages=9, n_kv_heads=2, head_dim=64, width=4, width_table=2,
                                                 ld_layer=9 * 2 * 64 * 64, ld_table=2, k_cache=P, v_cache=P, table=P, kv_lens=P, q_start=P,
                                                 path=P, accepted=P, kv_out=2 * P, status=P), **kw))


def fork(**kw):
    return ot.dflash_kv_fork_args(**dict(dict(dtype=1, batch=2, children=3, width=2, n_free=4, scratch_page=0, layers=3, n_pages=9, n_kv_heads=2,
                                              head_dim=64, ld_layer=9 * 2 * 64 * 64, ld_table=2, ld_out=2, k_cache=P, v_cache=P, parents=P,
                                              kv_lens=P, table=P, free_pages=P, used=P, refs=P, table_out=2 * P, lens_out=2 * P, used_out=P,
                                              status=P), **kw))


def release(**kw):
    return ot.dflash_kv_release_args(**dict(dict(batch=2, n=2, width=2, n_free=4, n_pages=9, reserved=0, ld_table=2, seqs=P, kv_lens=P, table=P,
                                                 free_pages=P, used=P, refs=P, used_out=P, status=P), **kw))


def logprobs(**kw):
    return ol.dflash_logprobs_args(**dict(dict(dtype=0, rows=4, vocab=100, n=2, k=5, inv_temperature=1.0, ld_logits=100, logits=P, tokens=P,
                                               logprobs=P, ranks=P, entropy=P, lse=P, top_ids=P, top_logprobs=P), **kw))


def grad(**kw):
    return ol.dflash_logprobs_grad_args(**dict(dict(dtype=0, rows=4, vocab=100, n=2, inv_temperature=1.0, reserved=0, ld_logits=100, ld_out=100,
                                                    logits=P, tokens=P, lse=P, grad_logprobs=P, entropy=P, grad_entropy=P, out=2 * P), **kw))


CACHES = [dict(dtype=2), dict(layers=0), dict(layers=1025), dict(n_pages=0), dict(n_pages=(1 << 24) + 1), dict(n_kv_heads=0), dict(head_dim=0),
          dict(head_dim=4), dict(head_dim=100), dict(k_cache=None), dict(v_cache=P + 8), dict(ld_layer=100), dict(ld_layer=9 * 2 * 64 * 64 + 4)]
REFUSED = {
    "tree_masks": (masks, [dict(batch=0), dict(batch=2049), dict(rows=-1), dict(rows=(1 << 20) + 1), dict(words=0), dict(words=(1 << 20) + 1, ld_mask=1 << 21),
                           dict(ld_mask=0), dict(base_pos=-1), dict(parents=None), dict(q_start=None), dict(kv_lens=None), dict(masks=None),
                           dict(status=None)]),
    "tree_attention": (attention, [dict(attn=x) for x in (dict(dtype=2), dict(head_dim=96), dict(batch=0), dict(q=None), dict(workspace_bytes=0),
                                                          dict(scale=0.0), dict(ld_table=1), dict(reserved=2))]
                       + [dict(masks=None), dict(words=0), dict(words=(1 << 20) + 1, ld_mask=1 << 21), dict(ld_mask=1), dict(reserved=1)]),
    "tree_accept": (accept, [dict(batch=0), dict(batch=2049), dict(rows=-1), dict(rows=(1 << 20) + 1), dict(width=0), dict(width=1025),
                             dict(reserved=1)] + [{n: None} for n in ("parents", "tokens", "posterior", "q_start", "path", "accepted", "bonus", "status")]),
    "kv_compact": (compact, CACHES + [dict(batch=0), dict(batch=2049), dict(width=0), dict(width=1025), dict(width_table=-1), dict(ld_table=1),
                                      dict(kv_out=P)] + [{n: None} for n in ("table", "kv_lens", "q_start", "path", "accepted", "kv_out", "status")]),
    "kv_fork": (fork, CACHES + [dict(batch=0), dict(batch=2049), dict(children=0), dict(children=2049), dict(width=0), dict(ld_table=1), dict(ld_out=1),
                                dict(n_free=-1), dict(table_out=P), dict(lens_out=P)]
                + [{n: None} for n in ("parents", "kv_lens", "table", "free_pages", "used", "refs", "table_out", "lens_out", "used_out", "status")]),
    "kv_release": (release, [dict(batch=0), dict(batch=2049), dict(n=0), dict(n=2049), dict(width=0), dict(width=(1 << 18) + 1, ld_table=1 << 19),
                             dict(ld_table=1), dict(n_free=-1), dict(n_pages=0), dict(reserved=1)]
                   + [{n: None} for n in ("seqs", "kv_lens", "table", "free_pages", "used", "refs", "used_out", "status")]),
    "token_logprobs": (logprobs, [dict(dtype=2), dict(rows=-1), dict(rows=(1 << 20) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1, ld_logits=1 << 31),
                                  dict(n=-1), dict(n=33), dict(k=-1), dict(k=33), dict(inv_temperature=0.0), dict(inv_temperature=-1.0),
                                  dict(inv_temperature=float("nan")), dict(inv_temperature=float("inf")), dict(inv_temperature=2.0 ** 20 * 1.001),
                                  dict(inv_temperature=2.0 ** -20 * 0.999), dict(logits=None), dict(tokens=None),
                                  dict(logits=P + 2), dict(ld_logits=99)]),
    "token_logprobs_grad": (grad, [dict(dtype=2), dict(rows=-1), dict(rows=(1 << 20) + 1), dict(vocab=0), dict(n=33), dict(inv_temperature=0.0),
                                   dict(inv_temperature=2.0 ** 21), dict(reserved=1), dict(logits=None), dict(out=None), dict(lse=None), dict(tokens=None), dict(grad_logprobs=None),
                                   dict(entropy=None), dict(logits=P + 1), dict(out=P + 2), dict(ld_logits=99), dict(ld_out=99),
                                   dict(out=P, ld_out=101), dict(rows=1 << 20, vocab=1 << 25, ld_logits=1 << 25, ld_out=1 << 25)]),
}


@pytest.mark.parametrize("name,i", [(n, i) for n, (_, cases) in REFUSED.items() for i in range(len(cases))])
def test_bad_arguments_are_refused(lib, name, i):
    make, cases = REFUSED[name]
    assert getattr(lib, "dflash_" + name)(ctypes.byref(make(**cases[i])), None) == dfl.DFLASH_E_INVAL, cases[i]
    assert dfl.dflash_last_error(None).startswith(name + ":")


@pytest.mark.parametrize("name", REFUSED)
def test_null_args(lib, name):
    assert getattr(lib, "dflash_" + name)(None, None) == dfl.DFLASH_E_INVAL
    assert dfl.dflash_last_error(None) == name + ": args is NULL"


def test_calls_without_rows_queue_nothing(lib):
    assert lib.dflash_token_logprobs(ctypes.byref(logprobs(rows=0, logits=None, tokens=None)), None) == dfl.DFLASH_OK
    assert lib.dflash_token_logprobs_grad(ctypes.byref(grad(rows=0)), None) == dfl.DFLASH_OK
    assert lib.dflash_tree_attention(ctypes.byref(attention(attn=dict(rows=0))), None) == dfl.DFLASH_OK


def test_the_bindings_refuse_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    c, x = torch.zeros(1, 1, 64, 64), torch.zeros(2, 8)
    calls = [lambda: dfl.tree_masks(i, i), lambda: dfl.tree_accept(i, i, i, i, width=2),
             lambda: dfl.tree_attention(torch.zeros(1, 1, 64), c, c, i[:1, None], i[:1], i, i[:1, None]),
             lambda: dfl.kv_compact(c, c, i[:, None], i, i, i[:, None], i), lambda: dfl.kv_fork(i, i, i[:, None], i, i[:1], i[:1], c, c),
             lambda: dfl.kv_release(i, i, i[:, None], i, i[:1], i), lambda: dfl.token_logprobs(x, i),
             lambda: dfl.token_logprobs_grad(x, i, x[:, 0], x[:, 0])]
    for f in calls:
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_the_grouped_checks_in_python_and_in_the_extension_agree(lib):
    """Addresses, layouts and refusals of the same tensors, wherever both forms are there."""
    if ops._ints is ops._PYTHON_GROUPS[0]:
        ops._use_extension()
    if ops._ints is ops._PYTHON_GROUPS[0]:
        pytest.skip("the extension has not been built")
    i, x = torch.arange(24, dtype=torch.int32), torch.zeros(3, 4, 2, 64, 8)
    calls = [(0, (d, "a", t, n, "b", i, 24)) for t in (i, i[:0], i[::2], i[3:4], i.view(4, 6).t(), i.long()) for n in (t.numel(), 24) for d in (-1, 0)]
    calls += [(0, (-1,)), (0, (-1, "a", i[:5], 5)), (0, (-1, "a", i, 24, "b", i[1:], 24))]
    wide = torch.zeros(3, 9, 2, 64, 8)
    views = [x, x[0], x[:1], x[:0], x[1:], x[:, :2], wide[:, :4], wide[:, 2:6], x[:, :, :1], x[..., :4], x.bfloat16(), x.half(), x.transpose(0, 1),
             x[:, :, :, :32], x[0, 0], x.expand(3, 4, 2, 64, 8)[:, :1]]
    calls += [(1, (k, v, d)) for k in views for v in views for d in (-1, 0)]
    calls += [(2, (d, "a", t, dt, n, "b", x, torch.float32, x.numel())) for t in (i, i[::2], x, x[:, :1], x.bfloat16())
              for dt in (torch.int32, torch.float32) for n in (t.numel(), 7) for d in (-1, 0)]
    leaf = torch.zeros(3, requires_grad=True)
    calls += [(3, a) for a in ((), (None, x), (x, leaf, None), (leaf.detach(),), (leaf,))]
    refused = 0
    for which, a in calls:
        got = []
        for f in (ops._PYTHON_GROUPS[which], (ops._ints, ops._caches, ops._flats, ops._free_of_grad)[which]):
            try:
                got.append(f(*a))
            except ValueError:
                got.append(ValueError)
        assert got[0] == got[1] and type(got[0]) is type(got[1]), (which, [y.shape if hasattr(y, "shape") else y for y in a])
        refused += got[0] is ValueError
    assert 0 < refused < len(calls)


# ---------------------------------------------------------------------------------------------- the oracles' pins
def test_oracle_chain_is_the_causal_attention():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 5, 2, 64, 8))
    q, table, kv, start = rng.standard_normal((7, 4, 8)), np.array([[1, 3], [4, 0]]), np.array([70, 4]), np.array([0, 3, 7])
    sees = [np.tril(np.ones((m, m), bool)) for m in (3, 4)]
    a = trees.tree_attention(q, k, v, np.array([2]), 10, table, kv, start, sees, 0.3)
    b = serving.shared_prefix_attention(q, k, v, np.array([2]), 10, table, kv, start, True, 0.3)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, rtol=1e-12, atol=1e-12)


def test_oracle_tree_words_and_acceptance():
    sees, depth = trees.ancestors([-1, 0, 0, 1, 3, -1])
    assert depth.tolist() == [0, 1, 1, 2, 3, 0]
    assert trees.words(sees, 1)[:, 0].tolist() == [1, 3, 5, 11, 27, 32]
    assert trees.words(np.eye(40, dtype=bool), 2)[31].tolist() == [-(2 ** 31), 0]
    assert trees.tree_accept([-1, 0, 0, 2, 2], [9, 5, 6, 7, 7], [6, 0, 7, 8, 1], 5) == ([0, 2, 3, -1, -1], 2, 8)
    assert trees.tree_accept([-1, 0, 0, 2, 2], [9, 5, 6, 7, 7], [6, 0, 7, 8, 1], 2) == ([0, 2], 1, 7)


def test_oracle_of_a_chain_accepts_what_the_block_rule_accepts():
    """A chain's acceptance is the round's: the longest prefix of drafts that the target agrees with."""
    rng = np.random.default_rng(1)
    for _ in range(50):
        m = int(rng.integers(1, 9))
        draft, post = rng.integers(0, 2, m), rng.integers(0, 2, m)
        want = 0
        while want < m - 1 and draft[want + 1] == post[want]:
            want += 1
        path, accepted, bonus = trees.tree_accept(np.arange(-1, m - 1), draft, post, m)
        assert accepted == want and bonus == post[want] and path[:want + 1] == list(range(want + 1))


def test_oracle_fork_and_release_restore_the_pool():
    table, kv = np.array([[5, 6, 9], [7, 9, 9]]), [100, 64]
    cache = np.arange(10 * 64, dtype=float).reshape(1, 10, 1, 64, 1)
    free = np.array([8, 4, 3, 2])
    t, lens, used, refs, (c,) = trees.kv_fork([0, 1, 0], kv, table, free, 1, np.zeros(10, int), [cache], 9)
    assert t.tolist() == [[5, 4, 9], [7, 9, 9], [5, 3, 9]] and lens == [100, 64, 100] and used == 3 and refs[[5, 7]].tolist() == [2, 1]
    assert (c[0, 4, 0, :36] == cache[0, 6, 0, :36]).all() and (c[0, 4, 0, 36:] == cache[0, 4, 0, 36:]).all()
    f, used, refs, status = trees.kv_release([0, 1, 2], lens, t, free, used, refs)
    assert f.tolist() == free.tolist() and used == 1 and not refs.any() and status == 0
    assert trees.kv_release([0, 0], kv, table, free, 3, refs)[3] == 32


def test_oracle_log_probabilities_and_their_gradient():
    x = np.random.default_rng(2).standard_normal((2, 30))
    x[1, 7] = -np.inf
    t, g, h = np.array([[3, -1], [7, 29]]), np.array([[0.5, 9.0], [0.0, -1.0]]), np.array([0.25, -0.5])
    lp, ranks, entropy, lse, ids, top = trees.token_logprobs(x, t, 3, 0.8)
    y = torch.tensor(x, requires_grad=True)
    logp = torch.log_softmax(y / 0.8, 1)
    np.testing.assert_allclose(lp[0, 0], logp[0, 3].item(), rtol=1e-12)
    assert np.isneginf(lp[1, 0]) and ranks[1, 0] == 29 and lp[0, 1] == 0 and ranks[0, 1] == -1
    np.testing.assert_allclose(lse, torch.logsumexp(y / 0.8, 1).detach().numpy(), rtol=1e-12)
    ent = torch.special.entr(logp.exp()).sum(1)
    np.testing.assert_allclose(entropy, ent.detach().numpy(), rtol=1e-12)
    np.testing.assert_array_equal(ids, torch.topk(y, 3)[1].numpy())
    np.testing.assert_allclose(top, torch.topk(logp, 3)[0].detach().numpy(), rtol=1e-12)
    fine = torch.where(torch.isinf(y), -80.0, y).detach().requires_grad_()  # (entr's own derivative at 0 is infinite)
    logp = torch.log_softmax(fine / 0.8, 1)
    (0.5 * logp[0, 3] - logp[1, 29] - (torch.tensor(h) * (logp.exp() * logp).sum(1)).sum()).backward()
    np.testing.assert_allclose(trees.token_logprobs_grad(x, t, g, h, 0.8), fine.grad.numpy(), rtol=1e-9, atol=1e-12)


def test_compact_refuses_one_cache_for_both(lib):
    assert lib.dflash_kv_compact(ctypes.byref(compact()), None) == dfl.DFLASH_E_INVAL
    assert dfl.dflash_last_error(None) == "kv_compact: v_cache may not be k_cache"


@pytest.mark.parametrize("name,make", [("token_logprobs", logprobs), ("token_logprobs_grad", grad)])
def test_parts_of_lse_are_aligned(lib, name, make):
    assert getattr(lib, "dflash_" + name)(ctypes.byref(make(lse_parts=P + 4)), None) == dfl.DFLASH_E_INVAL
    assert dfl.dflash_last_error(None) == name + ": lse_parts is not aligned to 8 bytes"


def test_oracle_release_behind_a_cut():
    table, free, refs = np.array([[4, 1, 2], [3, 5, 0]]), np.arange(6), np.zeros(6, int)
    f, used, refs, status = trees.kv_release([1, 0], [130, 70], table, free, 5, refs, keep=[65, 64])
    assert (status, used) == (0, 3) and f[3:5].tolist() == [5, 2]


LAYER = 9 * 2 * 64 * 64 * 2  # bytes of a layer of compact()'s and fork()'s caches


@pytest.mark.parametrize("name,make", [("kv_compact", compact), ("kv_fork", fork)])
@pytest.mark.parametrize("between,apart", [(LAYER, 16), (LAYER, LAYER - 16), (LAYER, -16), (LAYER, LAYER), (LAYER, 3 * LAYER - 16),
                                           (2 * LAYER, LAYER - 16), (2 * LAYER, 4 * LAYER), (2 * LAYER, -LAYER - 16), (3 * LAYER, 2 * LAYER + 16),
                                           (3 * LAYER, -6 * LAYER + 16)])
def test_caches_that_overlap_are_refused(lib, name, make, between, apart):
    a = make(k_cache=1 << 40, v_cache=(1 << 40) + apart, ld_layer=between // 2)
    assert getattr(lib, "dflash_" + name)(ctypes.byref(a), None) == dfl.DFLASH_E_INVAL
    assert dfl.dflash_last_error(None) == name + ": k_cache and v_cache overlap"


@pytest.mark.parametrize("name,make", [("kv_compact", compact), ("kv_fork", fork)])
@pytest.mark.parametrize("between,apart", [(LAYER, 3 * LAYER), (LAYER, -3 * LAYER), (2 * LAYER, LAYER), (2 * LAYER, -LAYER), (2 * LAYER, 3 * LAYER),
                                           (2 * LAYER, 5 * LAYER), (2 * LAYER, 5 * LAYER + 16), (3 * LAYER, LAYER + 16), (3 * LAYER, -4 * LAYER),
                                           (3 * LAYER, -2 * LAYER), (3 * LAYER, 2 * LAYER)])
def test_caches_beside_each_other_are_not(lib, name, make, between, apart):
    """(The call is refused for its NULL status, which is looked at behind the caches.)"""
    a = make(k_cache=1 << 40, v_cache=(1 << 40) + apart, ld_layer=between // 2, status=None)
    assert getattr(lib, "dflash_" + name)(ctypes.byref(a), None) == dfl.DFLASH_E_INVAL
    assert dfl.dflash_last_error(None) == name + ": NULL argument"
