"""Pins of the serving operators' oracles outside themselves: hand-made tables, attention against one
softmax over the concatenated keys (torch), logit rules in closed form."""
import numpy as np
import torch

from oracle import serving


def test_kv_tables_by_hand():
    # request 0: 63 cached + 2 new -> one page held, one taken; request 1: empty, nothing new;
    # request 2: 64 cached (a full page) + 65 new -> two taken
    table = np.array([[5, 99, 99], [99, 99, 99], [7, 99, 99]])
    free = np.array([40, 41, 42, 43, 44])
    t, used, q, seq, pos, slots, status = serving.kv_tables([63, 0, 64], [2, 0, 65], table, free, 1, 70, scratch_page=9,
                                                            base_pos=100)
    assert status == 0 and used == 4
    assert t.tolist() == [[5, 41, 9], [9, 9, 9], [7, 42, 43]]
    assert q.tolist() == [0, 2, 2, 67]
    assert seq[:3].tolist() == [0, 0, 2] and seq[66] == 2 and seq[67:].tolist() == [-1, -1, -1]
    assert pos[:3].tolist() == [163, 164, 164]
    assert slots[:3].tolist() == [5 * 64 + 63, 41 * 64, 42 * 64] and slots[66] == 43 * 64


def test_kv_tables_statuses():
    table = np.zeros((1, 2), np.int64)
    free = np.array([1, 2])
    assert serving.kv_tables([0], [129], table, free, 0, 200)[-1] == 3   # three pages: too wide, too many
    assert serving.kv_tables([0], [128], table, free, 1, 200)[-1] == 1
    assert serving.kv_tables([0], [128], table, free, 0, 127)[-1] == 4
    assert serving.kv_tables([-1], [1], table, free, 0, 9)[-1] == 8


def test_attention_is_one_softmax_over_prefix_and_own_keys():
    rng = np.random.default_rng(0)
    hkv, H, hd, pre = 2, 4, 64, 70
    k, v = rng.standard_normal((2, 6, hkv, 64, hd))
    q = rng.standard_normal((5, H, hd))
    out, lse, _ = serving.shared_prefix_attention(q, k, v, [3, 1], pre, np.array([[0, 5], [2, 4]]), [66, 2], [0, 3, 5], True,
                                                  0.125)
    K = np.concatenate([k[3], k[1][:, :6], k[0], k[5][:, :2]], 1)
    V = np.concatenate([v[3], v[1][:, :6], v[0], v[5][:, :2]], 1)
    for j in range(3):   # row j of three sees 70 + 64 + j keys
        z = torch.from_numpy(0.125 * np.einsum("hd,hkd->hk", q[j], K[[0, 0, 1, 1]]))[:, :70 + 64 + j]
        want = torch.einsum("hk,hkd->hd", torch.softmax(z, -1), torch.from_numpy(V[[0, 0, 1, 1]])[:, :70 + 64 + j])
        assert np.abs(out[j] - want.numpy()).max() < 1e-12
        assert np.abs(lse[j] - torch.logsumexp(z, -1).numpy()).max() < 1e-12


def test_attention_rows_without_keys():
    z = np.zeros((1, 1, 64, 64))
    out, lse, _ = serving.shared_prefix_attention(np.ones((2, 1, 64)), z, z, [], 0, np.zeros((1, 1), int), [1], [0, 2], True,
                                                  1.0)
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf   # row 0 of 2 comes before the only key
    assert lse[1, 0] == 0.0


def test_logit_rules_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 4.0, 0.5]] * 2)
    kw = dict(history=np.array([[0, 1, 3, 3, -1]]), hist_lens=[5], prompt_lens=[2], drafts=np.array([[4]]),
              repetition=[2.0], presence=[0.25], frequency=[0.5], bias_ids=np.array([[2, 2, -1]]),
              bias_values=np.array([[5.0, 7.0, 9.0]]), masks=np.array([[0b01110]], np.int32), mask_index=[-1, 0])
    y = serving.process_logits(x, 2, **kw)
    # prompt {0, 1}: repetition only; 3 twice: 4/2 - 2*0.5 - 0.25; 2: the last bias; 4 untouched in row 0
    assert y[0].tolist() == [1.0, -4.0, 8.0, 0.75, 0.5]
    # row 1 also follows the draft 4 (0.5/2 - 0.5 - 0.25), then its mask allows 1, 2, 3
    assert y[1].tolist() == [-np.inf, -4.0, 8.0, 0.75, -np.inf]
    kw["masks"] = np.array([[0]], np.int32)
    assert (serving.process_logits(x, 2, **kw)[1] == -np.inf).all()
