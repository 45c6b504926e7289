"""Oracles of the serving operators, in plain numpy loops: page tables from request lengths,
attention over a shared prefix and a sequence's own keys (fp64), and the logit rules (fp64)."""
from __future__ import annotations

import numpy as np

PAGE = 64


def kv_tables(kv_lens, new_lens, table, free_pages, used, rows, scratch_page=0, base_pos=0):
    """(table, used, q_start, row_seq, row_pos, slots, status); free_pages None: the table backs every token."""
    batch, width = table.shape
    out = table.copy()
    q_start = np.zeros(batch + 1, np.int64)
    row_seq, row_pos = np.full(rows, -1, np.int64), np.full(rows, -1, np.int64)
    slots = np.full(rows, -1, np.int64)
    status = 0
    if any(x < 0 for x in kv_lens) or any(x < 0 for x in new_lens) or (free_pages is not None and used < 0):
        status |= 8
    need = [-(-(int(c) + int(m)) // PAGE) if c >= 0 and m >= 0 else 0 for c, m in zip(kv_lens, new_lens)]
    old = [-(-int(c) // PAGE) if c >= 0 and m >= 0 else 0 for c, m in zip(kv_lens, new_lens)]
    if any(n > width for n in need):
        status |= 2
    if free_pages is not None and max(used, 0) + sum(need) - sum(old) > len(free_pages):
        status |= 1
    if sum(max(int(m), 0) for c, m in zip(kv_lens, new_lens) if c >= 0) > rows:
        status |= 4
    if status:
        return None, used, q_start, row_seq, row_pos, slots, status
    at = used
    for s in range(batch):
        if free_pages is not None:
            for j in range(old[s], need[s]):
                out[s, j] = free_pages[at]
                at += 1
        out[s, need[s]:] = scratch_page
        q_start[s + 1] = q_start[s] + new_lens[s]
        for j in range(int(new_lens[s])):
            r, i = int(q_start[s]) + j, int(kv_lens[s]) + j
            row_seq[r], row_pos[r] = s, base_pos + i
            slots[r] = int(out[s, i // PAGE]) * PAGE + i % PAGE
    return out, at, q_start, row_seq, row_pos, slots, status


def shared_prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len, table, kv_lens, q_start, causal, scale):
    """(out, lse, weight): float64 arrays [rows, H, hd], [rows, H] and sum_i p_i |v_i| [rows, H, hd] (what a
    relative error of the softmax weights is multiplied by); rows of no sequence stay NaN."""
    rows, H, hd = q.shape
    hkv = k_cache.shape[1]
    g = H // hkv
    out = np.full((rows, H, hd), np.nan)
    lse = np.full((rows, H), np.nan)
    weight = np.full((rows, H, hd), np.nan)

    def keys(cache, pages, n):
        x = cache[np.asarray(pages[: -(-n // PAGE)], np.int64)]          # [p, hkv, 64, hd]
        return x.transpose(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :n]

    for s in range(len(kv_lens)):
        a, b = int(q_start[s]), int(q_start[s + 1])
        n = int(kv_lens[s])
        if a == b:
            continue
        K = np.concatenate([keys(k_cache, prefix_pages, prefix_len), keys(k_cache, table[s], n)], 1).astype(np.float64)
        V = np.concatenate([keys(v_cache, prefix_pages, prefix_len), keys(v_cache, table[s], n)], 1).astype(np.float64)
        for r in range(a, b):
            last = prefix_len + (max(0, n - (b - a) + (r - a) + 1) if causal else n)
            for h in range(H):
                if last == 0:
                    out[r, h], lse[r, h], weight[r, h] = 0.0, -np.inf, 0.0
                    continue
                z = scale * (K[h // g, :last] @ q[r, h].astype(np.float64))
                m = z.max()
                p = np.exp(z - m)
                out[r, h] = p @ V[h // g, :last] / p.sum()
                weight[r, h] = p @ np.abs(V[h // g, :last]) / p.sum()
                lse[r, h] = m + np.log(p.sum())
    return out, lse, weight


def process_logits(logits, rows_per_seq=1, history=None, hist_lens=None, prompt_lens=None, drafts=None, repetition=None,
                   presence=None, frequency=None, bias_ids=None, bias_values=None, masks=None, mask_index=None):
    """float64 logits after the rules, one token at a time."""
    x = np.array(logits, np.float64)
    n, V = x.shape
    for r in range(n):
        s, j = divmod(r, rows_per_seq)
        if history is not None:
            width = history.shape[1]
            length = min(max(int(hist_lens[s]), 0), width)
            prompt = min(max(int(prompt_lens[s]), 0), length)
            after = [int(t) for t in history[s, prompt:length]]
            if drafts is not None:
                after += [int(t) for t in drafts[s, :j]]
            count = {}
            for t in after:
                if 0 <= t < V:
                    count[t] = count.get(t, 0) + 1
            seen = {int(t) for t in history[s, :prompt] if 0 <= t < V} | set(count)
            rep = 1.0 if repetition is None else float(repetition[s])
            for t in seen:
                x[r, t] = x[r, t] / rep if x[r, t] > 0 else x[r, t] * rep
            for t, c in count.items():
                x[r, t] -= (0.0 if frequency is None else float(frequency[s])) * c
                x[r, t] -= 0.0 if presence is None else float(presence[s])
        if bias_ids is not None:
            last = {int(t): float(b) for t, b in zip(bias_ids[s], bias_values[s]) if 0 <= t < V}
            for t, b in last.items():
                x[r, t] += b
        if masks is not None and 0 <= int(mask_index[r]) < len(masks):
            words = np.asarray(masks[int(mask_index[r])]).view(np.uint32)
            bits = (words[:, None] >> np.arange(32, dtype=np.uint32)) & 1
            x[r, bits.reshape(-1)[:V] == 0] = -np.inf
    return x
