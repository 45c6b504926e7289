"""Oracles of the operators around a tree of drafted tokens, of pages that several sequences hold and of token log
probabilities, in plain numpy loops (fp64)."""
from __future__ import annotations

import numpy as np

PAGE = 64


def ancestors(parents):
    """[m, m] truth values: node j sees node i (itself or an ancestor); depths [m]."""
    m = len(parents)
    sees, depth = np.zeros((m, m), bool), np.zeros(m, int)
    for j, p in enumerate(parents):
        if p >= 0:
            sees[j], depth[j] = sees[p], depth[p] + 1
        sees[j, j] = True
    return sees, depth


def words(sees, n):
    """Rows of truth values as n 32-bit words each (int32)."""
    bits = np.zeros((len(sees), 32 * n), np.uint64)
    bits[:, :sees.shape[1]] = sees
    packed = (bits.reshape(len(sees), n, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return packed.astype(np.uint32).view(np.int32)


def tree_attention(q, k_cache, v_cache, prefix_pages, prefix_len, table, kv_lens, q_start, sees, scale):
    """(out, lse, weight) as serving.shared_prefix_attention gives them; sees[s]: [m, m] truth values."""
    rows, H, hd = q.shape
    hkv = k_cache.shape[1]
    out, lse, weight = np.full((rows, H, hd), np.nan), np.full((rows, H), np.nan), np.full((rows, H, hd), np.nan)

    def keys(cache, pages, n):
        x = cache[np.asarray(pages[: -(-n // PAGE)], np.int64)]
        return x.transpose(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :n].astype(np.float64)

    for s in range(len(kv_lens)):
        a, b, n = int(q_start[s]), int(q_start[s + 1]), int(kv_lens[s])
        m = b - a
        K = np.concatenate([keys(k_cache, prefix_pages, prefix_len), keys(k_cache, table[s], n)], 1)
        V = np.concatenate([keys(v_cache, prefix_pages, prefix_len), keys(v_cache, table[s], n)], 1)
        for r in range(a, b):
            on = np.ones(prefix_len + n, bool)
            for i in range(m):
                if n - m + i >= 0:
                    on[prefix_len + n - m + i] = i < sees[s].shape[1] and sees[s][r - a, i]
            for h in range(H):
                if not on.any():
                    out[r, h], lse[r, h], weight[r, h] = 0.0, -np.inf, 0.0
                    continue
                z = scale * (K[h // (H // hkv)][on] @ q[r, h].astype(np.float64))
                p = np.exp(z - z.max())
                out[r, h] = p @ V[h // (H // hkv)][on] / p.sum()
                weight[r, h] = p @ np.abs(V[h // (H // hkv)][on]) / p.sum()
                lse[r, h] = z.max() + np.log(p.sum())
    return out, lse, weight


def tree_accept(parents, tokens, posterior, width):
    """(path, accepted, bonus) of one tree."""
    if len(parents) == 0:
        return [-1] * width, -1, -1
    path = [0]
    while len(path) < width:
        kids = [j for j in range(len(parents)) if parents[j] == path[-1] and tokens[j] == posterior[path[-1]]]
        if not kids:
            break
        path.append(kids[0])
    return path + [-1] * (width - len(path)), len(path) - 1, int(posterior[path[-1]])


def kv_compact(cache, table, kv_lens, q_start, path, accepted):
    """cache [layers, pages, H_kv, 64, hd] (a copy) and the lengths behind."""
    cache, out = cache.copy(), []
    for s in range(len(kv_lens)):
        m = int(q_start[s + 1] - q_start[s])
        first = int(kv_lens[s]) - m
        rows = [cache[:, table[s, (first + i) // PAGE], :, (first + i) % PAGE].copy() for i in path[s][:accepted[s] + 1]]
        for j, row in enumerate(rows):
            cache[:, table[s, (first + j) // PAGE], :, (first + j) % PAGE] = row
        out.append(first + accepted[s] + 1)
    return cache, out


def kv_fork(parents, kv_lens, table, free_pages, used, refs, caches, scratch):
    """(tables, lengths, used, refs, caches) of the children."""
    refs, caches = refs.copy(), [c.copy() for c in caches]
    tables = np.full((len(parents), table.shape[1]), scratch)
    for c, p in enumerate(parents):
        n = int(kv_lens[p])
        for j in range(n // PAGE):
            tables[c, j] = table[p, j]
            refs[table[p, j]] += 1
        if n % PAGE:
            tables[c, n // PAGE] = free_pages[used]
            for x in caches:
                x[:, free_pages[used], :, : n % PAGE] = x[:, table[p, n // PAGE], :, : n % PAGE]
            used += 1
    return tables, [int(kv_lens[p]) for p in parents], used, refs, caches


def kv_release(seqs, kv_lens, table, free_pages, used, refs, keep=None):
    """(free_pages, used, refs, status)."""
    names = [int(p) for s in seqs for p in table[s, -(-int(keep[s]) // PAGE) if keep is not None else 0: -(-int(kv_lens[s]) // PAGE)]]
    gone = [p for p in dict.fromkeys(names) if names.count(p) == refs[p] + 1]
    if any(names.count(p) > refs[p] + 1 for p in names):
        return free_pages, used, refs, 32
    if len(gone) > used:
        return free_pages, used, refs, 1
    refs, free_pages = refs.copy(), free_pages.copy()
    for p in names:
        refs[p] -= 1
    refs[gone] = 0
    free_pages[used - len(gone):used] = gone
    return free_pages, used - len(gone), refs, 0


def token_logprobs(logits, tokens, top, temperature=1.0):
    """(logprobs, ranks, entropy, lse, top_ids, top_logprobs) of fp64 rows; tokens [rows, n]."""
    rows, V = logits.shape
    logprobs, ranks = np.zeros(tokens.shape), np.full(tokens.shape, -1)
    entropy, lse = np.zeros(rows), np.zeros(rows)
    top_ids, top_logprobs = np.full((rows, top), -1), np.full((rows, top), -np.inf)
    for r in range(rows):
        x = logits[r].astype(np.float64)
        if np.isnan(x).any() or np.isposinf(x).any():
            logprobs[r] = np.where((tokens[r] >= 0) & (tokens[r] < V), np.nan, 0.0)
            entropy[r] = lse[r] = np.nan
            top_logprobs[r] = np.nan
            continue
        best = x.max()
        if np.isneginf(best):
            logp, entropy[r], lse[r] = np.full(V, -np.inf), 0.0, -np.inf
        else:
            z = (x - best) / temperature
            logp = z - np.log(np.exp(z).sum())
            p = np.exp(logp)
            entropy[r] = -(p[p > 0] * logp[p > 0]).sum()
            lse[r] = best / temperature + np.log(np.exp(z).sum())
        for i, t in enumerate(tokens[r]):
            if 0 <= t < V:
                logprobs[r, i] = logp[t]
                ranks[r, i] = (x > x[t]).sum() + (x[:t] == x[t]).sum()
        order = np.lexsort((np.arange(V), -x))[:top]
        order = order[x[order] > -np.inf]
        top_ids[r, : len(order)], top_logprobs[r, : len(order)] = order, logp[order]
    return logprobs, ranks, entropy, lse, top_ids, top_logprobs


def token_logprobs_grad(logits, tokens, grad_logprobs, grad_entropy, temperature=1.0):
    """Gradient of sum(grad_logprobs * logprobs) + sum(grad_entropy * entropy) by fp64 logits."""
    out = np.zeros(logits.shape)
    for r in range(len(logits)):
        x = logits[r].astype(np.float64)
        real = (tokens[r] >= 0) & (tokens[r] < len(x))
        p = np.zeros(len(x))
        if x.max() > -np.inf:
            z = (x - x.max()) / temperature
            p = np.exp(z) / np.exp(z).sum()
        out[r] = -p * grad_logprobs[r][real].sum()
        logp = np.log(np.where(p > 0, p, 1.0))
        out[r] -= grad_entropy[r] * p * (logp - (p * logp).sum())
        np.add.at(out[r], tokens[r][real], grad_logprobs[r][real])
    return out / temperature
