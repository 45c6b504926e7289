"""The operators around a tree of drafted tokens, as cases that can be timed: attention of a tree over a paged cache, the
bookkeeping of a verified tree (masks and positions before the pass, acceptance and compaction behind it), forking and releasing
sequences that share pages, and log probabilities of given tokens with their gradient.

Where ``own`` is false, ``run`` computes each operator in its plain form from elementary torch operations; where it is
true, it calls the library's operators."""
import numpy as np
import torch

own = False

PAGE = 64  # tokens per KV page
DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
NO_TOKEN = -1

# Head layouts (query heads, KV heads, head_dim) of the repository's workloads, and more group sizes.
HEADS = [(32, 8, 128), (8, 2, 128), (4, 1, 128), (4, 2, 64), (16, 8, 64), (8, 8, 128), (16, 2, 128), (6, 2, 128)]


def listed():
    return [
        # one sequence of the 512-token workload, a tree of 16 nodes: latency
        dict(name="attn_b1_m16_n512", op="attn", dtype="bf16", batch=1, heads=32, kv_heads=8, hd=128, prefix=0, own_lo=512,
             own_hi=512, m_lo=16, m_hi=16),
        # concurrency 32, ragged trees of up to 64 nodes behind an 8192-token prefix: tensor cores
        dict(name="attn_b32_m64_p8192", op="attn", dtype="bf16", batch=32, heads=32, kv_heads=8, hd=128, prefix=8192,
             own_lo=256, own_hi=2048, m_lo=33, m_hi=64),
        # the fp32 path with 64-wide heads: small trees of an odd size
        dict(name="attn_f32_b3_m9_n500", op="attn", dtype="f32", batch=3, heads=4, kv_heads=2, hd=64, prefix=0, own_lo=100,
             own_hi=500, m_lo=9, m_hi=9),
        # the tree's bookkeeping for one sequence, over the caches of a 5-layer drafter: latency
        dict(name="step_b1_m16_l5", op="step", dtype="bf16", batch=1, kv_heads=8, hd=128, layers=5, own_lo=512, own_hi=512,
             m_lo=16, m_hi=16, acc_hi=4),
        # concurrency 32 and the 36 layers of the target: up to eight drafts accepted
        dict(name="step_b32_m64_l36", op="step", dtype="bf16", batch=32, kv_heads=8, hd=128, layers=36, own_lo=30, own_hi=200,
             m_lo=33, m_hi=64, acc_hi=8),
        # four samples of one prompt on a drafter's caches: latency
        dict(name="fork_b1_n4_l5", op="pages", dtype="bf16", batch=1, kids=4, kv_heads=8, hd=128, layers=5, kv_lo=520, kv_hi=520),
        # eight samples of each of eight prompts, 36 layers: bandwidth
        dict(name="fork_b8_n64_l36", op="pages", dtype="bf16", batch=8, kids=64, kv_heads=8, hd=128, layers=36, kv_lo=256,
             kv_hi=960),
        # the log probability of one sampled token and its 20 alternatives at the Qwen3 vocabulary: latency
        dict(name="logprobs_r1_top20", op="logprobs", dtype="f32", rows=1, vocab=151936, n=1, top=20, masked=False),
        # 64 bf16 rows at the LLaMA-3.1 vocabulary, eight children a node
        dict(name="logprobs_r64_bf16_n8", op="logprobs", dtype="bf16", rows=64, vocab=128256, n=8, top=8, masked=False),
        # a verify pass of 32 blocks of 16, some rows behind grammar masks
        dict(name="logprobs_r512_top5", op="logprobs", dtype="f32", rows=512, vocab=151936, n=1, top=5, masked=True),
        # the gradient of a small training block in bf16
        dict(name="grad_r64_bf16", op="grad", dtype="bf16", rows=64, vocab=128256, n=1, masked=False, entropy=True),
        # 512 anchors' rows in fp32
        dict(name="grad_r512", op="grad", dtype="f32", rows=512, vocab=151936, n=1, masked=False, entropy=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attn", "attn", "step", "pages", "logprobs", "logprobs", "grad"])
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        h, hkv, hd = rng.choice(HEADS)
        m_hi = rng.choice([1, _log(rng, 2, 64), _log(rng, 2, 256)])
        batch = _log(rng, 1, max(1, min(64, 2048 // m_hi)))
        prefix = rng.choice([0, _log(rng, 1, 8192)])
        own_hi = rng.choice([0, _log(rng, 1, 4096), _log(rng, 1, 4096)])
        most = 2.0e9 if dtype == "f32" else 1.5e11  # flops
        while 4.0 * batch * m_hi * h * hd * (prefix + own_hi + m_hi) > most:
            prefix, own_hi, m_hi = prefix * 3 // 4, own_hi * 3 // 4, max(1, m_hi * 3 // 4)
        return dict(op=op, dtype=dtype, batch=batch, heads=h, kv_heads=hkv, hd=hd, prefix=prefix,
                    own_lo=rng.randint(0, own_hi), own_hi=own_hi, m_lo=rng.choice([m_hi, rng.randint(0, m_hi)]), m_hi=m_hi)
    if op == "step":
        _, hkv, hd = rng.choice(HEADS)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        m_hi = _log(rng, 1, 256)
        batch, layers, own_hi = _log(rng, 1, max(1, min(64, 2048 // m_hi))), rng.randint(1, 36), _log(rng, 1, 1024)
        while batch * layers * hkv * hd * (own_hi + m_hi + 64) * (8 if dtype == "f32" else 4) > 1.2e9:
            batch, layers, own_hi = max(1, batch * 3 // 4), max(1, layers * 3 // 4), own_hi * 3 // 4
        return dict(op=op, dtype=dtype, batch=batch, kv_heads=hkv, hd=hd, layers=layers, own_lo=rng.randint(0, own_hi),
                    own_hi=own_hi, m_lo=rng.randint(1, m_hi), m_hi=m_hi, acc_hi=rng.randint(0, 15))
    if op == "pages":
        _, hkv, hd = rng.choice(HEADS)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        batch, kids, layers, kv_hi = _log(rng, 1, 64), _log(rng, 1, 256), rng.randint(1, 36), _log(rng, 1, 4096)
        while layers * hkv * hd * (batch * (kv_hi + 64) + 64 * kids) * (8 if dtype == "f32" else 4) > 1.2e9:
            batch, kids, layers, kv_hi = (max(1, x * 3 // 4) for x in (batch, kids, layers, kv_hi))
        return dict(op=op, dtype=dtype, batch=batch, kids=kids, kv_heads=hkv, hd=hd, layers=layers,
                    kv_lo=rng.randint(0, kv_hi), kv_hi=kv_hi)
    rows, vocab = _log(rng, 1, 512), _log(rng, 1000, 152064)
    case = dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), rows=rows, vocab=vocab, n=rng.choice([1, 1, rng.randint(2, 8)]))
    if op == "logprobs":
        return dict(case, top=rng.choice([0, rng.randint(1, 8), rng.randint(1, 32)]), masked=rng.random() < 0.3)
    return dict(case, masked=rng.random() < 0.3, entropy=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------------- inputs
def _spread(g, lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], in a drawn order: their sum is the same for every seed."""
    return (lo + (hi - lo + 1) * (2 * torch.arange(n) + 1) // (2 * n))[torch.randperm(n, generator=g)]


def _ceil(a, b):
    return (a + b - 1) // b


def _i32(x):
    return torch.as_tensor(x).to(torch.int32).to(DEV)


DEPTH = 32  # nodes on a path from the root, at most


def _tree(rng, m, acc):
    """Parents of a tree of m nodes in drafting order (a parent before its children), a path of 1 + acc nodes from the root, and
    each node's ancestors (itself among them) as a whole number's bits.  The path's drafts lie behind the rows that the accepted
    ones move to."""
    path = np.concatenate([[0], np.sort(rng.choice(np.arange(acc + 1, m), acc, replace=False))]).astype(int)
    parent, depth, seen = np.full(m, -1), np.zeros(m, int), [1] * m
    on = {int(b): int(a) for a, b in zip(path[:-1], path[1:])}
    for j in range(1, m):
        p = on.get(j, int(j * rng.random() ** 1.5))  # early nodes have more children
        parent[j] = p if j in on or depth[p] < DEPTH - 18 else 0
        depth[j] = depth[parent[j]] + 1
        seen[j] = seen[parent[j]] | 1 << j
    return parent, path, depth, seen


def _words(bits, words):
    """Rows of 32-bit words (int32) of whole numbers' bits."""
    raw = b"".join(b.to_bytes(4 * words, "little") for b in bits)
    return torch.from_numpy(np.frombuffer(raw, np.int32).reshape(len(bits), words).copy()).to(DEV)


def _lengths(case, seed):
    """A case's generator and host lengths, the same for prepare() and exact(): nodes and own keys (those of the tree among
    them), or the parents' lengths."""
    g = torch.Generator().manual_seed(int(seed))
    if case["op"] == "pages":
        return g, _spread(g, case["kv_lo"], case["kv_hi"], case["batch"]), None
    m = _spread(g, case["m_lo"], case["m_hi"], case["batch"])
    return g, m, m + _spread(g, case["own_lo"], case["own_hi"], case["batch"])


def _tables(g, kv, kv_hi, n_pre, spare):
    """Prefix pages, page tables of sequences of kv <= kv_hi tokens (two entries to spare; a page behind the last stands for
    no page), the number of pages, and spare free ones."""
    used, width = _ceil(kv, PAGE), _ceil(kv_hi, PAGE) + 2
    n = n_pre + len(kv) * _ceil(kv_hi, PAGE) + spare + 1
    perm = torch.randperm(n - 1, generator=g)
    table = torch.full((len(kv), width), n - 1, dtype=torch.int64)
    table[torch.arange(width)[None, :] < used[:, None]] = perm[n_pre:n_pre + int(used.sum())]
    return perm[:n_pre], table, n, perm[n - 1 - spare:]


def prepare(case, seed):
    op, dt = case["op"], DTYPES[case["dtype"]]
    d = torch.Generator(DEV).manual_seed(int(seed) + 1)
    rng = np.random.default_rng(int(seed) + 2)

    def noise(*shape):
        return torch.randn(shape, generator=d, device=DEV)

    i32 = dict(dtype=torch.int32, device=DEV)
    if op == "attn":
        g, m, kv = _lengths(case, seed)
        h, hkv, hd, pre = case["heads"], case["kv_heads"], case["hd"], case["prefix"]
        pre_pages, table, n_pages, _ = _tables(g, kv, case["own_hi"] + case["m_hi"], _ceil(pre, PAGE), 0)
        rows, words = max(1, int(m.sum())), max(1, _ceil(int(m.max()), 32))
        bits = [b for n in m.tolist() if n for b in _tree(rng, n, 0)[3]] or [0]
        # normed and rotated queries and keys have unit RMS a channel, values a plain spread
        return dict(op=op, q=noise(rows, h, hd).to(dt), k=noise(n_pages, hkv, PAGE, hd).to(dt),
                    v=noise(n_pages, hkv, PAGE, hd).to(dt), prefix=pre, prefix_pages=_i32(pre_pages), table=_i32(table),
                    kv=_i32(kv), q_start=_i32(torch.cat([torch.zeros(1, dtype=torch.int64), m.cumsum(0)])),
                    masks=_words(bits, words), max_m=max(1, int(m.max())), out=torch.zeros((rows, h, hd), dtype=dt, device=DEV),
                    lse=torch.zeros((rows, h), device=DEV))
    if op == "step":
        g, m, kv = _lengths(case, seed)
        b, hkv, hd, layers, rows = case["batch"], case["kv_heads"], case["hd"], case["layers"], int(m.sum())
        _, table, n_pages, _ = _tables(g, kv, case["own_hi"] + case["m_hi"], 0, 0)
        parents, tokens, posterior = [], [], []
        for i, n in enumerate(m.tolist()):
            ids = rng.choice(100000, n + 1, replace=False)  # a tree's tokens differ
            parent, path, _, _ = _tree(rng, n, min(case["acc_hi"] * (i + 1) // b, (n - 1) // 2))
            post = rng.integers(0, 100000, n)
            post[path] = np.concatenate([ids[path[1:]], ids[n:]])
            parents.append(parent), tokens.append(ids[:n]), posterior.append(post)
        return dict(op=op, parents=_i32(np.concatenate(parents)), tokens=_i32(np.concatenate(tokens)),
                    posterior=_i32(np.concatenate(posterior)), max_m=int(m.max()), table=_i32(table), kv=_i32(kv),
                    q_start=_i32(torch.cat([torch.zeros(1, dtype=torch.int64), m.cumsum(0)])),
                    k=noise(layers, n_pages, hkv, PAGE, hd).to(dt), v=noise(layers, n_pages, hkv, PAGE, hd).to(dt),
                    masks=torch.empty((rows, _ceil(int(m.max()), 32)), **i32), depth=torch.empty(rows, **i32),
                    row_pos=torch.empty(rows, **i32), path=torch.empty((b, DEPTH), **i32), accepted=torch.empty(b, **i32),
                    bonus=torch.empty(b, **i32), kv_out=torch.empty(b, **i32), status=torch.empty((3, b), **i32))
    if op == "pages":
        g, kv, _ = _lengths(case, seed)
        b, kids, hkv, hd, layers = case["batch"], case["kids"], case["kv_heads"], case["hd"], case["layers"]
        taken, spare = 3, kids + 3  # pages of the free list that earlier steps took, and what is left
        _, table, n_pages, free = _tables(g, kv, case["kv_hi"], 0, taken + spare)
        return dict(op=op, kv=_i32(kv), table=_i32(table), parents=_i32(torch.arange(kids) % b), free=_i32(free),
                    used=_i32([taken]), refs=torch.zeros(n_pages, **i32), scratch=n_pages - 1,
                    k=noise(layers, n_pages, hkv, PAGE, hd).to(dt), v=noise(layers, n_pages, hkv, PAGE, hd).to(dt),
                    kid_table=torch.empty((kids, table.shape[1]), **i32), kid_lens=torch.empty(kids, **i32),
                    fork_used=torch.empty(1, **i32), used_out=torch.empty(1, **i32), all_kids=_i32(torch.arange(kids)),
                    status=torch.empty(2, **i32))
    rows, vocab, n = case["rows"], case["vocab"], case["n"]
    logits = 3.0 * noise(rows, vocab)
    if case["masked"]:  # every fourth row behind a grammar mask that allows a tenth of the vocabulary
        closed = torch.rand((_ceil(rows, 4), vocab), generator=d, device=DEV) > 0.1
        closed[:, ::7] = False
        logits[::4] = logits[::4].masked_fill(closed, float("-inf"))
    logits = logits.to(dt)
    # a sampled token is a likely one: the largest of a few drawn at random (an allowed one where there are masks)
    some = torch.randint(0, _ceil(vocab, 7), (rows, n, 64), generator=d, device=DEV) * 7
    tokens = some.gather(2, logits.gather(1, some.view(rows, -1)).view(some.shape).argmax(2, keepdim=True))[..., 0]
    tokens[rows // 2:, n - 1][1::5] = NO_TOKEN  # padding
    tokens = tokens.to(torch.int32)
    f32 = dict(dtype=torch.float32, device=DEV)
    if op == "logprobs":
        k = case["top"]
        return dict(op=op, logits=logits, tokens=tokens, top=k, logprobs=torch.empty((rows, n), **f32),
                    ranks=torch.empty((rows, n), **i32), entropy=torch.empty(rows, **f32), lse=torch.empty(rows, **f32),
                    top_ids=torch.empty((rows, k), **i32), top_logprobs=torch.empty((rows, k), **f32))
    x = logits.float()
    z = x - x.amax(1, keepdim=True)
    lse = z.exp().sum(1).log()
    entropy = lse - (z.exp() * z.clamp(min=-200)).sum(1) / z.exp().sum(1)
    return dict(op=op, logits=logits, tokens=tokens, lse=lse + x.amax(1), entropy=entropy,
                grad=noise(rows, n) / rows, grad_entropy=0.01 * noise(rows) / rows if case["entropy"] else None,
                out=torch.empty_like(logits))


# ---------------------------------------------------------------------------------------------------- one pass
def run(state):
    return {"attn": _attn, "step": _step, "pages": _pages, "logprobs": _logprobs, "grad": _grad}[state["op"]](state)


def _attn(s):
    if own:
        import block_diffusion_speculative_ctx_gb300 as dfl
        out, lse = dfl.tree_attention(s["q"], s["k"], s["v"], s["table"], s["kv"], s["q_start"], s["masks"],
                                      prefix_pages=s["prefix_pages"], prefix_len=s["prefix"], out=s["out"], lse=s["lse"])
        return [out, lse]
    q, start, kv = s["q"].float(), s["q_start"].long(), s["kv"].long()
    rows, h, hd = q.shape
    hkv = s["k"].shape[1]
    g, b, pre = h // hkv, kv.numel(), s["prefix"]
    scale = hd ** -0.5
    # row r is row j of sequence seq; rows padded to [batch, max_m]
    r = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(start[1:], r, right=True).clamp(max=b - 1)
    j, m = r - start[seq], start[1:] - start[:-1]
    pad = (start[:-1, None] + torch.arange(s["max_m"], device=DEV)).clamp(max=rows - 1)
    # the prefix: every row of a KV head's query group against the same keys
    kp = s["k"][s["prefix_pages"].long()].transpose(0, 1).reshape(hkv, -1, hd)[:, :pre].float()
    vp = s["v"][s["prefix_pages"].long()].transpose(0, 1).reshape(hkv, -1, hd)[:, :pre].float()
    qg = q.view(rows, hkv, g, hd)
    sp = (qg.permute(1, 0, 2, 3).reshape(hkv, rows * g, hd) @ kp.transpose(1, 2)).mul_(scale)
    sp = sp.view(hkv, rows, g, pre)
    # each sequence's own keys: the committed ones, and those of the tree that the row's mask names
    kq = s["k"][s["table"].long()].transpose(1, 2).reshape(b, hkv, -1, hd).float()
    vq = s["v"][s["table"].long()].transpose(1, 2).reshape(b, hkv, -1, hd).float()
    keys = kq.shape[2]
    node = torch.arange(keys, device=DEV) - (kv - m)[seq][:, None]
    at = node.clamp(0, 32 * s["masks"].shape[1] - 1)
    bit = (s["masks"].gather(1, at >> 5) >> (at & 31).to(torch.int32)) & 1
    sees = (node < 0) | ((node < m[seq][:, None]) & (bit == 1))
    qb = qg[pad].permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, hd)
    sq = (qb @ kq.transpose(2, 3)).mul_(scale).view(b, hkv, s["max_m"], g, keys)[seq, :, j].transpose(0, 1)
    sq = sq.masked_fill(~sees[None, :, None, :], float("-inf"))
    top = sq.amax(-1)
    if pre:
        top = torch.maximum(sp.amax(-1), top)
    top0 = torch.where(torch.isinf(top), torch.zeros_like(top), top)[..., None]
    pp, pq = (sp - top0).exp(), (sq - top0).exp()
    den = pp.sum(-1) + pq.sum(-1)
    op = (pp.view(hkv, rows * g, pre) @ vp).view(hkv, rows, g, hd)
    wide = torch.zeros((b, s["max_m"], hkv, g, keys), device=DEV)
    wide[seq, j] = pq.transpose(0, 1)
    oq = (wide.permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, keys) @ vq).view(b, hkv, s["max_m"], g, hd)[seq, :, j]
    out = (op.transpose(0, 1) + oq) / den.transpose(0, 1)[..., None].clamp(min=1e-30)
    lse = (top + den.log()).transpose(0, 1).reshape(rows, h)
    live = r < start[-1]
    return [torch.where(live[:, None, None], out.reshape(rows, h, hd), 0.0).to(s["q"].dtype),
            torch.where(live[:, None], lse, 0.0)]


def _step(s):
    if own:
        import block_diffusion_speculative_ctx_gb300 as dfl
        t = dfl.tree_masks(s["parents"], s["q_start"], kv_lens=s["kv"], masks=s["masks"], depth=s["depth"],
                           row_pos=s["row_pos"], status=s["status"][0])
        a = dfl.tree_accept(s["parents"], s["tokens"], s["posterior"], s["q_start"], path=s["path"], accepted=s["accepted"],
                            bonus=s["bonus"], status=s["status"][1])
        c = dfl.kv_compact(s["k"], s["v"], s["table"], s["kv"], s["q_start"], a.path, a.accepted, kv_out=s["kv_out"],
                           status=s["status"][2])
        return [t.masks, t.depth, t.row_pos, a.path, a.accepted, a.bonus, c.kv_lens, s["status"], s["k"], s["v"]]
    start, kv, wide = s["q_start"].long(), s["kv"].long(), s["max_m"]
    rows, b = s["parents"].numel(), kv.numel()
    m = start[1:] - start[:-1]
    seq = torch.searchsorted(start[1:], torch.arange(rows, device=DEV), right=True)
    j = torch.arange(rows, device=DEV) - start[seq]
    node = torch.arange(wide, device=DEV)
    pad = (start[:-1, None] + node).clamp(max=rows - 1)
    real = node < m[:, None]
    parent = torch.where(real, s["parents"].long()[pad], -1)
    # ancestors: the links' powers, as far as the deepest node
    link = torch.eye(wide, device=DEV) + (parent[:, :, None] == node).float()
    seen = (torch.linalg.matrix_power(link, DEPTH) > 0) & real[:, :, None]
    depth = seen.sum(2) - 1
    words = s["masks"].shape[1]
    bits = torch.zeros((b, wide, words * 32), dtype=torch.int64, device=DEV)
    bits[:, :, :wide] = seen.long()
    packed = (bits.view(b, wide, words, 32) << torch.arange(32, device=DEV)).sum(-1)
    masks = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)[seq, j]
    row_depth = depth[seq, j]
    row_pos = (kv - m)[seq] + row_depth
    # the drafted child that the target chose, the lowest where two hold its token
    token, post = s["tokens"].long()[pad], s["posterior"].long()[pad]
    hit = (parent >= 0) & (token == post.gather(1, parent.clamp(min=0)))
    first = torch.full((b, wide + 1), wide, device=DEV).scatter_reduce_(
        1, torch.where(hit, parent, wide), node.expand(b, wide), "amin")
    chosen = hit & (first.gather(1, parent.clamp(min=0)) == node)
    chosen[:, 0] = True
    on = (chosen[:, None, :] | ~seen).all(2) & seen[:, :, 0]
    accepted = on.sum(1) - 1
    path = torch.full((b, DEPTH + 1), -1, device=DEV).scatter_(1, torch.where(on, depth, DEPTH), node.expand(b, wide))
    path[:, DEPTH] = -1
    path = path[:, :DEPTH]
    last = path.gather(1, accepted[:, None])
    bonus = post.gather(1, last)[:, 0]
    # accepted rows to their places
    step = torch.arange(DEPTH, device=DEV).expand(b, DEPTH)
    moved = path >= 0
    src, dst = ((kv - m)[:, None] + path)[moved], ((kv - m)[:, None] + step)[moved]
    of = torch.arange(b, device=DEV)[:, None].expand(b, DEPTH)[moved]
    table = s["table"].long()
    for c in (s["k"], s["v"]):
        c[:, table[of, dst // PAGE], :, dst % PAGE] = c[:, table[of, src // PAGE], :, src % PAGE]
    return [masks, row_depth.to(torch.int32), row_pos.to(torch.int32), path.to(torch.int32), accepted.to(torch.int32),
            bonus.to(torch.int32), (kv - m + accepted + 1).to(torch.int32), torch.zeros_like(s["status"]), s["k"], s["v"]]


def _pages(s):
    if own:
        import block_diffusion_speculative_ctx_gb300 as dfl
        f = dfl.kv_fork(s["parents"], s["kv"], s["table"], s["free"], s["used"], s["refs"], s["k"], s["v"],
                        scratch_page=s["scratch"], table_out=s["kid_table"], lens_out=s["kid_lens"], used_out=s["fork_used"],
                        status=s["status"][:1])
        r = dfl.kv_release(s["all_kids"], f.kv_lens, f.table, s["free"], f.used, s["refs"], used_out=s["used_out"],
                           status=s["status"][1:])
        return [f.table, f.kv_lens, f.used, r.used, s["status"], s["free"], s["refs"], s["k"], s["v"]]
    parents = s["parents"].long()
    kv, rows = s["kv"].long()[parents], s["table"][parents]
    full, tail = kv // PAGE, kv % PAGE
    col = torch.arange(rows.shape[1], device=DEV)
    takes = (tail > 0).long()
    at = s["used"].long() + takes.cumsum(0) - takes
    fresh = s["free"][at]
    table = torch.where(col < full[:, None], rows, torch.where((col == full[:, None]) & (tail > 0)[:, None], fresh[:, None], s["scratch"]))
    fork_used = s["used"] + takes.sum().to(torch.int32)
    shared = col < full[:, None]
    s["refs"].index_add_(0, torch.where(shared, rows, 0).flatten().long(), shared.flatten().to(torch.int32))
    # the tokens of the page that ends inside
    copied = (torch.arange(PAGE, device=DEV) < tail[:, None]).nonzero()
    kid, t = copied[:, 0], copied[:, 1]
    src, dst = rows[kid, full[kid]].long(), fresh[kid].long()
    for c in (s["k"], s["v"]):
        c[:, dst, :, t] = c[:, src, :, t]
    # and back: every page of the children, in the order of the first child that holds it
    held = col < _ceil(kv, PAGE)[:, None]
    entry = torch.arange(held.numel(), device=DEV).view(held.shape)
    n_pages = s["refs"].numel()
    page = torch.where(held, table, n_pages).flatten().long()
    holders = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV).index_add_(0, page, torch.ones_like(page, dtype=torch.int32))[:-1]
    first = torch.full((n_pages + 1,), held.numel(), device=DEV).scatter_reduce_(0, page, entry.flatten(), "amin")[:-1]
    left = s["refs"] - holders
    gone = left < 0
    order = torch.where(gone, first, held.numel()).sort(stable=True)[1]
    place = torch.arange(s["free"].numel(), device=DEV) - (fork_used.long() - gone.sum())
    s["free"].copy_(torch.where((place >= 0) & (place < gone.sum()), order[place.clamp(0, n_pages - 1)].to(torch.int32), s["free"]))
    s["refs"].copy_(left.clamp(min=0))
    return [table.to(torch.int32), kv.to(torch.int32), fork_used, fork_used - gone.sum().to(torch.int32),
            torch.zeros_like(s["status"]), s["free"], s["refs"], s["k"], s["v"]]


def _logprobs(s):
    if own:
        import block_diffusion_speculative_ctx_gb300 as dfl
        t = dfl.token_logprobs(s["logits"], s["tokens"], top=s["top"], logprobs=s["logprobs"], ranks=s["ranks"],
                               entropy=s["entropy"], lse=s["lse"], top_ids=s["top_ids"] if s["top"] else None,
                               top_logprobs=s["top_logprobs"] if s["top"] else None)
        return [t.logprobs, t.ranks, t.entropy, t.lse] + ([t.top_ids, t.top_logprobs] if s["top"] else [])
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    z = x - top
    e = z.exp()
    total = e.sum(1, keepdim=True)
    log_total = total.log()
    entropy = (log_total - (e * z.clamp(min=-200.0)).sum(1, keepdim=True) / total)[:, 0]
    real, t = s["tokens"] >= 0, s["tokens"].long().clamp(min=0)
    logprobs = torch.where(real, z.gather(1, t) - log_total, 0.0)
    v = torch.arange(x.shape[1], device=DEV)
    xt = x.gather(1, t)
    ahead = [((x > xt[:, i:i + 1]) | ((x == xt[:, i:i + 1]) & (v < t[:, i:i + 1]))).sum(1) for i in range(t.shape[1])]
    ranks = torch.where(real, torch.stack(ahead, 1), -1).to(torch.int32)
    back = [logprobs, ranks, entropy, (top + log_total)[:, 0]]
    if s["top"]:
        best, ids = x.sort(dim=1, descending=True, stable=True)
        back += [ids[:, :s["top"]].to(torch.int32), best[:, :s["top"]] - top - log_total]
    return back


def _grad(s):
    if own:
        import block_diffusion_speculative_ctx_gb300 as dfl
        return dfl.token_logprobs_grad(s["logits"], s["tokens"], s["lse"], s["grad"], entropy=s["entropy"],
                                       grad_entropy=s["grad_entropy"], out=s["out"])
    z = s["logits"].float() - s["lse"][:, None]
    p = z.exp()
    real = s["tokens"] >= 0
    g = torch.where(real, s["grad"], 0.0)
    d = -p * g.sum(1, keepdim=True)
    if s["grad_entropy"] is not None:
        d -= s["grad_entropy"][:, None] * p * (z.clamp(min=-200.0) + s["entropy"][:, None])
    d.scatter_add_(1, s["tokens"].long().clamp(min=0), g)
    return d.to(s["logits"].dtype)


# ------------------------------------------------------------------------------------------------- 64-bit answers
def exact(case, seed):
    if case["op"] in ("step", "pages"):
        return None  # whole numbers, and copies of what the caches hold
    s = prepare(case, seed)
    if case["op"] == "attn":
        _, m, kv = _lengths(case, seed)
        q = s["q"].double()
        rows, h, hd = q.shape
        out, lse = torch.zeros_like(q), torch.zeros((rows, h), dtype=torch.float64, device=DEV)
        start = 0
        for i in range(case["batch"]):
            n, mine = int(m[i]), int(kv[i])
            if n == 0:
                continue
            pages = [s["prefix_pages"].long(), s["table"][i, : _ceil(mine, PAGE)].long()]
            keep = [case["prefix"], mine]
            k = torch.cat([s["k"][p].transpose(0, 1).flatten(1, 2)[:, :c] for p, c in zip(pages, keep)], 1).double()
            v = torch.cat([s["v"][p].transpose(0, 1).flatten(1, 2)[:, :c] for p, c in zip(pages, keep)], 1).double()
            k, v = (t.repeat_interleave(h // t.shape[0], 0) for t in (k, v))  # one copy a query head
            z = torch.einsum("rhd,hkd->hrk", q[start:start + n], k) / hd ** 0.5
            word = s["masks"][start:start + n]
            sees = ((word[:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1).flatten(1)[:, :n] == 1
            z[:, :, case["prefix"] + mine - n:].masked_fill_(~sees[None], float("-inf"))
            lse[start:start + n] = torch.logsumexp(z, -1).T
            out[start:start + n] = torch.einsum("hrk,hkd->rhd", torch.softmax(z, -1), v)
            start += n
        return [out, lse]
    rows, n = s["tokens"].shape
    real, t = s["tokens"] >= 0, s["tokens"].long().clamp(min=0)
    if case["op"] == "logprobs":
        logp = torch.log_softmax(s["logits"].double(), 1)
        entropy = torch.special.entr(logp.exp()).sum(1)
        back = [torch.where(real, logp.gather(1, t), 0.0), None, entropy, torch.logsumexp(s["logits"].double(), 1)]
        return back + ([None, logp.topk(case["top"], 1)[0]] if case["top"] else [])
    g = torch.where(real, s["grad"], 0.0).double()
    out = torch.empty(s["logits"].shape, dtype=torch.float64, device=DEV)
    for r in range(rows):
        logp = torch.log_softmax(s["logits"][r].double(), 0)
        p = logp.exp()
        d = -p * g[r].sum()
        if s["grad_entropy"] is not None:
            entropy = torch.special.entr(p).sum()
            d -= s["grad_entropy"][r].double() * (-torch.special.entr(p) + p * entropy)
        out[r] = d.index_add_(0, t[r], g[r])
    return out


def work(case):
    """Each input read once and each output written once; lengths that are drawn count at their mean."""
    e, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op == "attn":
        b, m, h, hd = case["batch"], (case["m_lo"] + case["m_hi"]) / 2, case["heads"], case["hd"]
        mine, rows = (case["own_lo"] + case["own_hi"]) / 2, b * m
        return {"bytes": 2 * e * hd * (case["kv_heads"] * (case["prefix"] + b * (mine + m)) + rows * h) + 4 * rows * h
                + rows * _ceil(case["m_hi"], 32) * 4,
                "flops": 4 * rows * h * hd * (case["prefix"] + mine + min(m, 6.0))}
    if op == "step":
        b, m = case["batch"], (case["m_lo"] + case["m_hi"]) / 2
        moved = sum(min(case["acc_hi"] * (i + 1) // b, (case["m_lo"] - 1) // 2) for i in range(b))
        return {"bytes": b * m * (4 * _ceil(case["m_hi"], 32) + 24) + b * (DEPTH * 4 + 20)
                + moved * case["layers"] * 4 * e * case["kv_heads"] * case["hd"], "flops": 0}
    if op == "pages":
        kv = (case["kv_lo"] + case["kv_hi"]) / 2
        tail = PAGE / 2 if case["kv_hi"] != case["kv_lo"] else kv % PAGE
        return {"bytes": case["kids"] * (tail * case["layers"] * 4 * e * case["kv_heads"] * case["hd"]
                                         + 8 * _ceil(case["kv_hi"], PAGE) + 24 * kv / PAGE), "flops": 0}
    rows, vocab, n = case["rows"], case["vocab"], case["n"]
    if op == "logprobs":
        return {"bytes": rows * (e * vocab + 12 * n + 8 * case["top"] + 8), "flops": 0}
    return {"bytes": rows * (2 * e * vocab + 8 * n + 12), "flops": 0}
