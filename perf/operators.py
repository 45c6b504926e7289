"""The serving operators next to the draft-and-verify round, as cases that can be timed: page tables and slot maps
from request lengths, attention of a batch that shares a prefix, and the logit rules (penalties, biases, grammar masks).

Where ``own`` is false, ``run`` computes each operator in its plain form from elementary torch operations; where it is
true, it calls the library's operators."""
import torch

own = False

PAGE = 64  # tokens per KV page
DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# Head layouts (query heads, KV heads, head_dim) of the repository's workloads, and two more group sizes.
HEADS = [(32, 8, 128), (8, 2, 128), (4, 1, 128), (4, 2, 64), (16, 8, 64), (8, 8, 128), (16, 2, 128), (6, 2, 128)]


def listed():
    return [
        # one decode step of the concurrency-32 workload: every request appends one token
        dict(name="tables_step_b32", op="tables", batch=32, kv_lo=256, kv_hi=2303, new_lo=1, new_hi=1, width=40, base=0),
        # 1024 requests (the largest session) behind an 8192-token prefix, a 16-row block each
        dict(name="tables_block_b1024", op="tables", batch=1024, kv_lo=0, kv_hi=2303, new_lo=16, new_hi=16, width=160,
             base=8192),
        # one single-token step of four requests behind a short system prompt: latency
        dict(name="attn_step_b4_p512", op="attn", dtype="bf16", batch=4, heads=32, kv_heads=8, hd=128, prefix=512,
             kv_lo=1, kv_hi=100, q_lo=1, q_hi=1, causal=True),
        # single-token steps of the concurrency-32 workload behind an 8192-token prefix: cache bandwidth
        dict(name="attn_step_b32_p8192", op="attn", dtype="bf16", batch=32, heads=32, kv_heads=8, hd=128, prefix=8192,
             kv_lo=256, kv_hi=2048, q_lo=1, q_hi=1, causal=True),
        # the drafter's bidirectional block of 16 for a batch of 8 behind a prefix that ends inside a page
        dict(name="attn_draft_b8_p1000", op="attn", dtype="bf16", batch=8, heads=32, kv_heads=8, hd=128, prefix=1000,
             kv_lo=16, kv_hi=300, q_lo=16, q_hi=16, causal=False),
        # verify blocks of 16 rows at concurrency 32 behind an 8192-token prefix: tensor cores
        dict(name="attn_verify_b32_p8192", op="attn", dtype="bf16", batch=32, heads=32, kv_heads=8, hd=128, prefix=8192,
             kv_lo=256, kv_hi=2048, q_lo=16, q_hi=16, causal=True),
        # prefill of 32 ragged questions (their own keys only) behind a 2100-token prompt
        dict(name="attn_suffix_b32_p2100", op="attn", dtype="bf16", batch=32, heads=32, kv_heads=8, hd=128, prefix=2100,
             kv_lo=0, kv_hi=0, q_lo=5, q_hi=130, causal=True),
        # the fp32 path with 64-wide heads: blocks of four
        dict(name="attn_block_f32_b3_p500", op="attn", dtype="f32", batch=3, heads=4, kv_heads=2, hd=64, prefix=500,
             kv_lo=4, kv_hi=60, q_lo=4, q_hi=4, causal=True),
        # one decode row at the Qwen3 vocabulary: latency
        dict(name="logits_step_b1", op="logits", dtype="f32", batch=1, rows=1, vocab=151936, hist_lo=512, hist_hi=768,
             n_bias=16, n_masks=0),
        # a verify block of 16 rows, each behind its drafts, with a mask a row (grammar state after each draft)
        dict(name="logits_verify_b1_r16", op="logits", dtype="f32", batch=1, rows=16, vocab=151936, hist_lo=512,
             hist_hi=8448, n_bias=64, n_masks=16),
        # 64 decode rows in bf16 at the LLaMA-3.1 vocabulary
        dict(name="logits_step_b64_bf16", op="logits", dtype="bf16", batch=64, rows=1, vocab=128256, hist_lo=1,
             hist_hi=2303, n_bias=300, n_masks=9),
        # the verify pass of the concurrency-32 workload, blocks of 16
        dict(name="logits_verify_b32_r16", op="logits", dtype="f32", batch=32, rows=16, vocab=151936, hist_lo=256,
             hist_hi=2303, n_bias=32, n_masks=64),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["tables", "attn", "attn", "logits"])
    if op == "tables":
        batch = _log(rng, 1, 1024)
        new_hi = _log(rng, 1, min(2048, 16384 // batch))
        kv_hi = rng.randint(0, 8192)
        return dict(op=op, batch=batch, kv_lo=rng.randint(0, kv_hi), kv_hi=kv_hi, new_lo=rng.randint(0, new_hi),
                    new_hi=new_hi, width=(kv_hi + new_hi) // PAGE + 1 + rng.randint(0, 24), base=rng.randint(0, 8192))
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        h, hkv, hd = rng.choice(HEADS)
        q_hi = rng.choice([1, rng.randint(2, 32), _log(rng, 2, 400)])
        batch = _log(rng, 1, max(1, min(64, 2048 // q_hi)))
        prefix = _log(rng, 1, 16384)
        kv_hi = rng.choice([0, _log(rng, 1, 2048), _log(rng, 1, 2048)])
        most = 2.0e9 if dtype == "f32" else 5e10  # flops
        while 4.0 * batch * q_hi * h * hd * (prefix + kv_hi + q_hi) > most:
            prefix, kv_hi, q_hi = max(1, prefix * 3 // 4), kv_hi * 3 // 4, max(1, q_hi * 3 // 4)
        return dict(op=op, dtype=dtype, batch=batch, heads=h, kv_heads=hkv, hd=hd, prefix=prefix,
                    kv_lo=rng.randint(0, kv_hi), kv_hi=kv_hi, q_lo=rng.choice([q_hi, rng.randint(0, q_hi)]), q_hi=q_hi,
                    causal=rng.random() < 0.7)
    batch, rows, vocab = _log(rng, 1, 64), rng.choice([1, rng.randint(2, 32)]), _log(rng, 1000, 152064)
    while batch * rows > 512:
        batch, rows = max(1, batch * 3 // 4), max(1, rows * 3 // 4)
    hist_hi = _log(rng, 1, 8448)
    return dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), batch=batch, rows=rows, vocab=vocab,
                hist_lo=rng.randint(0, hist_hi), hist_hi=hist_hi, n_bias=rng.choice([0, _log(rng, 1, 512)]),
                n_masks=rng.choice([0, rng.randint(1, 64)]))


# ------------------------------------------------------------------------------------------------------- inputs
def _lens(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int64)


def _spread(g, lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], in a drawn order: their sum is the same for every seed."""
    return (lo + (hi - lo + 1) * (2 * torch.arange(n) + 1) // (2 * n))[torch.randperm(n, generator=g)]


def _ceil(a, b):
    return (a + b - 1) // b


def _i32(x):
    return x.to(torch.int32).to(DEV)


def _lengths(case, seed):
    """The host lengths of a case, the same for prepare(), exact() and the seed that they are given."""
    g = torch.Generator().manual_seed(int(seed))
    b = case["batch"]
    if case["op"] == "tables":
        return g, _lens(g, case["kv_lo"], case["kv_hi"], b), _spread(g, case["new_lo"], case["new_hi"], b)
    if case["op"] == "attn":
        q = _spread(g, case["q_lo"], case["q_hi"], b)
        kv = _lens(g, case["kv_lo"], case["kv_hi"], b) + (q if case["kv_hi"] == 0 or case["q_hi"] > 1 else 0)
        return g, kv, q
    hist = _lens(g, case["hist_lo"], case["hist_hi"], b)
    prompt = (hist.double() * torch.rand(b, generator=g, dtype=torch.float64)).long()
    return g, hist, prompt


def prepare(case, seed):
    g, a, n = _lengths(case, seed)
    d = torch.Generator(DEV).manual_seed(int(seed) + 1)
    b = case["batch"]
    if case["op"] == "tables":
        old, width = _ceil(a, PAGE), case["width"]
        n_pages = int(_ceil(a + n, PAGE).sum()) + 7
        perm = torch.randperm(n_pages, generator=g)
        table = torch.full((b, width), n_pages, dtype=torch.int64)  # unbacked entries: the scratch page
        held = torch.arange(width)[None, :] < old[:, None]
        table[held] = perm[: int(old.sum())]
        total = int(n.sum())
        i32 = dict(dtype=torch.int32, device=DEV)
        return dict(op="tables", kv=_i32(a), new=_i32(n), table=_i32(table), free=_i32(perm[int(old.sum()):]),
                    used=torch.zeros(1, **i32), scratch=n_pages, base=case["base"], rows=total,
                    out_table=torch.empty((b, width), **i32), out_used=torch.empty(1, **i32),
                    q_start=torch.empty(b + 1, **i32), row_seq=torch.empty(total, **i32),
                    row_pos=torch.empty(total, **i32), slots=torch.empty(total, dtype=torch.int64, device=DEV),
                    status=torch.empty(1, **i32))
    if case["op"] == "attn":
        dt = DTYPES[case["dtype"]]
        h, hkv, hd, pre = case["heads"], case["kv_heads"], case["hd"], case["prefix"]
        width = max(1, int(_ceil(a, PAGE).max()))
        n_pre = _ceil(pre, PAGE)
        n_pages = n_pre + int(_ceil(a, PAGE).sum()) + 1
        perm = torch.randperm(n_pages, generator=g)
        table = torch.full((b, width), int(perm[-1]), dtype=torch.int64)
        table[torch.arange(width)[None, :] < _ceil(a, PAGE)[:, None]] = perm[n_pre:-1]
        rows = max(1, int(n.sum()))
        # normed and rotated queries and keys have unit RMS a channel, values a plain spread
        q = torch.randn((rows, h, hd), generator=d, device=DEV).to(dt)
        k = torch.randn((n_pages, hkv, PAGE, hd), generator=d, device=DEV).to(dt)
        v = torch.randn((n_pages, hkv, PAGE, hd), generator=d, device=DEV).to(dt)
        start = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
        return dict(op="attn", q=q, k=k, v=v, prefix_pages=_i32(perm[:n_pre]), prefix=pre, table=_i32(table), kv=_i32(a),
                    q_start=_i32(start), max_q=max(1, int(n.max())), causal=case["causal"],
                    out=torch.zeros_like(q), lse=torch.zeros((rows, h), device=DEV))
    rows, vocab, nb, nm = case["rows"], case["vocab"], case["n_bias"], case["n_masks"]
    logits = (3.0 * torch.randn((b * rows, vocab), generator=d, device=DEV)).to(DTYPES[case["dtype"]])
    cap = max(1, int(a.max()))
    # tokens repeat as text does: ids spread over the logarithm
    ids = torch.exp(torch.rand((b, cap), generator=d, device=DEV) * torch.log(torch.tensor(float(vocab), device=DEV)))
    history = ids.to(torch.int64).clamp_(0, vocab - 1).to(torch.int32)
    drafts = torch.randint(0, vocab, (b, max(rows - 1, 1)), generator=d, device=DEV, dtype=torch.int32)
    rep = 1.0 + 0.5 * torch.rand(b, generator=d, device=DEV)
    pres = torch.rand(b, generator=d, device=DEV) - 0.25
    freq = torch.rand(b, generator=d, device=DEV) - 0.25
    bias_ids = bias = masks = mask_index = None
    if nb:
        bias_ids = torch.randint(0, vocab, (b, nb), generator=d, device=DEV)
        bias_ids = (bias_ids // nb * nb + torch.arange(nb, device=DEV))  # distinct within a request
        bias_ids = torch.where(bias_ids < vocab, bias_ids, -1).to(torch.int32)  # -1: an unused entry
        bias = 10.0 * torch.randn((b, nb), generator=d, device=DEV)
    if nm:
        # grammar states: most allow nearly everything (text) or a handful (structure)
        words = _ceil(vocab, 32)
        dens = torch.tensor([0.98, 0.001, 0.5, 0.9], device=DEV)[torch.arange(nm, device=DEV) % 4]
        bits = (torch.rand((nm, words * 32), generator=d, device=DEV) < dens[:, None]).view(nm, words, 32).long()
        packed = (bits << torch.arange(32, device=DEV)).sum(-1)
        masks = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)
        mask_index = torch.randint(-1, nm, (b * rows,), generator=d, device=DEV, dtype=torch.int32)  # -1: free text
    return dict(op="logits", logits=logits, rows=rows, history=history, hist=_i32(a), prompt=_i32(n), drafts=drafts,
                rep=rep, pres=pres, freq=freq, bias_ids=bias_ids, bias=bias, masks=masks, mask_index=mask_index,
                out=torch.empty_like(logits))


# ---------------------------------------------------------------------------------------------------- one pass
def run(state):
    return {"tables": _tables, "attn": _attn, "logits": _logits}[state["op"]](state)


def _tables(s):
    if own:
        import block_diffusion_speculative_ctx_gb300 as dfl
        t = dfl.kv_tables(s["kv"], s["new"], s["table"], s["free"], s["used"], scratch_page=s["scratch"],
                          base_pos=s["base"], table_out=s["out_table"], used_out=s["out_used"], q_start=s["q_start"],
                          row_seq=s["row_seq"], row_pos=s["row_pos"], slots=s["slots"], status=s["status"])
        return [t.table, t.used, t.q_start, t.row_seq, t.row_pos, t.slots, t.status]
    kv, new = s["kv"].long(), s["new"].long()
    b, width = s["table"].shape
    old, need = _ceil(kv, PAGE), _ceil(kv + new, PAGE)
    add = need - old
    taken = add.cumsum(0)
    col = torch.arange(width, device=DEV)
    pick = (s["used"].long() + (taken - add)[:, None] + col[None, :] - old[:, None]).clamp(0, max(s["free"].numel() - 1, 0))
    fresh = s["free"][pick] if s["free"].numel() else torch.full_like(s["table"], s["scratch"])
    table = torch.where(col[None, :] < old[:, None], s["table"],
                        torch.where(col[None, :] < need[:, None], fresh, s["scratch"]))
    q_start = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), new.cumsum(0)])
    r = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(q_start[1:], r, right=True).clamp(max=b - 1)
    i = kv[seq] + r - q_start[seq]
    slots = table[seq, i // PAGE].long() * PAGE + i % PAGE
    short = (s["used"].long() + taken[-1:] > s["free"].numel()).int()
    wide = (need > width).any().int() * 2
    return [table, (s["used"] + taken[-1:]).to(torch.int32), q_start.to(torch.int32), seq.to(torch.int32),
            (s["base"] + i).to(torch.int32), slots, (short + wide).to(torch.int32)]


def _attn(s):
    if own:
        import block_diffusion_speculative_ctx_gb300 as dfl
        out, lse = dfl.shared_prefix_attention(s["q"], s["k"], s["v"], s["prefix_pages"], s["prefix"], s["table"],
                                               s["kv"], s["q_start"], causal=s["causal"], out=s["out"],
                                               lse=s["lse"])
        return [out, lse]
    q, start, kv = s["q"].float(), s["q_start"].long(), s["kv"].long()
    rows, h, hd = q.shape
    hkv = s["k"].shape[1]
    g, b, pre = h // hkv, kv.numel(), s["prefix"]
    scale = hd ** -0.5
    # row r is row j of sequence seq; rows padded to [batch, max_q]
    r = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(start[1:], r, right=True).clamp(max=b - 1)
    j, m = r - start[seq], (start[1:] - start[:-1])
    pad = (start[:-1, None] + torch.arange(s["max_q"], device=DEV)).clamp(max=rows - 1)
    lim = (kv[seq] - m[seq] + j + 1 if s["causal"] else kv[seq]).clamp(min=0)
    # the prefix: every row of a KV head's query group against the same keys
    kp = s["k"][s["prefix_pages"].long()].transpose(0, 1).reshape(hkv, -1, hd)[:, :pre].float()
    vp = s["v"][s["prefix_pages"].long()].transpose(0, 1).reshape(hkv, -1, hd)[:, :pre].float()
    qg = q.view(rows, hkv, g, hd)
    sp = (qg.permute(1, 0, 2, 3).reshape(hkv, rows * g, hd) @ kp.transpose(1, 2)).mul_(scale)
    sp = sp.view(hkv, rows, g, pre)
    # each sequence's own keys
    kq = s["k"][s["table"].long()].transpose(1, 2).reshape(b, hkv, -1, hd).float()
    vq = s["v"][s["table"].long()].transpose(1, 2).reshape(b, hkv, -1, hd).float()
    keys = kq.shape[2]
    qb = qg[pad].permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, hd)
    sq = (qb @ kq.transpose(2, 3)).mul_(scale).view(b, hkv, s["max_q"], g, keys)[seq, :, j].transpose(0, 1)
    sq = sq.masked_fill(torch.arange(keys, device=DEV) >= lim[None, :, None, None], float("-inf"))
    top = torch.maximum(sp.amax(-1), sq.amax(-1))
    top0 = torch.where(torch.isinf(top), torch.zeros_like(top), top)[..., None]
    pp, pq = (sp - top0).exp(), (sq - top0).exp()
    den = pp.sum(-1) + pq.sum(-1)
    op = (pp.view(hkv, rows * g, pre) @ vp).view(hkv, rows, g, hd)
    wide = torch.zeros((b, s["max_q"], hkv, g, keys), device=DEV)
    wide[seq, j] = pq.transpose(0, 1)
    oq = (wide.permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, keys) @ vq).view(b, hkv, s["max_q"], g, hd)[seq, :, j]
    out = (op.transpose(0, 1) + oq) / den.transpose(0, 1)[..., None].clamp(min=1e-30)
    lse = (top + den.log()).transpose(0, 1).reshape(rows, h)
    live = r < start[-1]
    return [torch.where(live[:, None, None], out.reshape(rows, h, hd), 0.0).to(s["q"].dtype),
            torch.where(live[:, None], lse, 0.0)]


def _logits(s):
    if own:
        import block_diffusion_speculative_ctx_gb300 as dfl
        return dfl.process_logits(s["logits"], rows_per_seq=s["rows"], history=s["history"], hist_lens=s["hist"],
                                  prompt_lens=s["prompt"], drafts=s["drafts"] if s["rows"] > 1 else None,
                                  repetition=s["rep"], presence=s["pres"], frequency=s["freq"],
                                  bias_ids=s["bias_ids"], bias_values=s["bias"], masks=s["masks"],
                                  mask_index=s["mask_index"], out=s["out"])
    x = s["logits"].float()
    n, vocab = x.shape
    rows = s["rows"]
    b = n // rows
    at = torch.arange(s["history"].shape[1], device=DEV)[None, :]
    tok = s["history"].long()
    said = ((at >= s["prompt"][:, None]) & (at < s["hist"][:, None])).float()
    count = torch.zeros((b, vocab), device=DEV).scatter_add_(1, tok, said)
    seen = torch.zeros((b, vocab), device=DEV).scatter_add_(1, tok, (at < s["hist"][:, None]).float())
    if rows > 1:  # row j also follows the first j drafts
        step = torch.zeros((b, rows, vocab), device=DEV)
        step[:, 1:].scatter_(2, s["drafts"].long()[:, :, None], 1.0)
        step = step.cumsum(1)
        count, seen = (count[:, None] + step).view(n, vocab), (seen[:, None] + step).view(n, vocab)
    rep = s["rep"].repeat_interleave(rows)[:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"].repeat_interleave(rows)[:, None] * count
    x = x - s["pres"].repeat_interleave(rows)[:, None] * (count > 0)
    if s["bias"] is not None:
        add = torch.zeros((b, vocab + 1), device=DEV)
        add.scatter_(1, torch.where(s["bias_ids"] < 0, vocab, s["bias_ids"]).long(), s["bias"])
        x = x + add[:, :vocab].repeat_interleave(rows, 0)
    if s["masks"] is not None:
        v = torch.arange(vocab, device=DEV)
        bits = (s["masks"][:, v // 32] >> (v % 32).to(torch.int32)) & 1
        i = s["mask_index"].long()
        x = x.masked_fill((bits[i.clamp(min=0)] == 0) & (i >= 0)[:, None], float("-inf"))
    return x.to(s["logits"].dtype)


# ------------------------------------------------------------------------------------------------- 64-bit answers
def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    _, a, n = _lengths(case, seed)
    if case["op"] == "attn":
        q = s["q"].double()
        rows, h, hd = q.shape
        out, lse = torch.zeros_like(q), torch.zeros((rows, h), dtype=torch.float64, device=DEV)
        start = 0
        for i in range(case["batch"]):
            m, own_keys = int(n[i]), int(a[i])
            if m == 0:
                continue
            pages = [s["prefix_pages"].long(), s["table"][i, : _ceil(own_keys, PAGE)].long()]
            keep = [case["prefix"], own_keys]
            k = torch.cat([s["k"][p].transpose(0, 1).flatten(1, 2)[:, :c] for p, c in zip(pages, keep)], 1).double()
            v = torch.cat([s["v"][p].transpose(0, 1).flatten(1, 2)[:, :c] for p, c in zip(pages, keep)], 1).double()
            k, v = (t.repeat_interleave(h // t.shape[0], 0) for t in (k, v))  # one copy a query head
            z = torch.einsum("rhd,hkd->hrk", q[start:start + m], k) / hd ** 0.5
            if case["causal"]:
                last = case["prefix"] + own_keys - m + torch.arange(m, device=DEV)
                z.masked_fill_(torch.arange(k.shape[1], device=DEV)[None, :] > last[:, None], float("-inf"))
            lse[start:start + m] = torch.logsumexp(z, -1).T
            out[start:start + m] = torch.einsum("hrk,hkd->rhd", torch.softmax(z, -1), v)
            start += m
        return [out, lse]
    x = s["logits"].double()
    vocab, rows = case["vocab"], case["rows"]
    for i in range(case["batch"]):
        count = torch.bincount(s["history"][i, int(n[i]): int(a[i])].long(), minlength=vocab).double()
        seen = torch.bincount(s["history"][i, : int(a[i])].long(), minlength=vocab) > 0
        rep, pres, freq = (s[k][i].double() for k in ("rep", "pres", "freq"))
        for j in range(rows):
            if j:
                count[int(s["drafts"][i, j - 1])] += 1
                seen[int(s["drafts"][i, j - 1])] = True
            z = x[i * rows + j]
            z = torch.where(seen & (z > 0), z / rep, torch.where(seen, z * rep, z))
            z = z - freq * count - pres * (count > 0).double()
            if s["bias"] is not None:
                used = s["bias_ids"][i] >= 0
                z[s["bias_ids"][i][used].long()] += s["bias"][i][used].double()
            if s["masks"] is not None and int(s["mask_index"][i * rows + j]) >= 0:
                word = s["masks"][int(s["mask_index"][i * rows + j])]
                bit = (word[:, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
                z[bit.flatten()[:vocab] == 0] = float("-inf")
            x[i * rows + j] = z
    return x


def work(case):
    """Each input read once and each output written once; lengths that are drawn count at their mean."""
    b = case["batch"]
    if case["op"] == "tables":
        rows = b * (case["new_lo"] + case["new_hi"]) / 2
        return {"bytes": b * case["width"] * 8 + rows * 16 + b * 12 + rows / PAGE * 4, "flops": 0}
    if case["op"] == "attn":
        e = 2 if case["dtype"] == "bf16" else 4
        q = (case["q_lo"] + case["q_hi"]) / 2
        kv = (case["kv_lo"] + case["kv_hi"]) / 2 + (q if case["kv_hi"] == 0 or case["q_hi"] > 1 else 0)
        rows, h, hd = b * q, case["heads"], case["hd"]
        seen = kv - (q - 1) / 2 if case["causal"] else kv
        return {"bytes": 2 * e * hd * (case["kv_heads"] * (case["prefix"] + b * kv) + rows * h) + 4 * rows * h,
                "flops": 4 * rows * h * hd * (case["prefix"] + seen)}
    e = 2 if case["dtype"] == "bf16" else 4
    n, vocab = b * case["rows"], case["vocab"]
    return {"bytes": 2 * e * n * vocab + b * (2 * (case["hist_lo"] + case["hist_hi"]) + 8 * case["n_bias"])
            + min(n, case["n_masks"]) * vocab / 8, "flops": 0}
