"""The operators of trees of drafted tokens and of shared pages on the GPU against their fp64 oracles, at the sizes, masks
and faults where they can go wrong."""
import numpy as np
import pytest
import torch

from oracle import trees

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # largest relative error of one rounding


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_ctx_gb300 import build
    build.build()


def dfl():
    import block_diffusion_speculative_ctx_gb300 as m
    return m


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def host(t):
    return t.cpu().numpy()


def random_tree(rng, m, chain=0.3):
    """Parents of m nodes: a chain's next link with some probability, any earlier node otherwise."""
    return np.array([-1] + [j - 1 if rng.random() < chain else rng.integers(0, j) for j in range(1, m)], int)[:m]


def starts(m):
    return np.concatenate([[0], np.cumsum(m)])


# --------------------------------------------------------------------------------------------------------- masks
@pytest.mark.parametrize("sizes,chain", [([1], 0), ([0, 3, 0], .5), ([32, 33, 31], .3), ([64, 65, 1, 0], .9), ([1024], 1.0),
                                         ([1000, 24], 0.0), ([7] * 2048, .5)])
def test_tree_masks(sizes, chain):
    rng = np.random.default_rng(sum(sizes))
    forest = [random_tree(rng, m, chain) for m in sizes]
    words = max(1, -(-max(sizes) // 32)) + 1
    kv = rng.integers(0, 5000, len(sizes)) + np.array(sizes)
    t = dfl().tree_masks(i32(np.concatenate(forest)), i32(starts(sizes)), kv_lens=i32(kv), base_pos=17, words=words)
    assert (host(t.status) == 0).all()
    got = [host(x) for x in (t.masks, t.depth, t.row_pos)]
    for s, p in enumerate(forest):
        at = slice(*starts(sizes)[s:s + 2])
        sees, depth = trees.ancestors(p)
        np.testing.assert_array_equal(got[0][at], trees.words(sees, words))
        np.testing.assert_array_equal(got[1][at], depth)
        np.testing.assert_array_equal(got[2][at], 17 + kv[s] - len(p) + depth)


def test_tree_masks_forests_strides_and_rows_of_no_tree():
    """Several roots; masks a slice of a wider matrix; rows before the first tree and behind the last keep what they held."""
    p = np.array([9, 9, -1, 0, -1, 2, 1, -1, 9])
    wide = torch.full((9, 5), 77, dtype=torch.int32, device="cuda")
    depth = torch.full((9,), 66, dtype=torch.int32, device="cuda")
    t = dfl().tree_masks(i32(p), i32([2, 7, 8]), masks=wide[:, 1:3], depth=depth)
    sees, d = trees.ancestors(p[2:7])
    want = np.full((9, 5), 77)
    want[2:7, 1:3], want[7, 1:3] = trees.words(sees, 2), [1, 0]
    np.testing.assert_array_equal(host(wide), want)
    np.testing.assert_array_equal(host(t.depth), [66, 66, *d, 0, 66])
    assert t.row_pos is None


@pytest.mark.parametrize("fault,status", [("forward", 1), ("self", 1), ("below", 1), ("wide", 2), ("many", 2), ("falls", 4), ("rows", 4)])
def test_tree_masks_and_acceptance_report_bad_trees(fault, status):
    """One bad sequence of three: its rows say so, the others are what they are."""
    m = [5, 40 if fault != "many" else 1025, 6]
    rng = np.random.default_rng(1)
    forest = [random_tree(rng, n) for n in m]
    start, words = starts(m), 1 if fault == "wide" else 33
    if fault == "forward":
        forest[1][3] = 4
    elif fault == "self":
        forest[1][0] = 0
    elif fault == "below":
        forest[1][7] = -2
    par, rows = np.concatenate(forest), int(sum(m))
    if fault == "falls":
        start[1] = start[2] + 1
    elif fault == "rows":
        start[2:] = [rows + 1, rows + 1]
    masks, depth = torch.full((rows, words), 3, dtype=torch.int32, device="cuda"), torch.full((rows,), 3, dtype=torch.int32, device="cuda")
    t = dfl().tree_masks(i32(par), i32(start), masks=masks, depth=depth, kv_lens=i32([50, 2000, 60]))
    got = host(t.status)
    assert got[1] == status
    a = dfl().tree_accept(i32(par), i32(np.zeros(rows)), i32(np.zeros(rows)), i32(start), width=4)
    if fault != "wide":  # (acceptance has no words)
        assert host(a.status)[1] == status and host(a.accepted)[1] == host(a.bonus)[1] == -1 and (host(a.path)[1] == -1).all()
    if status != 4:
        at = slice(start[1], start[2])
        assert (host(t.masks)[at] == 0).all() and (host(t.depth)[at] == -1).all() and (host(t.row_pos)[at] == -1).all()
        for s in (0, 2):
            assert got[s] == 0 and host(a.status)[s] == 0
            sees, d = trees.ancestors(forest[s])
            np.testing.assert_array_equal(host(t.masks)[start[s]:start[s + 1]], trees.words(sees, words))
    elif fault == "falls":
        assert got[0] == 0 and got[2] == 0  # (their rows are what their own starts say)
    else:
        assert got[0] == 0 and got[2] == 4 and (host(t.masks)[start[1]:] == 3).all() and (host(t.depth)[start[1]:] == 3).all()


# ----------------------------------------------------------------------------------------------------- attention
def attn_case(dtype, heads, prefix, own, m, seed, stale=np.nan, random_masks=False, q_scale=1.0):
    """Slots behind the last key of a list hold `stale`; own keys are own[s] committed ones and the m[s] nodes."""
    H, hkv, hd = heads
    g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    m = np.asarray(m)
    kv = np.asarray(own) + m
    n_pre, npg = -(-prefix // 64), -(-kv // 64)
    n_pages = n_pre + int(npg.sum()) + 2
    perm = rng.permutation(n_pages)
    table = np.full((len(kv), max(1, int(npg.max()) + 1)), -1)  # entries past a sequence's pages are never read
    k, v = (torch.randn((n_pages, hkv, 64, hd), generator=g).to(DT[dtype]).float().numpy() for _ in range(2))
    live = np.zeros((n_pages, 64), bool)

    def fill(pages, n):
        for i, p in enumerate(pages):
            live[p, :min(64, n - 64 * i)] = True

    fill(perm[:n_pre], prefix)
    at = n_pre
    for s in range(len(kv)):
        table[s, :npg[s]] = perm[at:at + npg[s]]
        fill(table[s, :npg[s]], int(kv[s]))
        at += npg[s]
    for c in (k, v):
        c[~live[:, None, :].repeat(hkv, 1)] = stale
    words = max(1, -(-int(m.max()) // 32))
    sees = [rng.random((n, n)) < 0.4 if random_masks else trees.ancestors(random_tree(rng, n))[0] for n in m]
    q = (q_scale * torch.randn((int(m.sum()), H, hd), generator=g)).to(DT[dtype]).float().numpy()
    return dict(q=q, k=k, v=v, pre=perm[:n_pre], prefix=prefix, table=table, kv=kv, start=starts(m), sees=sees, dtype=dtype,
                hd=hd, masks=np.concatenate([trees.words(x, words) for x in sees]))


def attn_run(c, **kw):
    dt = DT[c["dtype"]]
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dt).cuda()  # noqa: E731
    x = [up(c["q"]), up(c["k"]), up(c["v"]), i32(c["table"]), i32(c["kv"]), i32(c["start"]), i32(c["masks"])]
    if c["prefix"]:
        kw = dict(prefix_pages=i32(c["pre"]), prefix_len=c["prefix"], **kw)
    return x, kw


def attn_check(c, got, scale=None, rows=slice(None), weight_step=None):
    """Error bounds.  u = 2^-24.  A score is a sum of hd products in fp32, off by at most hd u sum|q_i k_i| scale =: z;
    each softmax weight is then off by a factor of at most exp(2 z) and by the rounding of the exponent's argument,
    |score| u log2(e), plus exp2 itself (2^-22) and the n-term sums (n u).  In bf16 each weight is also rounded once
    (half a step, 2^-8; held as a pair, half a step of half a step).  The output is rounded once to its type."""
    scale = c["hd"] ** -0.5 if scale is None else scale
    out, lse, weight = (x[rows] for x in trees.tree_attention(c["q"], c["k"], c["v"], c["pre"], c["prefix"], c["table"], c["kv"],
                                                              c["start"], c["sees"], scale))
    u, n = 2.0 ** -24, c["prefix"] + int(c["kv"].max())
    kmax = np.abs(np.where(np.isfinite(c["k"]), c["k"], 0)).sum(-1).max()
    qk = scale * float(np.abs(c["q"]).max()) * kmax if c["q"].size else 0.0  # >= sum|q_i k_i| scale
    z = c["hd"] * u * qk
    delta = 2 * z + 4 * qk * u + 2.0 ** -22 + (n + 64) * u
    if weight_step is None:
        weight_step = 2.0 ** -8 if c["dtype"] == "bf16" else 0.0
    tol = HALF[c["dtype"]] * np.abs(out) + (delta + weight_step) * weight + 1e-30
    g, gl = host(got[0].float()).astype(np.float64), host(got[1])
    assert np.isfinite(g).all()
    bad = np.abs(g - out) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(g - out) / tol).max()), np.argwhere(bad)[:4])
    inf = np.isneginf(lse)
    assert (np.isneginf(gl) == inf).all()
    ltol = z + 4 * qk * u + (n + 64) * u + 2.0 ** -21 + np.abs(np.where(inf, 0, lse)) * 2.0 ** -22
    assert (np.abs(np.where(inf, 0, gl) - np.where(inf, 0, lse)) <= ltol).all()


ATTN = [
    # heads (H, H_kv, hd), prefix, committed own keys, nodes
    ((8, 2, 128), 0, [0], [1]),
    ((8, 2, 128), 0, [100], [1]),                          # a single token
    ((8, 2, 128), 70, [0, 64, 63, 1], [1, 1, 2, 0]),
    ((32, 8, 128), 0, [512], [16]),
    ((32, 8, 128), 500, [48, 47, 49, 130], [16, 16, 16, 16]),   # trees that end on, before and behind a page's end
    ((8, 2, 128), 129, [31, 32, 33], [33, 64, 32]),
    ((32, 8, 128), 1000, [300, 0, 77], [64, 64, 61]),           # both streams
    ((4, 1, 128), 0, [20, 5], [100, 129]),
    ((4, 2, 64), 333, [10, 64, 65], [9, 9, 9]),
    ((16, 8, 64), 64, [200, 33], [80, 9]),
    ((8, 8, 128), 40, [65, 1], [33, 140]),                      # one query head a KV head
    ((6, 2, 128), 257, [50, 80], [45, 44]),
    ((14, 2, 128), 19, [30, 20], [20, 37]),
    ((64, 1, 128), 0, [9, 3], [9, 3]),
    ((2, 1, 64), 0, [10], [300]),
]


@pytest.mark.parametrize("random_masks", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(ATTN)))
def test_tree_attention(i, dtype, random_masks):
    """Trees, and masks of any sets (some of them empty)."""
    c = attn_case(dtype, *ATTN[i], seed=300 + i, random_masks=random_masks)
    x, kw = attn_run(c)
    attn_check(c, dfl().tree_attention(*x, **kw))


@pytest.mark.parametrize("i", [3, 5, 6, 9])
def test_tree_attention_weight_pairs(i):
    c = attn_case("bf16", *ATTN[i], seed=400 + i)
    x, kw = attn_run(c)
    attn_check(c, dfl().tree_attention(*x, weight_pairs=True, **kw), weight_step=2.0 ** -16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_attention_of_a_chain_is_the_causal_one(dtype):
    """A chain's masks say what the causal rule says: the same products in the same order, the same bits."""
    c = attn_case(dtype, (8, 2, 128), 200, [77, 0, 130], [40, 70, 1], seed=9)
    chain = [np.arange(-1, n - 1) for n in (40, 70, 1)]
    t = dfl().tree_masks(i32(np.concatenate(chain)), i32(c["start"]), words=3)
    x, kw = attn_run(c)
    got = dfl().tree_attention(*x[:6], t.masks, **kw)
    want = dfl().shared_prefix_attention(*x[:3], kw["prefix_pages"], 200, *x[3:6], causal=True)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [12, 70])
def test_tree_attention_ignores_what_no_row_sees(dtype, m):
    """Empty rows give 0 and -inf; nodes that no row sees (a padded tree's) may hold NaN or infinities."""
    c = attn_case(dtype, (8, 2, 128), 0, [0, 90], [m, m], seed=5, random_masks=True)
    for s in range(2):
        c["sees"][s][[0, m // 2, m - 1]] = False
        c["sees"][s][:, [0, 3, m - 2, m - 1]] = False
        for n, i in enumerate((0, 3, m - 2, m - 1)):
            at = c["kv"][s] - m + i
            c["k"][c["table"][s, at // 64], :, at % 64] = (np.nan, np.inf, -np.inf, np.nan)[n]
            c["v"][c["table"][s, at // 64], :, at % 64] = (np.inf, np.nan, -np.inf, np.nan)[n]
    words = c["masks"].shape[1]
    c["masks"] = np.concatenate([trees.words(x, words) for x in c["sees"]])
    x, kw = attn_run(c)
    got = dfl().tree_attention(*x, **kw)
    attn_check(c, got)
    assert (host(got[0].float())[0] == 0).all() and np.isneginf(host(got[1])[0]).all()


def test_tree_attention_words_bits_and_lengths_at_their_edges():
    """Bits of nodes that are not there count for nothing, nodes behind the last word are not seen, and of a tree with more
    nodes than own keys the first ones have none."""
    c = attn_case("bf16", (8, 2, 128), 64, [10, 0, 30], [40, 5, 6], seed=6, random_masks=True)
    x, kw = attn_run(c)
    want = dfl().tree_attention(*x, **kw)
    more = x[6].clone()
    for s, n in enumerate((40, 5, 6)):
        at = slice(c["start"][s], c["start"][s + 1])
        if n < 32:
            more[at, 0] |= -1 << n
        more[at, 1] |= -1 << max(n - 32, 0)
    got = dfl().tree_attention(*x[:6], more, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c["sees"][0][:, 32:] = False
    attn_check(c, dfl().tree_attention(*x[:6], more[:, :1], **kw))
    c = attn_case("bf16", (8, 2, 128), 64, [0], [9], seed=7, random_masks=True)
    c["kv"][:] = 4  # nodes 5 .. 8 are keys 0 .. 3
    x, kw = attn_run(c)
    attn_check(c, dfl().tree_attention(*x, **kw))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_attention_strides_and_rows_behind(dtype):
    c = attn_case(dtype, (8, 2, 128), 150, [70, 20], [2, 3], seed=21)
    x, kw = attn_run(c)
    fused = torch.full((9, 12, 128), 7.0, dtype=x[0].dtype, device="cuda")
    fused[2:7, :8] = x[0]
    out = torch.full((9, 16, 128), 5.0, dtype=x[0].dtype, device="cuda")
    lse = torch.full((9, 8), 5.0, device="cuda")
    wide = torch.cat([torch.full((2, 3), -9, dtype=torch.int32, device="cuda"), x[3]], 1)
    masks = torch.full((9, 4), -1, dtype=torch.int32, device="cuda")
    masks[2:7, 2:3] = x[6]
    o, l = dfl().tree_attention(fused[:, :8], x[1], x[2], wide[:, 3:], x[4], x[5] + 2, masks[:, 2:3], out=out[:, :8], lse=lse, **kw)
    attn_check(c, (o[2:7], l[2:7]))
    keep = torch.tensor([0, 1, 7, 8])
    assert (out[keep] == 5.0).all() and (lse[keep] == 5.0).all() and (out[:, 8:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_attention_reports_bad_pages_and_lengths_as_nan(dtype):
    c = attn_case(dtype, (8, 2, 128), 0, [100, 100, 100], [8, 8, 8], seed=22)
    x, kw = attn_run(c)
    x[3] = x[3].clone()
    x[3][0, 1] = c["k"].shape[0]
    x[4] = torch.tensor([108, 108, 64 * x[3].shape[1] + 1], dtype=torch.int32, device="cuda")
    out, lse = dfl().tree_attention(*x)
    for s in (0, 2):
        assert torch.isnan(out[8 * s:8 * s + 8]).all() and torch.isnan(lse[8 * s:8 * s + 8]).all()
    attn_check(c, (out[8:16], lse[8:16]), rows=slice(8, 16))


# ------------------------------------------------------------------------------------- acceptance and compaction
def forest_case(rng, sizes, vocab):
    forest = [random_tree(rng, m) for m in sizes]
    tokens = [rng.integers(0, vocab, m) for m in sizes]
    post = [rng.integers(0, vocab, m) for m in sizes]
    for p, t, o in zip(forest, tokens, post):  # the target often agrees with some child
        for j in range(1, len(p)):
            if rng.random() < 0.5:
                o[p[j]] = t[j]
    return forest, tokens, post


@pytest.mark.parametrize("sizes,vocab,width", [([1], 5, 1), ([0, 4, 0, 1], 3, 3), ([64, 33, 16], 4, 32), ([1024, 7], 3, 1024),
                                               ([1024], 2, 8), ([9] * 2048, 4, 9)])
def test_tree_accept(sizes, vocab, width):
    """Few distinct tokens: children that share one, and paths that the width ends."""
    forest, tokens, post = forest_case(np.random.default_rng(len(sizes) + width), sizes, vocab)
    a = dfl().tree_accept(*(i32(np.concatenate(x)) for x in (forest, tokens, post)), i32(starts(sizes)), width=width)
    want = [trees.tree_accept(*x, width) for x in zip(forest, tokens, post)]
    np.testing.assert_array_equal(host(a.path), [w[0] for w in want])
    np.testing.assert_array_equal(host(a.accepted), [w[1] for w in want])
    np.testing.assert_array_equal(host(a.bonus), [w[2] for w in want])
    assert (host(a.status) == 0).all()


def test_tree_accept_does_not_leave_the_root():
    """Other roots are no children of the first, whatever they hold."""
    a = dfl().tree_accept(i32([-1, -1, 1]), i32([5, 6, 6]), i32([6, 6, 6]), i32([0, 3]), width=3)
    assert host(a.path).tolist() == [[0, -1, -1]] and int(a.accepted) == 0 and int(a.bonus) == 6


def cache_case(rng, dtype, layers, hkv, hd, kv, slack=2, stride=0):
    """Two caches whose layers are `stride` elements further apart than they need, and a table."""
    used = -(-np.asarray(kv) // 64)
    n = int(used.sum()) + slack
    perm = rng.permutation(n)
    table, at = np.full((len(kv), int(used.max()) + 1), n - 1), 0
    for s, u in enumerate(used):
        table[s, :u] = perm[at:at + u]
        at += u
    size = n * hkv * 64 * hd
    caches = []
    for i in range(2):
        store = torch.randn(layers * (size + stride), generator=torch.Generator().manual_seed(i + n)).to(DT[dtype]).cuda()
        caches.append(store.as_strided((layers, n, hkv, 64, hd), (size + stride, hkv * 64 * hd, 64 * hd, hd, 1)))
    return caches, table, perm[at:]


@pytest.mark.parametrize("dtype,layers,hkv,hd,stride", [("bf16", 3, 8, 128, 64), ("f32", 1, 2, 64, 0), ("bf16", 2, 3, 8, 8), ("f32", 2, 5, 100, 0)])
def test_kv_compact(dtype, layers, hkv, hd, stride):
    rng = np.random.default_rng(3)
    m, own = [1, 64, 30, 0, 200, 5], [0, 20, 62, 64, 3, 123]
    kv = np.array(m) + np.array(own)
    (k, v), table, _ = cache_case(rng, dtype, layers, hkv, hd, kv, stride=stride)
    width = 40
    path = np.full((6, width), -1)
    accepted = np.array([0, 21, 29, -1, 39, 2])
    for s in range(6):
        path[s, :accepted[s] + 1] = np.sort(rng.choice(m[s], accepted[s] + 1, replace=False))
    path[2, :30] = np.arange(30)                    # nothing moves
    path[5, :3] = [0, 1, 4]                         # the first ones are in place
    want = [trees.kv_compact(host(c.float()), table, kv, starts(m), path, accepted) for c in (k, v)]
    outside = [c.as_strided((c.stride(0) * layers,), (1,)).clone() for c in (k, v)]
    got = dfl().kv_compact(k, v, i32(table), i32(kv), i32(starts(m)), i32(path), i32(accepted))
    for c, w, o in zip((k, v), want, outside):
        np.testing.assert_array_equal(host(c.float()), w[0])
        if stride:
            now = c.as_strided((layers, c.stride(0)), (c.stride(0), 1))[:, -stride:]
            assert torch.equal(now, o.view(layers, -1)[:, -stride:])
    assert host(got.kv_lens).tolist() == want[0][1] and (host(got.status) == 0).all()


@pytest.mark.parametrize("fault,status", [("falls", 1), ("twice", 1), ("outside", 1), ("negative", 1), ("wide", 1), ("start", 4),
                                          ("short", 8), ("long", 8), ("page", 16)])
def test_kv_compact_leaves_what_it_cannot_read(fault, status):
    rng = np.random.default_rng(4)
    m, kv = [10, 10], np.array([70, 75])
    (k, v), table, _ = cache_case(rng, "bf16", 2, 2, 64, kv)
    path, accepted, start = np.array([[0, 2, 5, -1], [0, 4, 9, -1]]), np.array([2, 2]), starts(m)
    if fault in ("falls", "twice", "outside", "negative"):
        path[1, 2] = {"falls": 3, "twice": 4, "outside": 10, "negative": -1}[fault]
    elif fault == "wide":
        accepted[1] = 4
    elif fault == "start":
        start = np.array([0, 10, 9])
    elif fault == "short":
        kv[1] = 9
    elif fault == "long":
        kv[1] = 64 * table.shape[1] + 1
    else:
        table[1, 1] = k.shape[1]
    before = [host(c.float()) for c in (k, v)]
    want = [trees.kv_compact(c, table[:1], kv[:1], start[:2], path[:1], accepted[:1])[0] for c in before]
    got = dfl().kv_compact(k, v, i32(table), i32(kv), i32(start), i32(path), i32(accepted))
    assert host(got.status).tolist() == [0, status] and host(got.kv_lens).tolist() == [63, kv[1]]
    for c, w in zip((k, v), want):
        np.testing.assert_array_equal(host(c.float()), w)


# -------------------------------------------------------------------------------------------------- shared pages
def fork_state(rng, kv, dtype="bf16", layers=2, hkv=2, hd=64, free=40):
    (k, v), table, spare = cache_case(rng, dtype, layers, hkv, hd, kv, slack=free + 1)
    scratch = k.shape[1] - 1
    return dict(k=k, v=v, table=table, spare=spare[spare != scratch], refs=np.zeros(scratch + 1, int), scratch=scratch)


@pytest.mark.parametrize("dtype,kv,parents,layers,hkv,hd", [
    ("bf16", [0], [0], 1, 1, 64), ("bf16", [64], [0, 0], 1, 1, 64), ("f32", [65], [0] * 5, 2, 2, 64),
    ("bf16", [700, 63, 128, 1], [3, 0, 0, 2, 1, 3, 0], 3, 8, 128), ("f32", [200, 10], [1, 0], 1, 3, 4)])
def test_kv_fork_and_release(dtype, kv, parents, layers, hkv, hd):
    rng = np.random.default_rng(len(parents))
    f = fork_state(rng, kv, dtype, layers, hkv, hd)
    free = f["spare"]
    want = trees.kv_fork(parents, kv, f["table"], free, 3, f["refs"], [host(c.float()) for c in (f["k"], f["v"])], f["scratch"])
    fl, used, refs, table = i32(free), i32([3]), i32(f["refs"]), i32(f["table"])
    got = dfl().kv_fork(i32(parents), i32(kv), table, fl, used, refs, f["k"], f["v"], scratch_page=f["scratch"], used_out=used)
    assert int(got.status) == 0 and int(got.used) == want[2]
    np.testing.assert_array_equal(host(got.table), want[0])
    np.testing.assert_array_equal(host(got.kv_lens), want[1])
    np.testing.assert_array_equal(host(refs), want[3])
    for c, w in zip((f["k"], f["v"]), want[4]):
        np.testing.assert_array_equal(host(c.float()), w)
    # every second child leaves, then its siblings
    n = len(parents)
    for seqs in (list(range(0, n, 2)), list(range(1, n, 2))):
        if not seqs:
            continue
        w = trees.kv_release(seqs, host(got.kv_lens), host(got.table), host(fl), int(used), host(refs))
        r = dfl().kv_release(i32(seqs), got.kv_lens, got.table, fl, used, refs, used_out=used)
        assert int(r.status) == w[3] == 0 and int(r.used) == w[1]
        np.testing.assert_array_equal(host(fl), w[0])
        np.testing.assert_array_equal(host(refs), w[2])
    assert int(used) == 3 and sorted(host(fl)) == sorted(free) and (host(refs) == 0).all()


@pytest.mark.parametrize("n,width,batch", [(1, 700, 1), (40, 300, 40), (2048, 9, 2048), (600, 30, 700)])
def test_kv_release_in_the_order_of_mention(n, width, batch):
    """Pages shared at random, many at once (clusters of one to eight CTAs): the list and the counts."""
    rng = np.random.default_rng(n)
    kv = rng.integers(0, 64 * width + 1, batch)
    pages = -(-kv // 64)
    total = int(pages.sum())
    n_pages = total + 5
    table = np.full((batch, width), -5)
    perm, at = rng.permutation(n_pages), 0
    refs = np.zeros(n_pages, int)
    for s in range(batch):
        table[s, :pages[s]] = perm[at:at + pages[s]]
        at += pages[s]
        share = min(int(rng.integers(0, 4)), pages[s], pages[s - 1]) if s else 0
        for j in range(share):  # its first pages are the ones of the sequence before
            if table[s - 1, j] not in table[s]:
                table[s, j] = table[s - 1, j]
                refs[table[s, j]] += 1
    seqs = rng.permutation(batch)[:n]
    held = np.unique(np.concatenate([table[s, :pages[s]] for s in range(batch)] + [[]])).astype(int)
    free = rng.permutation(n_pages)
    used = len(held) + 1
    want = release_of(seqs, kv, table, free, used, refs)
    fl, u, rf, st = i32(free), i32([used]), i32(refs), i32(table)
    r = dfl().kv_release(i32(seqs), i32(kv), st, fl, u, rf)
    assert int(r.status) == 0 and int(r.used) == want[1] and int(u) == used
    np.testing.assert_array_equal(host(fl), want[0])
    np.testing.assert_array_equal(host(rf), want[2])


def release_of(seqs, kv, table, free, used, refs):
    """trees.kv_release without its quadratic count (valid inputs)."""
    names = np.concatenate([table[s, : -(-int(kv[s]) // 64)] for s in seqs] + [[]]).astype(int)
    count = np.bincount(names, minlength=len(refs))
    assert (count <= refs + 1).all()
    _, first = np.unique(names, return_index=True)
    gone = [p for p in names[np.sort(first)] if count[p] == refs[p] + 1]
    free, left = free.copy(), np.maximum(refs - count, 0)
    free[used - len(gone):used] = gone
    return free, used - len(gone), left


@pytest.mark.parametrize("fault,status", [("pool", 1), ("width", 2), ("negative", 8), ("parent", 8), ("used", 8)])
def test_kv_fork_takes_nothing_when_it_cannot(fault, status):
    rng = np.random.default_rng(7)
    kv, parents, used = [100, 200, 65], [0, 1, 2, 0], 2
    f = fork_state(rng, kv)
    free, table = f["spare"], f["table"]
    if fault == "pool":
        free = free[:5]
    elif fault == "width":
        table = table[:, :3]
    elif fault == "negative":
        kv = [100, -1, 65]
    elif fault == "parent":
        parents = [0, 3, 2, 0]
    else:
        used = -1
    refs, out = i32(f["refs"]), torch.full((4, table.shape[1]), 99, dtype=torch.int32, device="cuda")
    before = [f["k"].clone(), f["v"].clone()]
    got = dfl().kv_fork(i32(parents), i32(kv), i32(table), i32(free), i32([used]), refs, f["k"], f["v"], table_out=out)
    assert int(got.status) == status and int(got.used) == used and (host(got.kv_lens) == 0).all()
    assert (host(out) == 99).all() and (host(refs) == 0).all()
    assert torch.equal(before[0], f["k"]) and torch.equal(before[1], f["v"])


def test_kv_fork_leaves_bad_pages_out():
    rng = np.random.default_rng(8)
    kv, parents = [130, 200], [0, 1]
    f = fork_state(rng, kv)
    table = f["table"].copy()
    table[0, 1], table[1, 3] = -1, f["k"].shape[1]  # a shared one, and one that ends inside
    before = [f["k"].clone(), f["v"].clone()]
    refs = i32(f["refs"])
    got = dfl().kv_fork(i32(parents), i32(kv), i32(table), i32(f["spare"]), i32([0]), refs, f["k"], f["v"])
    assert int(got.status) == 16 and int(got.used) == 2
    want = np.zeros(len(f["refs"]), int)
    want[[table[0, 0], *table[1, :3]]] = 1
    np.testing.assert_array_equal(host(refs), want)
    assert torch.equal(f["k"][:, f["spare"][0], :, :2], before[0][:, table[0, 2], :, :2])
    assert torch.equal(f["k"][:, f["spare"][1]], before[0][:, f["spare"][1]])


@pytest.mark.parametrize("fault,status", [("taken", 1), ("width", 2), ("negative", 8), ("twice", 8), ("seq", 8), ("used", 8),
                                          ("page", 16), ("refs", 16), ("held", 32)])
@pytest.mark.parametrize("many", [False, True])
def test_kv_release_changes_nothing_when_it_cannot(fault, status, many):
    """In one CTA, and in a cluster of eight."""
    batch = 300 if many else 3
    kv, width = np.full(batch, 180), 3
    table = np.arange(3 * batch).reshape(batch, 3)
    refs, seqs, free, used = np.zeros(3 * batch, int), np.arange(batch), np.arange(3 * batch + 4), 3 * batch
    table[1, 0] = table[0, 0]
    refs[table[0, 0]] = 1  # held by two
    if fault == "taken":
        used = 3 * batch - 2
    elif fault == "width":
        kv[-1] = 193
    elif fault == "negative":
        kv[-1] = -1
    elif fault == "twice":
        seqs[-1] = 0
    elif fault == "seq":
        seqs[-1] = batch
    elif fault == "used":
        used = 3 * batch + 5
    elif fault == "page":
        table[-1, 2] = 3 * batch
    elif fault == "refs":
        refs[table[-1, 2]] = -1
    else:
        refs[table[0, 0]] = 0
    wide = i32(np.concatenate([table, np.zeros((batch, 4))], 1))[:, :width]
    fl, u, rf, uo = i32(free), i32([used]), i32(refs), i32([-7])
    r = dfl().kv_release(i32(seqs), i32(kv), wide, fl, u, rf, used_out=uo)
    assert int(r.status) == status and int(r.used) == used
    np.testing.assert_array_equal(host(fl), free)
    np.testing.assert_array_equal(host(rf), refs)


@pytest.mark.parametrize("batch,width", [(1, 1), (3, 5), (500, 40)])
def test_kv_release_behind_a_cut(batch, width):
    """Sequences that live on with fewer tokens: whole ones, none, and cuts at and inside pages; of one CTA and of a cluster."""
    rng = np.random.default_rng(batch)
    kv = rng.integers(0, 64 * width + 1, batch)
    keep = np.minimum(kv, rng.integers(0, 64 * width + 1, batch))
    keep[::3] = keep[::3] // 64 * 64
    keep[-1] = kv[-1]
    pages = -(-kv // 64)
    table, perm, at = np.full((batch, width), -5), rng.permutation(int(pages.sum()) + 3), 0
    for s in range(batch):
        table[s, :pages[s]] = perm[at:at + pages[s]]
        at += pages[s]
    seqs, used = rng.permutation(batch)[:max(1, batch - 1)], at + 1
    want = trees.kv_release(seqs, kv, table, np.arange(len(perm)), used, np.zeros(len(perm), int), keep)
    fl, u, refs = i32(np.arange(len(perm))), i32([used]), i32(np.zeros(len(perm)))
    r = dfl().kv_release(i32(seqs), i32(kv), i32(table), fl, u, refs, keep_lens=i32(keep), used_out=u)
    assert int(r.status) == want[3] == 0 and int(u) == want[1]
    np.testing.assert_array_equal(host(fl), want[0])
    np.testing.assert_array_equal(host(refs), want[2])


@pytest.mark.parametrize("cut", [-1, 101])
def test_kv_release_refuses_a_cut_outside_the_sequence(cut):
    fl, u, refs = i32([0, 1, 2, 3]), i32([4]), i32([0] * 4)
    r = dfl().kv_release(i32([1, 0]), i32([100, 100]), i32([[0, 1], [2, 3]]), fl, u, refs, keep_lens=i32([cut, 0]), used_out=u)
    assert int(r.status) == 8 and int(u) == 4 and (host(refs) == 0).all() and host(fl).tolist() == [0, 1, 2, 3]


def test_steps_of_trees_lose_no_page():
    """Trees that reach past a page and are cut before it, over many steps: the pages taken are the ones that hold tokens."""
    d = dfl()
    rng = np.random.default_rng(21)
    batch, m, n_pages, width = 4, 40, 60, 12
    k, v = (torch.zeros((n_pages + 1, 1, 64, 8), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fl, used, refs = i32(rng.permutation(n_pages)), i32([0]), i32(np.zeros(n_pages + 1))
    lens, table, new = i32(np.zeros(batch)), i32(np.full((batch, width), n_pages)), i32([m] * batch)
    q_start, seqs = i32(np.arange(batch + 1) * m), i32(np.arange(batch))
    for it in range(60):
        t = d.kv_tables(lens, new, table, fl, used, rows=batch * m, scratch_page=n_pages, table_out=table, used_out=used)
        assert int(t.status) == 0
        kv = lens + new
        acc = rng.integers(0, 9, batch)
        path = np.full((batch, 9), -1)
        for s in range(batch):
            path[s, :acc[s] + 1] = np.concatenate([[0], 1 + np.sort(rng.choice(m - 1, acc[s], replace=False))])
        c = d.kv_compact(k, v, table, kv, q_start, i32(path), i32(acc))
        r = d.kv_release(seqs, kv, table, fl, used, refs, keep_lens=c.kv_lens, used_out=used)
        assert (host(c.status) == 0).all() and int(r.status) == 0
        lens = c.kv_lens
        held = -(-host(lens) // 64)
        assert int(used) == held.sum()
        mine = np.concatenate([host(table)[s, :held[s]] for s in range(batch)])
        assert sorted(np.concatenate([mine, host(fl)[int(used):]])) == list(range(n_pages))


def test_pages_and_layers_behind_2_31_elements():
    """Caches of more than 2^31 elements a layer, and layers as far apart: the last page's tokens move, and are copied and read."""
    hkv, hd = 8, 128
    pages = (1 << 31) // (hkv * 64 * hd) + 2
    layer = pages * hkv * 64 * hd
    store = [torch.zeros(layer + 128 * hkv * 64 * hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = (x.as_strided((2, pages, hkv, 64, hd), (128 * hkv * 64 * hd, hkv * 64 * hd, 64 * hd, hd, 1)) for x in store)
    with pytest.raises(Exception, match="ld_layer"):  # (layers that overlap)
        dfl().kv_compact(k, v, i32([[0]]), i32([1]), i32([0, 1]), i32([[0]]), i32([0]))
    k, v = (x[:layer].view(pages, hkv, 64, hd) for x in store)
    g = torch.Generator().manual_seed(1)
    last = pages - 1
    for x in (k, v):
        x[last - 1:] = torch.randn((2, hkv, 64, hd), generator=g).to(torch.bfloat16).cuda()
    table, kv, start = i32([[last - 1, last]]), i32([90]), i32([0, 12])
    before = k[last].clone()
    got = dfl().kv_compact(k, v, table, kv, start, i32([[0, 3, 11, -1]]), i32([2]))
    assert int(got.status) == 0 and int(got.kv_lens) == 81
    assert torch.equal(k[last, :, 15], before[:, 17]) and torch.equal(k[last, :, 16], before[:, 25])  # nodes 3 and 11, to 79 and 80
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    f = dfl().kv_fork(i32([0]), got.kv_lens, table, i32([pages // 2 + 5]), i32([0]), refs, k, v)
    assert int(f.status) == 0 and torch.equal(k[pages // 2 + 5, :, :17], k[last, :, :17]) and int(refs[last - 1]) == 1
    c = dict(q=torch.randn((1, 8, hd), generator=g).to(torch.bfloat16).float().numpy(), k=host(k[last - 1:].float()), v=host(v[last - 1:].float()), pre=[],
             prefix=0, table=np.array([[0, 1]]), kv=np.array([81]), start=np.array([0, 1]), sees=[np.ones((1, 1), bool)], dtype="bf16", hd=hd)
    q = torch.from_numpy(c["q"]).to(torch.bfloat16).cuda()
    attn_check(c, dfl().tree_attention(q, k, v, table, got.kv_lens, i32([0, 1]), i32([[1]])))


# ------------------------------------------------------------------------------------------ a run of them together
@pytest.mark.parametrize("graph", [False, True])
def test_a_verified_tree_from_masks_to_the_next_step(graph):
    """Two samples of one prompt: forked, their trees verified and committed three times, released; eager, and the step captured
    and replayed.  The attention of the step behind a commit sees exactly the committed keys."""
    d = dfl()
    rng = np.random.default_rng(11)
    H, hkv, hd, layers, m, width = 8, 2, 128, 2, 12, 6
    f = fork_state(rng, [100], layers=layers, hkv=hkv, hd=hd)
    fl, used, refs = i32(f["spare"]), i32([0]), i32(f["refs"])
    k, v = f["k"], f["v"]
    kids = d.kv_fork(i32([0, 0]), i32([100]), i32(np.pad(f["table"], ((0, 0), (0, 2)), constant_values=f["scratch"])), fl, used, refs, k, v,
                     scratch_page=f["scratch"], used_out=used)
    table, lens = kids.table, kids.kv_lens.clone()
    new, q_start = i32([m, m]), i32([0, m, 2 * m])
    par, tok, post = (i32(np.zeros(2 * m)) for _ in range(3))
    q, keys, values = (torch.zeros((2 * m, n, hd), dtype=torch.bfloat16, device="cuda") for n in (H, hkv, hkv))

    def step():
        t = d.kv_tables(lens, new, table, fl, used, rows=2 * m, scratch_page=f["scratch"], table_out=table, used_out=used)
        kv = lens + new
        masks = d.tree_masks(par, q_start, kv_lens=kv, words=1)
        for c, x in ((k, keys), (v, values)):
            c[0][t.slots // 64, :, t.slots % 64] = x
            c[1][t.slots // 64, :, t.slots % 64] = x + 1
        out, lse = d.tree_attention(q, k[0], v[0], table, kv, q_start, masks.masks)
        a = d.tree_accept(par, tok, post, q_start, width=width)
        c = d.kv_compact(k, v, table, kv, q_start, a.path, a.accepted)
        lens.copy_(c.kv_lens)
        return out, lse, masks, a, c, t

    if graph:
        state = [x.clone() for x in (k, v, table, lens, fl, used, refs)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for x, y in zip((k, v, table, lens, fl, used, refs), state):
            x.copy_(y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
    # what layer 0 holds of each sequence
    prompt = [host(c[:, f["table"][0, :2]].float()).transpose(0, 2, 1, 3, 4).reshape(layers, hkv, 128, hd)[:, :, :100] for c in (k, v)]
    held = [[prompt[0][0], prompt[1][0]] for _ in range(2)]
    for it in range(3):
        forest, tokens, posterior = forest_case(rng, [m, m], 4)
        for dst, x in ((par, forest), (tok, tokens), (post, posterior)):
            dst.copy_(i32(np.concatenate(x)))
        for x in (q, keys, values):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(it)).to(x.dtype))
        if graph:
            g.replay()
        else:
            got = step()
        out, lse, masks, a, c, t = got
        assert int(t.status) == 0 and (host(masks.status) == 0).all() and (host(a.status) == 0).all() and (host(c.status) == 0).all()
        for s in range(2):
            own = slice(s * m, (s + 1) * m)
            K = np.concatenate([held[s][0], host(keys[own].float()).transpose(1, 0, 2)], 1)
            V = np.concatenate([held[s][1], host(values[own].float()).transpose(1, 0, 2)], 1)
            sees, depth = trees.ancestors(forest[s])
            n = K.shape[1]
            on = np.concatenate([np.ones((m, n - m), bool), sees], 1)
            z = np.einsum("rhd,hkd->rhk", host(q[own].float()).astype(np.float64), K.repeat(H // hkv, 0)) * hd ** -0.5
            z = np.where(on[:, None], z, -np.inf)
            p = np.exp(z - z.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            want = np.einsum("rhk,hkd->rhd", p, V.repeat(H // hkv, 0))
            weight = np.einsum("rhk,hkd->rhd", p, np.abs(V).repeat(H // hkv, 0))
            # one rounding of the output and one of each weight (2^-8 each); fp32 scores of |s| < 64 move a weight by less than 2^-12
            assert (np.abs(host(out[own].float()) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12) * weight).all()
            np.testing.assert_array_equal(host(masks.row_pos)[own], n - m + depth)
            path, acc, bonus = trees.tree_accept(forest[s], tokens[s], posterior[s], width)
            assert host(a.path)[s].tolist() == path and int(a.accepted[s]) == acc and int(a.bonus[s]) == bonus
            kept = np.concatenate([np.arange(n - m), n - m + np.array(path[:acc + 1])])
            held[s] = [K[:, kept], V[:, kept]]
            assert int(lens[s]) == len(kept) == int(c.kv_lens[s])
            for x, w in ((k, held[s][0]), (v, held[s][1])):
                rows = host(x[0][table[s].long()].float()).transpose(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :len(kept)]
                np.testing.assert_array_equal(rows, w)
    r = d.kv_release(i32([0, 1]), lens, table, fl, used, refs, used_out=used)
    assert int(r.status) == 0 and int(used) == 0 and (host(refs) == 0).all()
    assert sorted(host(fl)) == sorted(f["spare"])


def test_the_operators_on_a_side_stream_beside_others():
    """Calls on two streams at once, each with tensors of its own."""
    c = [attn_case("bf16", (32, 8, 128), 300, [700, 90], [40, 64], seed=80 + i) for i in range(2)]
    x = [attn_run(y) for y in c]
    want = [[t.clone() for t in dfl().tree_attention(*a, **kw)] for a, kw in x]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(8):
        got.append((0, dfl().tree_attention(*x[0][0], **x[0][1])))
        with torch.cuda.stream(s):
            got.append((1, dfl().tree_attention(*x[1][0], **x[1][1])))
    torch.cuda.synchronize()
    for i, (o, l) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def cut_case(kind, many):
    """Pages 0 and 1 hold 128 tokens of sequences 0 and 1, which have a page of their own each behind them; 2 is alone."""
    kv, keep, seqs = [200, 200, 130], [200, 100, 70], [1]
    table, refs, status = [[0, 1, 2, 3], [0, 1, 4, 5], [6, 7, 8, 9]], np.zeros(10, int), 64
    refs[:2] = 1
    if kind == "last page":         # nothing is given back, and the page is written to all the same
        kv, keep = [128, 128, 130], [128, 100, 70]
    elif kind == "both":
        keep, seqs = [120, 100, 70], [0, 1]
    elif kind == "first page":
        keep = [200, 63, 70]
    elif kind == "whole pages":     # a new page is written to next
        keep, status = [200, 64, 70], 0
    elif kind == "nothing left":
        keep, status = [200, 0, 70], 0
    elif kind == "no cut":
        kv, keep, status = [100, 100, 130], [100, 100, 70], 0
    elif kind == "others end":      # the other holder leaves in the same call
        keep, seqs, status = [0, 100, 70], [0, 1], 0
    elif kind == "alone":
        seqs, status = [2], 0
    elif kind == "held by fewer":   # page 1 is sequence 1's alone, and another gives it back
        refs[1], keep, seqs, status = 0, [0, 100, 70], [0, 1], 32
    elif kind == "bad page":
        table[2][1], seqs, status = 10, [2], 16
    elif kind == "bad count":
        refs[7], seqs, status = -1, [2], 16
    if many:  # hundreds of others end with it: a cluster of eight CTAs
        n = 400
        table += (10 + np.arange(4 * n).reshape(n, 4)).tolist()
        kv, keep, seqs = kv + [250] * n, keep + [0] * n, list(range(3, 3 + n)) + seqs
        refs = np.concatenate([refs, np.zeros(4 * n, int)])
        table = [[p if kind != "bad page" or p != 10 or s != 2 else len(refs) for p in row] for s, row in enumerate(table)]
    free = np.arange(len(refs), len(refs) + len(refs) + 4)
    return kv, keep, seqs, np.array(table), refs, free, status


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("kind", ["shared", "last page", "both", "first page", "whole pages", "nothing left", "no cut", "others end", "alone",
                                  "held by fewer", "bad page", "bad count"])
def test_kv_release_refuses_a_cut_into_a_page_that_others_hold(kind, many):
    """The page that a cut ends in is written to next: with another holder left the call says so and changes nothing."""
    kv, keep, seqs, table, refs, free, status = cut_case(kind, many)
    used = len(refs)
    fl, u, rf = i32(free), i32([used]), i32(refs)
    r = dfl().kv_release(i32(seqs), i32(kv), i32(table), fl, u, rf, keep_lens=i32(keep), used_out=u)
    assert int(r.status) == status
    if status == 0:
        free, used, refs, _ = trees.kv_release(seqs, kv, table, free, used, refs, keep)
    assert int(u) == used
    np.testing.assert_array_equal(host(fl), free)
    np.testing.assert_array_equal(host(rf), refs)


def test_a_fork_that_is_cut_back_takes_a_page_of_its_own():
    """What a caller does instead: the sequence forks itself at the shorter length, which copies the page, and ends."""
    rng = np.random.default_rng(31)
    f = fork_state(rng, [128])
    fl, used, refs = i32(f["spare"]), i32([0]), i32(f["refs"])
    k, v, table = f["k"], f["v"], i32(f["table"])
    kid = dfl().kv_fork(i32([0]), i32([128]), table, fl, used, refs, k, v, scratch_page=f["scratch"], used_out=used)
    cut = dfl().kv_release(i32([0]), kid.kv_lens, kid.table, fl, used, refs, keep_lens=i32([100]), used_out=used)
    assert int(cut.status) == 64 and int(used) == 0
    short = dfl().kv_fork(i32([0]), i32([100]), kid.table, fl, used, refs, k, v, scratch_page=f["scratch"], used_out=used)
    end = dfl().kv_release(i32([0]), kid.kv_lens, kid.table, fl, used, refs, used_out=used)
    assert int(short.status) == int(end.status) == 0 and int(used) == 1
    pages, parent = host(short.table)[0], f["table"][0]
    assert pages[0] == parent[0] and pages[1] == f["spare"][0]
    assert host(refs)[parent[0]] == 1 and host(refs)[parent[1]] == 0 and host(refs)[pages[1]] == 0
    assert torch.equal(k[:, pages[1], :, :36], k[:, parent[1], :, :36])


def test_a_sequence_ends_once():
    """The counts know holders beyond the first, not whether a page is free: a call after the one that ended a sequence cannot tell
    that it names the same one, and takes the pages again, or finds more of them than were taken."""
    table, kv = i32([[0, 1], [2, 3]]), i32([100, 100])
    fl, used, refs = i32([0, 1, 2, 3]), i32([4]), i32([0] * 4)
    for status, left, want in ((0, 2, [0, 1, 0, 1]), (0, 0, [0, 1, 0, 1]), (1, 0, [0, 1, 0, 1])):
        r = dfl().kv_release(i32([0]), kv, table, fl, used, refs, used_out=used)
        assert int(r.status) == status and int(used) == left and host(fl).tolist() == want and (host(refs) == 0).all()


@pytest.mark.parametrize("base,kv,m,status,first", [
    (0, 3, 5, 8, None), (0, -1, 5, 8, None), (17, -1, 5, 8, None), (17, 3, 5, 0, 15), (2, 3, 5, 0, 0), (1, 3, 5, 8, None),
    (1 << 30, (1 << 31) - 1, 5, 8, None), (1 << 30, (1 << 30) + 1, 5, 8, None), (1 << 30, 1 << 30, 5, 0, (1 << 31) - 5),
    (0, (1 << 31) - 1, 1, 0, (1 << 31) - 2), (0, -1, 0, 8, None)])
def test_tree_masks_of_lengths_below_the_tree_and_beyond_a_position(base, kv, m, status, first):
    """A length below m counts from behind the cache's begin, as in the attention, where base_pos leaves room; masks and depths
    do not depend on it."""
    p = random_tree(np.random.default_rng(m), m, 0.9)
    t = dfl().tree_masks(i32(np.concatenate([p, [-1, 0]])), i32([0, m, m + 2]), kv_lens=i32([kv, 2]), base_pos=base, words=1)
    assert host(t.status).tolist() == [status, 0]
    sees, depth = trees.ancestors(p)
    np.testing.assert_array_equal(host(t.masks)[:m], trees.words(sees, 1))
    np.testing.assert_array_equal(host(t.depth)[:m], depth)
    np.testing.assert_array_equal(host(t.row_pos), np.concatenate([first + depth if status == 0 else np.full(m, -1), [base, base + 1]]))


def test_tree_masks_report_a_bad_tree_and_its_bad_length():
    t = dfl().tree_masks(i32([-1, 1]), i32([0, 2]), kv_lens=i32([-4]), words=1)
    assert host(t.status).tolist() == [9] and host(t.row_pos).tolist() == host(t.depth).tolist() == [-1, -1]
    assert (host(t.masks) == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_kv_compact_and_fork_of_interleaved_caches(dtype):
    """Keys and values of a layer beside each other in one tensor: views that interleave and do not overlap."""
    rng = np.random.default_rng(9)
    kv, layers, hkv, hd = np.array([90, 130]), 3, 2, 64
    (k, v), table, spare = cache_case(rng, dtype, layers, hkv, hd, kv, slack=4)
    both = torch.stack([k, v], 1)
    ki, vi = both[:, 0], both[:, 1]
    start, path, acc = i32([0, 9, 20]), i32([[0, 3, 8, -1], [0, 1, 10, -1]]), i32([2, 2])
    got = [dfl().kv_compact(*x, i32(table), i32(kv), start, path, acc) for x in ((k, v), (ki, vi))]
    assert all((host(g.status) == 0).all() for g in got) and torch.equal(got[0].kv_lens, got[1].kv_lens)
    assert torch.equal(both, torch.stack([k, v], 1))
    for x in ((k, v), (ki, vi)):
        f = dfl().kv_fork(i32([1, 0]), got[0].kv_lens, i32(table), i32(spare), i32([0]), i32(np.zeros(k.shape[1])), *x)
        assert int(f.status) == 0
    assert torch.equal(both, torch.stack([k, v], 1))


def test_kv_compact_of_a_refused_tree_takes_the_step_back():
    """tree_accept gives a bad tree accepted = -1, and compaction then keeps none of its nodes, the root neither."""
    rng = np.random.default_rng(6)
    kv = np.array([70, 75])
    (k, v), table, _ = cache_case(rng, "bf16", 2, 2, 64, kv)
    a = dfl().tree_accept(i32([-1, 0, 0, -1, 2, 0]), i32(np.zeros(6)), i32(np.zeros(6)), i32([0, 3, 6]), width=3)
    assert host(a.status).tolist() == [0, 1] and host(a.accepted)[1] == -1
    before = [x[:, table[1, :2]].clone() for x in (k, v)]
    c = dfl().kv_compact(k, v, i32(table), i32(kv), i32([0, 3, 6]), a.path, a.accepted)
    assert host(c.status).tolist() == [0, 0] and host(c.kv_lens).tolist() == [69, 72]
    assert all(torch.equal(x[:, table[1, :2]], b) for x, b in zip((k, v), before))


def test_steps_and_pages_on_a_side_stream_beside_others():
    """Masks, acceptance, compaction, fork and release on two streams at once, each with tensors of its own: what they give alone."""
    d = dfl()
    sizes, n = [40, 33, 64, 17], 4
    kv = np.array([300, 120, 700, 64]) + sizes

    def state(i):
        rng = np.random.default_rng(50 + i)
        forest, tokens, posterior = forest_case(rng, sizes, 5)
        f = fork_state(rng, kv, layers=6, hkv=8, hd=128, free=60)
        table = np.pad(f["table"], ((0, 0), (0, 2)), constant_values=f["scratch"])
        return dict(par=i32(np.concatenate(forest)), tok=i32(np.concatenate(tokens)), post=i32(np.concatenate(posterior)), k=f["k"], v=f["v"],
                    start=i32(starts(sizes)), kv=i32(kv), table=i32(table), fl=i32(f["spare"]), used=i32([2]), refs=i32(f["refs"]),
                    parents=i32(np.arange(3 * n) % n), kids=i32(np.arange(3 * n)), scratch=f["scratch"])

    def run(s):
        t = d.tree_masks(s["par"], s["start"], kv_lens=s["kv"], words=2)
        a = d.tree_accept(s["par"], s["tok"], s["post"], s["start"], width=9)
        c = d.kv_compact(s["k"], s["v"], s["table"], s["kv"], s["start"], a.path, a.accepted)
        f = d.kv_fork(s["parents"], c.kv_lens, s["table"], s["fl"], s["used"], s["refs"], s["k"], s["v"], scratch_page=s["scratch"],
                      used_out=s["used"])
        held = s["refs"].clone()
        r = d.kv_release(s["kids"], f.kv_lens, f.table, s["fl"], s["used"], s["refs"], used_out=s["used"])
        return [*t, *a, *c, f.table, f.kv_lens, f.status, held, r.status, s["fl"], s["used"], s["refs"], s["k"], s["v"]]

    want = [[x.clone() for x in run(state(i))] for i in range(2)]
    both = [[state(i) for _ in range(4)] for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = [[], []]
    for j in range(4):
        got[0].append(run(both[0][j]))
        with torch.cuda.stream(side):
            got[1].append(run(both[1][j]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(g, want[i]))
