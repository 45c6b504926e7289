"""The serving operators on the GPU against their fp64 oracles, at the lengths, masks, strides and
orders where they can go wrong."""
import numpy as np
import pytest
import torch

from oracle import serving

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


# ------------------------------------------------------------------------------------------------ page tables
def tables_case(batch, kv_hi, new_hi, width_extra, slack, seed, base=0, rows_extra=0):
    rng = np.random.default_rng(seed)
    kv = rng.integers(0, kv_hi + 1, batch)
    new = rng.integers(0, new_hi + 1, batch)
    old, need = -(-kv // 64), -(-(kv + new) // 64)
    width = int(need.max()) + width_extra
    n_pages = int(need.sum()) + slack + 5
    perm = rng.permutation(n_pages)
    table = np.full((batch, width), n_pages)
    at = 0
    for s in range(batch):
        table[s, :old[s]] = perm[at:at + old[s]]
        at += old[s]
    free = perm[at:at + int((need - old).sum()) + slack]
    return kv, new, table, free, int(new.sum()) + rows_extra, n_pages, base


def run_tables(kv, new, table, free, rows, scratch, base, used=0, in_place=False):
    t = i32(table)
    f = None if free is None else i32(free)
    u = None if free is None else i32([used])
    kw = dict(table_out=t, used_out=u) if in_place else {}
    return dfl().kv_tables(i32(kv), i32(new), t, f, u, rows=rows, scratch_page=scratch, base_pos=base, **kw)


def check_tables(got, want, check_table=True):
    table, used, q_start, row_seq, row_pos, slots, status = want
    assert int(got.status) == status
    for name, g, w in (("q_start", got.q_start, q_start), ("row_seq", got.row_seq, row_seq),
                       ("row_pos", got.row_pos, row_pos), ("slots", got.slots, slots)):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    if check_table and table is not None and got.table is not None:
        np.testing.assert_array_equal(got.table.cpu().numpy(), table)
    if got.used is not None:
        assert int(got.used) == used


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,kv_hi,new_hi,width_extra,slack,base,rows_extra", [
    (1, 0, 1, 0, 0, 0, 0), (1, 0, 0, 3, 2, 0, 4), (3, 130, 70, 1, 0, 17, 0), (32, 2303, 1, 4, 9, 8192, 3),
    (33, 64, 64, 0, 1, 0, 1), (511, 90, 3, 2, 0, 0, 0), (513, 300, 40, 1, 7, 64, 100), (1024, 2303, 16, 5, 0, 8192, 0),
    (2048, 130, 20, 0, 3, 1, 5)])
def test_kv_tables(batch, kv_hi, new_hi, width_extra, slack, base, rows_extra, in_place):
    kv, new, table, free, rows, scratch, base = tables_case(batch, kv_hi, new_hi, width_extra, slack, batch, base, rows_extra)
    if batch == 1 and new_hi:
        new[:] = 1
        rows, free = 1 + rows_extra, np.array([3])
        table = np.full((1, 1 + width_extra), scratch)
    pad = np.concatenate([np.array([-7, -8]), free])  # two pages taken by earlier steps
    want = serving.kv_tables(kv, new, table, pad, 2, rows, scratch, base)
    assert want[-1] == 0
    check_tables(run_tables(kv, new, table, pad, rows, scratch, base, used=2, in_place=in_place), want)


@pytest.mark.parametrize("fault", ["pool", "width", "rows", "negative", "used"])
def test_kv_tables_reports_what_only_the_device_sees(fault):
    kv, new, table, free, rows, scratch, base = tables_case(70, 200, 90, 0, 0, 5)
    new[69] = 300 - kv[69]
    table = np.concatenate([table, np.full((70, 1), scratch)], 1)  # 300 tokens: five pages
    free = np.arange(1000, 1000 + int((-(-(kv + new) // 64) - -(-kv // 64)).sum()))
    rows, used = int(new.sum()), 0
    assert serving.kv_tables(kv, new, table, free, 0, rows, scratch)[-1] == 0
    if fault == "pool":
        free = free[:-1]
    elif fault == "width":
        table = table[:, :4]
    elif fault == "rows":
        rows -= 1
    elif fault == "negative":
        new[13] = -1
    else:
        used = -1
    want = serving.kv_tables(kv, new, table, free, used, rows, scratch)
    assert want[-1] != 0
    t = i32(table)
    got = run_tables(kv, new, table, free, rows, scratch, 0, used=used, in_place=True)
    check_tables(got, want)
    torch.testing.assert_close(got.table, t)  # nothing taken


def test_kv_tables_from_a_table_that_backs_every_token():
    """No free list: the maps alone, read from a table that is a slice of a wider one."""
    kv, new, table, free, rows, scratch, base = tables_case(40, 500, 100, 1, 0, 9)
    full = serving.kv_tables(kv, new, table, free, 0, rows, scratch, 0)[0]
    want = serving.kv_tables(kv, new, full, None, 0, rows + 6, scratch, 1000)
    wide = i32(np.concatenate([np.full((40, 3), -5), full], 1))
    got = dfl().kv_tables(i32(kv), i32(new), wide[:, 3:], rows=rows + 6, base_pos=1000)
    check_tables(got, want, check_table=False)
    assert got.table is None and got.used is None


def test_kv_tables_chained_steps_in_a_graph():
    """Ten captured decode steps in place: lengths advance on the device, pages come off one list."""
    batch, width = 5, 4
    kv = np.array([0, 1, 62, 63, 64])
    table = np.full((batch, width), 77)
    perm = np.arange(30)
    for s in range(batch):
        table[s, :-(-kv[s] // 64)] = 50 + s
    t, k, one, f, u = i32(table), i32(kv), i32([1] * batch), i32(perm), i32([0])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [dfl().kv_tables(k, one, t, f, u, rows=batch, scratch_page=77, table_out=t, used_out=u, status=st)]  # step 0
    k += 1
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        o = dfl().kv_tables(k, one, t, f, u, rows=batch, scratch_page=77, table_out=t, used_out=u, status=st)
        k += 1
    want_t, used, hk = table, 0, kv.copy()
    for step in range(10):
        want_t, used, *_, slots, status = serving.kv_tables(hk, [1] * batch, want_t, perm, used, batch, 77)
        hk += 1
        if step:
            g.replay()
        got = (outs[0] if step == 0 else o).slots
        np.testing.assert_array_equal(got.cpu().numpy(), slots)
        np.testing.assert_array_equal(t.cpu().numpy(), want_t)
        assert int(u) == used and int(st) == 0 == status


# ------------------------------------------------------------------------------------ shared-prefix attention
def attn_case(dtype, heads, prefix, kv, q, seed, stale=float("nan"), extra_pages=2, q_scale=1.0):
    """Inputs on the host (float32 values of the type) with every slot past a valid token at ``stale``."""
    H, hkv, hd = heads
    g = torch.Generator().manual_seed(seed)
    kv, q = np.asarray(kv), np.asarray(q)
    n_pre = -(-prefix // 64)
    npg = -(-kv // 64)
    n_pages = n_pre + int(npg.sum()) + extra_pages
    perm = torch.randperm(n_pages, generator=g).numpy()
    width = max(1, int(npg.max()) + 1)
    table = np.full((len(kv), width), -1)  # entries past a sequence's pages are never read
    k = torch.randn((n_pages, hkv, 64, hd), generator=g).to(DT[dtype]).float().numpy()
    v = torch.randn((n_pages, hkv, 64, hd), generator=g).to(DT[dtype]).float().numpy()
    live = np.zeros((n_pages, 64), bool)
    pre = perm[:n_pre]
    at = n_pre

    def fill(pages, n):
        for i, p in enumerate(pages):
            live[p, :min(64, n - 64 * i)] = True

    fill(pre, prefix)
    for s in range(len(kv)):
        table[s, :npg[s]] = perm[at:at + npg[s]]
        fill(table[s, :npg[s]], int(kv[s]))
        at += npg[s]
    for c in (k, v):
        c[~live[:, None, :].repeat(hkv, 1)] = stale
    rows = int(q.sum())
    qq = (q_scale * torch.randn((rows, H, hd), generator=g)).to(DT[dtype]).float().numpy()
    return dict(q=qq, k=k, v=v, pre=pre, prefix=prefix, table=table, kv=kv,
                start=np.concatenate([[0], np.cumsum(q)]), dtype=dtype, hd=hd)


def attn_inputs(c):
    dt = DT[c["dtype"]]
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dt).cuda()  # noqa: E731
    return (up(c["q"]), up(c["k"]), up(c["v"]), i32(c["pre"]) if c["prefix"] else None, c["prefix"], i32(c["table"]),
            i32(c["kv"]), i32(c["start"]))


def attn_check(c, got, causal, scale=None):
    """Error bounds.  u = 2^-24.  A score is a sum of hd products in fp32, off by at most
    hd u sum|q_i k_i| scale =: z; each softmax weight is then off by a factor of at most exp(2 z) and by
    the rounding of the exponent's argument, |score| u log2(e), plus exp2 itself (2^-22) and the n-term
    sums (n u).  In bf16 each weight is also rounded once (half a step, 2^-8).  The output is rounded
    once to its type."""
    scale = c["hd"] ** -0.5 if scale is None else scale
    out, lse, weight = serving.shared_prefix_attention(c["q"], c["k"], c["v"], c["pre"], c["prefix"], c["table"], c["kv"],
                                                       c["start"], causal, scale)
    u = 2.0 ** -24
    n = c["prefix"] + int(max(c["kv"].max(), 0))
    kmax = np.nanmax(np.abs(np.where(np.isfinite(c["k"]), c["k"], 0)).sum(-1)) if c["k"].size else 0.0
    qk = scale * float(np.abs(c["q"]).max()) * kmax          # >= sum|q_i k_i| scale
    z = c["hd"] * u * qk
    delta = 2 * z + 4 * qk * u + 2.0 ** -22 + (n + 64) * u
    tol = HALF[c["dtype"]] * np.abs(out) + (delta + (2.0 ** -8 if c["dtype"] == "bf16" else 0)) * weight + 1e-30
    g, gl = got[0].float().cpu().numpy().astype(np.float64), got[1].cpu().numpy().astype(np.float64)
    assert np.isfinite(g).all()
    bad = np.abs(g - out) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(g - out) / tol).max()), np.argwhere(bad)[:4])
    inf = np.isneginf(lse)
    assert (np.isneginf(gl) == inf).all()
    ltol = z + 4 * qk * u + (n + 64) * u + 2.0 ** -21 + np.abs(np.where(inf, 0, lse)) * 2.0 ** -22
    assert (np.abs(np.where(inf, 0, gl) - np.where(inf, 0, lse)) <= ltol).all()


ATTN = [
    # heads (H, H_kv, hd), prefix, own keys, rows, causal
    ((8, 2, 128), 64, [1], [1], True),
    ((8, 2, 128), 1, [0], [1], False),
    ((8, 2, 128), 0, [5, 70], [1, 3], True),
    ((8, 2, 128), 63, [0, 0, 0], [1, 0, 2], True),
    ((32, 8, 128), 500, [1, 100, 64, 63], [1, 1, 1, 1], True),
    ((32, 8, 128), 129, [16, 300, 17], [16, 16, 16], False),
    ((32, 8, 128), 700, [16, 300, 17, 90], [16, 16, 16, 16], True),
    ((4, 1, 128), 200, [130, 1, 40, 7], [130, 1, 40, 7], True),       # ragged suffixes, their own keys only
    ((4, 2, 64), 333, [10, 64, 65], [4, 4, 4], True),
    ((16, 8, 64), 1000, [200, 33], [8, 9], False),
    ((8, 8, 128), 400, [65, 1], [33, 1], True),                       # one query head a KV head
    ((6, 2, 128), 257, [50, 80], [45, 44], True),                     # three: 128 is not a multiple
    ((14, 2, 128), 190, [30, 20], [20, 20], True),                    # seven
    ((64, 1, 128), 150, [9, 3], [9, 3], True),                        # 64
    ((5, 1, 64), 320, [2, 1, 0, 9], [2, 1, 0, 3], True),
    ((8, 2, 128), 64, [2, 5], [6, 5], True),                          # more rows than own keys: rows that see the prefix only
    ((8, 2, 128), 0, [2, 0], [6, 1], True),                           # ... and rows that see nothing
    ((8, 2, 128), 2100, [3, 500, 1029], [2, 1, 5], True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(ATTN)))
def test_shared_prefix_attention(i, dtype):
    heads, prefix, kv, q, causal = ATTN[i]
    c = attn_case(dtype, heads, prefix, kv, q, seed=100 + i)
    attn_check(c, dfl().shared_prefix_attention(*attn_inputs(c), causal=causal), causal)


@pytest.mark.parametrize("i", range(len(ATTN)))
def test_shared_prefix_attention_weight_pairs(i):
    """bf16 with each weight as a pair: what the second value leaves of a weight is half a step of half a step (2^-16) where
    attn_check has half a step; the other terms are its.  lse is that of the plain call, bit for bit."""
    heads, prefix, kv, q, causal = ATTN[i]
    c = attn_case("bf16", heads, prefix, kv, q, seed=100 + i)
    x = attn_inputs(c)
    got = dfl().shared_prefix_attention(*x, causal=causal, weight_pairs=True)
    attn_check(c, got, causal)
    assert torch.equal(got[1], dfl().shared_prefix_attention(*x, causal=causal)[1])
    scale, u = c["hd"] ** -0.5, 2.0 ** -24
    out, _, weight = serving.shared_prefix_attention(c["q"], c["k"], c["v"], c["pre"], c["prefix"], c["table"], c["kv"],
                                                     c["start"], causal, scale)
    n = c["prefix"] + int(c["kv"].max())
    qk = scale * float(np.abs(c["q"]).max()) * np.nanmax(np.abs(np.where(np.isfinite(c["k"]), c["k"], 0)).sum(-1))
    delta = 2 * c["hd"] * u * qk + 4 * qk * u + 2.0 ** -22 + (n + 64) * u
    tol = HALF["bf16"] * np.abs(out) + (delta + 2.0 ** -16) * weight + 1e-30
    err = np.abs(got[0].float().cpu().numpy() - out)
    assert (err <= tol).all(), float((err / tol).max())


def test_shared_prefix_attention_weight_pairs_in_fp32_change_nothing():
    c = attn_case("f32", (8, 2, 128), 300, [70, 3], [2, 3], seed=5)
    x = attn_inputs(c)
    a, b = dfl().shared_prefix_attention(*x), dfl().shared_prefix_attention(*x, weight_pairs=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch", [300, 2048])
def test_shared_prefix_attention_many_short_sequences(dtype, batch):
    rng = np.random.default_rng(3)
    kv = rng.integers(0, 90, batch)
    c = attn_case(dtype, (2, 1, 64), 130, kv, rng.integers(0, 3, batch), seed=4)
    attn_check(c, dfl().shared_prefix_attention(*attn_inputs(c)), True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_prefix_attention_peaked_scores(dtype):
    """Scores that span hundreds: the running maximum moves far and often."""
    c = attn_case(dtype, (8, 2, 128), 900, [40, 200], [3, 5], seed=8, q_scale=30.0)
    attn_check(c, dfl().shared_prefix_attention(*attn_inputs(c), scale=0.2), True, scale=0.2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_prefix_attention_strides_and_rows_behind(dtype):
    """q is a slice of a fused q/k/v buffer, out of a wider one, table of a wider table; rows of no
    sequence (before the first and behind the last) keep what they held."""
    c = attn_case(dtype, (8, 2, 128), 150, [70, 20], [2, 3], seed=21)
    q, k, v, pre, n, table, kv, start = attn_inputs(c)
    fused = torch.full((9, 12, 128), 7.0, dtype=q.dtype, device="cuda")
    fused[2:7, :8] = q
    out = torch.full((9, 16, 128), 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full((9, 8), 5.0, device="cuda")
    wide = torch.cat([torch.full((2, 3), -9, dtype=torch.int32, device="cuda"), table], 1)
    o, l = dfl().shared_prefix_attention(fused[:, :8], k, v, pre, n, wide[:, 3:], kv, start + 2, out=out[:, :8], lse=lse)
    attn_check(c, (o[2:7], l[2:7]), True)
    keep = torch.tensor([0, 1, 7, 8])
    assert (out[keep] == 5.0).all() and (lse[keep] == 5.0).all() and (out[:, 8:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_prefix_attention_equals_itself(dtype):
    """The same call twice gives the same bits."""
    c = attn_case(dtype, (32, 8, 128), 1500, [400, 33, 1000], [16, 16, 16], seed=31)
    x = attn_inputs(c)
    a, b = (dfl().shared_prefix_attention(*x) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_shared_prefix_attention_workspaces_of_its_own():
    """No workspace given: calls of growing and shrinking sizes on the default stream (which share one) while others
    run on a side stream (one each) give what calls with a workspace of their own give, bit for bit."""
    cases = [attn_inputs(attn_case("bf16", (8, 2, 128), p, kv, q, seed=71 + p)) for p, kv, q in
             ((100, [70, 3], [2, 3]), (3000, [400, 90, 65, 10], [90, 1, 64, 17]), (500, [20], [20]))]
    own = [torch.empty(dfl().shared_prefix_workspace(x[0], x[1], x[6].numel()), dtype=torch.uint8, device="cuda") for x in cases]
    want = [[t.clone() for t in dfl().shared_prefix_attention(*x, workspace=w)] for x, w in zip(cases, own)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(12):
        got.append((i % 3, dfl().shared_prefix_attention(*cases[i % 3])))
        with torch.cuda.stream(side):
            got.append(((i + 1) % 3, dfl().shared_prefix_attention(*cases[(i + 1) % 3])))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_shared_prefix_attention_from_two_threads():
    """Two host threads with calls of different shapes on the default stream, which share the kept workspace: each
    result is that of a call with a workspace of its own, bit for bit."""
    import threading
    cases = [attn_inputs(attn_case("bf16", heads, p, kv, q, seed=77 + p)) for heads, p, kv, q in
             (((8, 2, 128), 100, [70, 3], [2, 3]), ((32, 8, 128), 900, [400, 90, 65, 10], [9, 1, 64, 17]))]
    own = [torch.empty(dfl().shared_prefix_workspace(x[0], x[1], x[6].numel()), dtype=torch.uint8, device="cuda") for x in cases]
    want = [[t.clone() for t in dfl().shared_prefix_attention(*x, workspace=w)] for x, w in zip(cases, own)]
    torch.cuda.synchronize()
    wrong = [0, 0]

    def work(i):
        for _ in range(20):
            got = [dfl().shared_prefix_attention(*cases[i]) for _ in range(50)]
            wrong[i] += sum(not (torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])) for o, l in got)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at", [16, 32, 48, 240, 4080])
def test_shared_prefix_attention_wherever_its_workspace_begins(dtype, at):
    """A workspace of exactly the size asked for, on any 16-byte boundary: the same bits, and nothing written beside it."""
    c = attn_case(dtype, (8, 2, 128), 300, [70, 3, 130], [2, 3, 40], seed=75)
    x = attn_inputs(c)
    want = dfl().shared_prefix_attention(*x)
    n = dfl().shared_prefix_workspace(x[0], x[1], 3)
    buf = torch.full((4096 + n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = dfl().shared_prefix_attention(*x, workspace=buf[at:at + n])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (buf[:at] == 0xA5).all() and (buf[at + n:] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch", [31, 32, 33, 65])
def test_shared_prefix_attention_batches_around_a_warp(dtype, batch):
    """The plan is made by a warp up to 32 sequences and by the whole CTA beyond; empty sequences first, last and
    between; then a row start that decreases, in either."""
    rng = np.random.default_rng(batch)
    q = rng.integers(0, 4, batch)
    q[[0, batch // 2, batch - 1]] = 0
    c = attn_case(dtype, (4, 2, 64), 200, rng.integers(0, 150, batch), q, seed=batch)
    x = list(attn_inputs(c))
    attn_check(c, dfl().shared_prefix_attention(*x), True)
    x[7] = x[7].clone()
    x[7][batch // 2] = -1
    out, lse = dfl().shared_prefix_attention(*x)
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_prefix_attention_in_place(dtype):
    """out is q: the queries have all been read before the first result is written."""
    c = attn_case(dtype, (32, 8, 128), 700, [400, 33, 90], [16, 1, 50], seed=33)
    x = attn_inputs(c)
    want = dfl().shared_prefix_attention(*x)
    got = dfl().shared_prefix_attention(*x, out=x[0])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fault", ["table", "table_negative", "prefix", "kv_len", "kv_negative", "q_start"])
def test_shared_prefix_attention_reports_bad_metadata(dtype, fault):
    """A page, length or row start out of range: NaN in the rows it concerns, the others as they should be."""
    c = attn_case(dtype, (8, 2, 128), 100, [70, 130, 20], [2, 2, 2], seed=41)
    x = list(attn_inputs(c))
    if fault.startswith("table"):
        x[5][1, 1] = c["k"].shape[0] if fault == "table" else -1
    elif fault == "prefix":
        x[3][1] = 1 << 30
    elif fault == "kv_len":
        x[6][1] = 64 * c["table"].shape[1] + 1
    elif fault == "kv_negative":
        x[6][1] = -3
    else:
        x[7][2] = 1  # sequence 1 would have -1 rows
    out = torch.zeros_like(x[0])
    lse = torch.zeros(x[0].shape[:2], device="cuda")
    dfl().shared_prefix_attention(*x, out=out, lse=lse)
    if fault in ("prefix", "q_start"):  # every row's keys, or whose rows they are, cannot be told
        assert out.isnan().all() and lse.isnan().all()
        return
    assert out[2:4].isnan().all() and lse[2:4].isnan().all()
    # the other rows as without the fault, within the bounds (not bit for bit: how the keys are split
    # depends on every sequence's length, and each split adds its partial sums in another order)
    good = dfl().shared_prefix_attention(*attn_inputs(c))
    out[2:4], lse[2:4] = good[0][2:4], good[1][2:4]
    attn_check(c, (out, lse), True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [0, 2, 3])
def test_shared_prefix_attention_bad_page_of_many_rows(dtype, page):
    """A sequence of several row tiles: every row that sees the bad page is NaN, a row before it NaN or right, and the other
    sequence and the rows of none are as they should be."""
    c = attn_case(dtype, (8, 2, 128), 100, [200, 70], [200, 70], seed=43)
    x = list(attn_inputs(c))
    good = dfl().shared_prefix_attention(*x)
    x[5][0, page] = -7
    x[7] = x[7] + 2
    out, lse = torch.full((274, 8, 128), 5.0, dtype=x[0].dtype, device="cuda"), torch.full((274, 8), 5.0, device="cuda")
    q = torch.zeros_like(out)
    q[2:272] = x[0]
    dfl().shared_prefix_attention(q, *x[1:], out=out, lse=lse)
    assert (out[[0, 1, 272, 273]] == 5.0).all() and (lse[[0, 1, 272, 273]] == 5.0).all()
    out, lse = out[2:272], lse[2:272]
    assert out[64 * page:200].isnan().all() and lse[64 * page:200].isnan().all()
    assert not lse[200:].isnan().any()
    nan = lse.isnan()
    assert torch.equal(out.isnan(), nan[..., None].expand_as(out))
    attn_check(c, (torch.where(nan[..., None], good[0], out), torch.where(nan, good[1], lse)), True)


def test_shared_prefix_attention_past_32_bit_offsets():
    """Pages whose element offset passes 2^31 (and whose byte offset passes 2^32)."""
    hkv, hd = 8, 128
    n_pages = (1 << 31) // (hkv * 64 * hd) + 40
    c = attn_case("bf16", (16, hkv, hd), 100, [70, 5], [2, 1], seed=51, extra_pages=0)
    k = torch.empty((n_pages, hkv, 64, hd), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    x = list(attn_inputs(c))
    n = c["k"].shape[0]
    k[-n:], v[-n:] = x[1], x[2]
    x[1], x[2] = k, v
    x[3] = x[3] + (n_pages - n)
    x[5] = torch.where(x[5] >= 0, x[5] + (n_pages - n), x[5])
    attn_check(c, dfl().shared_prefix_attention(*x), True)


def sampled_case(c, q, rows):
    """The case with some of its rows alone (their queries in q): each a sequence of its own that sees what the row saw."""
    start, kv = c["start"], c["kv"]
    s = np.searchsorted(start, rows, "right") - 1
    m, j = start[s + 1] - start[s], rows - start[s]
    return dict(c, q=q, table=c["table"][s], kv=np.maximum(kv[s] - m + j + 1, 0), start=np.arange(len(rows) + 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_prefix_attention_one_long_sequence_of_2048(dtype):
    """600000 rows of one sequence next to 2047 single ones, 64 KV heads: sequences x the longest one's rows x KV heads
    passes 2^31, the rows' own number does not."""
    H, hd, long = 64, 64, 600000
    kv, q = np.zeros(2048, np.int64), np.ones(2048, np.int64)
    kv[[0, 699, 700, 701, 2047]], q[700] = [3, 1, 150, 64, 65], long
    c = attn_case(dtype, (H, H, hd), 70, kv, np.zeros(2048, np.int64), seed=81)
    x = list(attn_inputs(c))
    rows = int(q.sum())
    x[0] = torch.empty((rows, H, hd), dtype=DT[dtype], device="cuda")
    torch.manual_seed(82)
    torch.cuda.manual_seed(82)
    for part in x[0].split(1 << 16):
        part.normal_()
    c["start"] = np.concatenate([[0], np.cumsum(q)])
    x[7] = i32(c["start"])
    out, lse = dfl().shared_prefix_attention(*x)
    pick = np.array([0, 1, 699, 700, 701, 700 + 127, 700 + 131072, 700 + 524287, 700 + 599849, 700 + 599850, 700 + 599999,
                     700 + long, 700 + long + 1, rows - 1])
    t = torch.from_numpy(pick).cuda()
    some = sampled_case(c, x[0][t].float().cpu().numpy(), pick)
    attn_check(some, (out[t], lse[t]), True)
    for part in lse.split(1 << 16):
        assert part.isfinite().all()
    del x, out, lse
    torch.cuda.empty_cache()


def test_shared_prefix_attention_graph_streams_and_workspaces():
    """Captured once, replayed with other lengths, pages and queries in place, while an eager call runs on a
    second stream with a workspace of its own."""
    c1 = attn_case("bf16", (8, 2, 128), 300, [100, 20, 64], [4, 4, 4], seed=61)
    c2 = attn_case("bf16", (8, 2, 128), 300, [10, 128, 65], [4, 4, 4], seed=62, extra_pages=2)
    x1, x2 = attn_inputs(c1), attn_inputs(c2)
    n = max(x1[1].shape[0], x2[1].shape[0])
    w = max(x1[5].shape[1], x2[5].shape[1])
    buf = [torch.zeros_like(x1[0]), torch.zeros((n, 2, 64, 128), dtype=torch.bfloat16, device="cuda"),
           torch.zeros((n, 2, 64, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(x1[3]), 300,
           torch.full((3, w), -1, dtype=torch.int32, device="cuda"), torch.zeros_like(x1[6]), x1[7]]

    def load(x):
        buf[0].copy_(x[0])
        for i in (1, 2):
            buf[i][: x[i].shape[0]] = x[i]
        buf[3].copy_(x[3])
        buf[5].fill_(-1)
        buf[5][:, : x[5].shape[1]] = x[5]
        buf[6].copy_(x[6])

    load(x1)
    out, lse = torch.zeros_like(x1[0]), torch.zeros((12, 8), device="cuda")
    dfl().shared_prefix_attention(*buf, out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dfl().shared_prefix_attention(*buf, out=out, lse=lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c, x in ((c2, x2), (c1, x1), (c2, x2)):
        load(x)
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            other = dfl().shared_prefix_attention(*x1)
        torch.cuda.synchronize()
        attn_check(c, (out, lse), True)
        attn_check(c1, other, True)


# ------------------------------------------------------------------------------------------------ logit rules
def rules_case(dtype, batch, rows, vocab, seed, hist=40, n_bias=5, n_masks=3, ld_extra=0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((4 * rng.standard_normal((batch * rows, vocab + ld_extra))).astype(np.float32)).to(DT[dtype])
    kw = {}
    if hist:
        lens = rng.integers(0, hist + 1, batch)
        kw.update(history=rng.integers(-2, max(2, min(vocab, hist // 2)) + 2, (batch, hist)), hist_lens=lens,
                  prompt_lens=(lens * rng.random(batch)).astype(int), repetition=1 + rng.random(batch),
                  presence=rng.random(batch) - 0.3, frequency=rng.random(batch) - 0.3)
        if rows > 1:
            kw["drafts"] = rng.integers(-1, min(vocab, 12) + 1, (batch, rows - 1))
    if n_bias:
        kw.update(bias_ids=rng.integers(-1, min(vocab, 3 * n_bias) + 1, (batch, n_bias)),
                  bias_values=10 * rng.standard_normal((batch, n_bias)))
    if n_masks:
        words = (vocab + 31) // 32
        masks = rng.integers(0, 2 ** 32, (n_masks, words), dtype=np.uint64).astype(np.uint32).view(np.int32)
        masks[0] = 0   # allows nothing
        kw.update(masks=masks, mask_index=rng.integers(-1, n_masks + 1, batch * rows))
    return x, kw


def rules_dev(kw):
    f32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.float32).cuda()  # noqa: E731
    return {k: f32(a) if k in ("repetition", "presence", "frequency", "bias_values") else i32(a) for k, a in kw.items()}


def rules_check(dtype, x, kw, rows, got):
    """At most four roundings to fp32 on top of exact arithmetic, each of an intermediate value no larger than
    |x| rep + |freq| c + |pres| + |bias| =: big, then one rounding to the type of the result."""
    kw = {k: (np.asarray(a, np.float32) if k in ("repetition", "presence", "frequency", "bias_values") else a)
          for k, a in kw.items()}
    host = x.float().numpy()
    want = serving.process_logits(host, rows, **kw)
    g = got.float().cpu().numpy().astype(np.float64)
    inf = np.isneginf(want)
    np.testing.assert_array_equal(np.isneginf(g), inf)
    same = host.astype(np.float64) == want
    np.testing.assert_array_equal(g[same], want[same])   # untouched tokens come through bit for bit
    hist = kw["history"].shape[1] if "history" in kw else 0
    big = np.abs(host).max() * 2 + (hist + rows) * 0.7 + 0.7 + (np.abs(kw["bias_values"]).max() if "bias_ids" in kw else 0)
    tol = 4 * 2.0 ** -24 * big + HALF[dtype] * np.abs(np.where(inf, 0, want))
    assert (np.abs(np.where(inf, 0, g) - np.where(inf, 0, want)) <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,rows,vocab,hist,n_bias,n_masks", [
    (1, 1, 1, 1, 1, 1), (1, 1, 31, 3, 0, 1), (2, 1, 32, 0, 4, 2), (3, 5, 33, 9, 2, 3), (2, 32, 1000, 700, 40, 5),
    (5, 4, 4097, 50, 5, 4), (1, 16, 5001, 3000, 7, 3), (7, 1, 3001, 60, 0, 0), (2, 2, 40000, 0, 0, 2), (3, 3, 70001, 100, 9, 2),
    (1, 2, 151936, 300, 16, 4), (160, 2, 1024, 30, 3, 5), (2, 1, 5000, 0, 0, 0)])
def test_process_logits(dtype, batch, rows, vocab, hist, n_bias, n_masks):
    x, kw = rules_case(dtype, batch, rows, vocab, seed=vocab + rows, hist=hist, n_bias=n_bias, n_masks=n_masks)
    d = rules_dev(kw)
    rules_check(dtype, x, kw, rows, dfl().process_logits(x.cuda(), rows_per_seq=rows, **d))
    y = x.cuda()
    assert dfl().process_logits(y, rows_per_seq=rows, out=y, **d) is y   # in place
    rules_check(dtype, x, kw, rows, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_process_logits_strides(dtype):
    """Rows padded to another stride in and out; what lies behind the vocabulary is left alone."""
    x, kw = rules_case(dtype, 3, 2, 1003, seed=5, ld_extra=21)
    src = x.cuda()
    out = torch.full((6, 1030), 3.0, dtype=src.dtype, device="cuda")
    dfl().process_logits(src[:, :1003], rows_per_seq=2, out=out[:, :1003], **rules_dev(kw))
    rules_check(dtype, x[:, :1003], kw, 2, out[:, :1003])
    assert (out[:, 1003:] == 3.0).all()
    dfl().process_logits(src[:, :1003], rows_per_seq=2, out=src[:, :1003], **rules_dev(kw))
    rules_check(dtype, x[:, :1003], kw, 2, src[:, :1003])
    assert torch.equal(src[:, 1003:].cpu(), x[:, 1003:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at,to,ld,ld_out", [(0, 0, 6151, 6151), (1, 1, 6152, 6152), (3, 3, 6157, 6165), (5, 5, 6150, 6150),
                                             (2, 0, 6152, 6152), (0, 0, 6151, 6153), (7, 7, 6145, 6145)])
def test_process_logits_wherever_rows_begin(dtype, at, to, ld, ld_out):
    """Logits and out begin `at` and `to` elements behind a 16-byte boundary, with any row stride; everything around
    the rows is left alone, and a row in place only where the rules change it."""
    rows, vocab = 4, 6145
    x, kw = rules_case(dtype, 2, rows, vocab, seed=at + ld, hist=60, n_bias=30, n_masks=3)
    buf = torch.full((8 * max(ld, ld_out) + 16,), 7.0, dtype=x.dtype, device="cuda")
    src = buf[at:at + 8 * ld].view(8, ld)[:, :vocab]
    src.copy_(x)
    dst_buf = torch.full_like(buf, 3.0)
    dst = dst_buf[to:to + 8 * ld_out].view(8, ld_out)[:, :vocab]
    d = rules_dev(kw)
    rules_check(dtype, x, kw, rows, dfl().process_logits(src, rows_per_seq=rows, out=dst, **d))
    around = torch.ones_like(dst_buf, dtype=torch.bool)
    around[to:to + 8 * ld_out].view(8, ld_out)[:, :vocab] = False
    assert (dst_buf[around] == 3.0).all()
    rules_check(dtype, x, kw, rows, dfl().process_logits(src, rows_per_seq=rows, out=src, **d))
    around[:] = True
    around[at:at + 8 * ld].view(8, ld)[:, :vocab] = False
    assert (buf[around] == 7.0).all()


def test_process_logits_special_values():
    """Infinities and NaN pass through the rules as IEEE arithmetic has it; a mask covers them."""
    x = torch.tensor([[float("nan"), float("inf"), float("-inf"), float("nan"), float("inf"), -0.0, 0.0, 1.0]])
    kw = dict(history=np.array([[0, 1, 2, 5, 6]]), hist_lens=[5], prompt_lens=[0], repetition=[2.0], frequency=[0.5],
              masks=np.array([[0b11100111]], np.int32), mask_index=[0])
    y = dfl().process_logits(x.cuda(), **rules_dev(kw))[0].cpu()
    assert y[0].isnan() and y[1] == float("inf") and y[2] == float("-inf")
    assert y[3] == float("-inf") and y[4] == float("-inf")
    assert y[5] == -0.5 and y[6] == -0.5 and y[7] == 1.0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_process_logits_repetition_over_its_range(dtype):
    """Positive logits over the repetition penalty, others times it.  A quotient has the rounding of a reciprocal, that of a
    product and that to the type (u = 2^-24: 2 u + u^2, and half a step of the type) and, where it is subnormal, up to a
    step of the format in place of each; a product is rounded once in fp32, bit for bit."""
    rep = torch.tensor([1.1, 3.0, 0.7, 2.0 ** -126, 1.3 * 2.0 ** -120, 2.0 ** 126, 1.9 * 2.0 ** 125, 49.0, 1.0, 2.0 ** -64])
    n = len(rep)
    g = torch.Generator().manual_seed(6)
    x = torch.randn((n, 2000), generator=g).to(DT[dtype])
    x[3:5] *= 2.0 ** -20
    x[:, 7] = float("inf")
    hist = torch.arange(2000, dtype=torch.int32).repeat(n, 1)
    lens = i32([2000] * n)
    for prompt in (lens, i32([0] * n)):   # seen in the prompt, or after it
        y = dfl().process_logits(x.cuda(), history=hist.cuda(), hist_lens=lens, prompt_lens=prompt, repetition=rep.cuda()).cpu()
        pos, f = x.float() > 0, x.float()
        times = (f * rep[:, None]).to(DT[dtype])
        assert torch.equal(y[~pos], times[~pos])
        want = x.double() / rep.double()[:, None]
        finite = pos & want.isfinite()
        assert (y[pos & ~finite] == float("inf")).all()
        half, step = (0.0, 2.0 ** -149) if dtype == "f32" else (2.0 ** -8, 2.0 ** -133)
        tol = (2 * 2.0 ** -24 + 2.0 ** -48 + half) * want.abs() * (1 + 2.0 ** -8) + 2 * step * (want.abs() < 2.0 ** -126)
        assert ((y.double() - want).abs()[finite] <= tol[finite]).all()


def test_process_logits_duplicates_and_padding():
    """The same id many times in the history, the drafts and the bias list (its last entry counts)."""
    x = torch.zeros(4, 64)
    kw = dict(history=np.full((1, 5000), 9), hist_lens=[7000], prompt_lens=[1000], drafts=np.full((1, 3), 9),
              frequency=[0.25], presence=[1.0], bias_ids=np.array([[9] * 40 + [-1, 64, 9, 70]]),
              bias_values=np.arange(44)[None])
    y = dfl().process_logits(x.cuda(), rows_per_seq=4, **rules_dev(kw)).cpu()
    want = torch.tensor([42.0 - 1.0 - 0.25 * (4000 + j) for j in range(4)])
    assert torch.equal(y[:, 9], want) and (y[:, :9] == 0).all() and (y[:, 10:] == 0).all()


def test_process_logits_on_a_side_stream_and_in_a_graph():
    x, kw = rules_case("f32", 4, 3, 6000, seed=77)
    d = rules_dev(kw)
    src, out = x.cuda(), torch.empty(12, 6000, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y = dfl().process_logits(src, rows_per_seq=3, **d)
    side.synchronize()
    rules_check("f32", x, kw, 3, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dfl().process_logits(src, rows_per_seq=3, out=out, **d)
    x2, kw2 = rules_case("f32", 4, 3, 6000, seed=78)
    src.copy_(x2)
    for k, t in rules_dev(kw2).items():
        d[k].copy_(t)
    g.replay()
    torch.cuda.synchronize()
    rules_check("f32", x2, kw2, 3, out)


# ------------------------------------------------------------------------------------------- refusals, chain
def test_the_bindings_refuse():
    m = dfl()
    c = attn_case("bf16", (8, 2, 128), 64, [5], [1], seed=1)
    q, k, v, pre, n, table, kv, start = x = attn_inputs(c)
    for bad in ((q.half(),) + x[1:], (q, k.float()) + x[2:], (q[:, :7],) + x[1:], (q.cpu(),) + x[1:],
                (q, k, v, pre[:0], n, table, kv, start), (q, k, v, None, n, table, kv, start),
                (q, k, v, pre, n, table.long(), kv, start), (q, k, v, pre, n, table, kv, start[:1]),
                (q.transpose(1, 2).contiguous().transpose(1, 2),) + x[1:]):
        with pytest.raises((ValueError, m.DFlashError)):
            m.shared_prefix_attention(*bad)
    with pytest.raises(ValueError, match="gradient"):
        m.shared_prefix_attention(q.clone().requires_grad_(), *x[1:])
    with torch.no_grad():
        m.shared_prefix_attention(q.clone().requires_grad_(), *x[1:])
    with pytest.raises(m.DFlashError, match="workspace"):
        m.shared_prefix_attention(*x, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(m.DFlashError, match="scale"):
        m.shared_prefix_attention(*x, scale=0.0)
    z = torch.zeros(4, 50, device="cuda")
    for kw in (dict(rows_per_seq=3), dict(rows_per_seq=33), dict(drafts=i32([[1]])), dict(repetition=z[:, 0]),
               dict(masks=i32([[1]]), mask_index=i32([0, 0, 0, 0])), dict(bias_ids=i32([[1]] * 4)),
               dict(out=z.t()), dict(history=i32([[1]]), hist_lens=i32([1]), prompt_lens=i32([1]))):
        with pytest.raises(ValueError):
            m.process_logits(z, **kw)
    with pytest.raises(ValueError):
        m.kv_tables(i32([1]), i32([1]), i32([[0]]))
    with pytest.raises(ValueError):
        m.kv_tables(i32([1]), i32([1]), i32([[0]]), i32([1]), rows=1)
    for bad in (dict(base_pos=1 << 40), dict(scratch_page=0.5)):
        with pytest.raises(ValueError, match="integer"):
            m.kv_tables(i32([1]), i32([1]), i32([[0]]), rows=1, **bad)
    with pytest.raises(ValueError, match="integer"):
        m.shared_prefix_attention(*x[:4], 5.0, *x[5:])


def test_autograd_sees_what_the_operators_write():
    """Outputs that require a gradient and inputs with a tangent are refused; a tensor that autograd has saved and that a
    call then writes over stops the backward pass, as any other write in place does."""
    m = dfl()
    c = attn_case("f32", (8, 2, 128), 64, [5], [1], seed=1)
    x = attn_inputs(c)
    out, lse = torch.zeros_like(x[0]), torch.zeros(1, 8, device="cuda")
    for kw in (dict(out=out.clone().requires_grad_()), dict(out=out, lse=lse.clone().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            m.shared_prefix_attention(*x, **kw)
        with torch.no_grad():
            m.shared_prefix_attention(*x, **kw)
    z = torch.zeros(2, 50, device="cuda")
    with pytest.raises(ValueError, match="gradient"):
        m.process_logits(z, out=z.clone().requires_grad_())
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            m.process_logits(torch.autograd.forward_ad.make_dual(z, torch.ones_like(z)))

    w = torch.ones(2, 50, device="cuda", requires_grad=True)
    table = i32([[7, 7]])

    def process(t):
        m.process_logits(t, bias_ids=i32([[3], [4]]), bias_values=torch.ones(2, 1, device="cuda"), out=t)

    def attend(t):
        m.shared_prefix_attention(*x, out=t)

    for write, t in ((process, z.clone()), (attend, out.clone())):
        y = (t * torch.ones_like(t, requires_grad=True)).sum()   # saves t
        write(t)
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
    y = w.index_select(1, table[0]).sum()   # saves the indices
    m.kv_tables(i32([3]), i32([1]), table, i32([9]), i32([0]), rows=1, table_out=table)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    with torch.inference_mode():
        t = torch.zeros(2, 50, device="cuda")
        process(t)
    process(t)


def test_an_empty_batch_of_rows():
    c = attn_case("bf16", (8, 2, 128), 64, [5], [0], seed=1)
    out, lse = dfl().shared_prefix_attention(*attn_inputs(c))
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_step_of_all_three(dtype):
    """A serving step as it is used: pages and slots from the lengths, the new tokens' keys and values
    scattered by slot, attention behind the prefix, then a head and its logit rules."""
    rng = np.random.default_rng(12)
    H, hkv, hd, prefix, V = 8, 2, 128, 90, 777
    kv, new = np.array([0, 60, 128, 7]), np.array([5, 5, 5, 5])
    c = attn_case(dtype, (H, hkv, hd), prefix, kv, new, seed=13, extra_pages=12, stale=0.0)
    q, k, v, pre, n, table, kvd, _ = attn_inputs(c)
    table = torch.cat([table, table[:, :1]], 1)
    used_pages = set(c["pre"].tolist()) | {int(p) for s in range(4) for p in c["table"][s, : -(-kv[s] // 64)]}
    free = [p for p in range(c["k"].shape[0]) if p not in used_pages]
    t = dfl().kv_tables(kvd, i32(new), table, i32(free), i32([0]), rows=20, base_pos=prefix)
    nk, nv = (torch.from_numpy(rng.standard_normal((20, hkv, hd))).to(q.dtype).cuda() for _ in range(2))
    page, at = t.slots // 64, t.slots % 64
    k[page, :, at], v[page, :, at] = nk, nv
    out, lse = dfl().shared_prefix_attention(q, k, v, pre, n, t.table, kvd + i32(new), t.q_start)
    assert int(t.status) == 0
    c.update(k=k.float().cpu().numpy(), v=v.float().cpu().numpy(), table=t.table.cpu().numpy(), kv=kv + new)
    attn_check(c, (out, lse), True)
    head = torch.from_numpy(rng.standard_normal((V, H * hd)).astype(np.float32)).cuda()
    logits = out.float().view(20, -1) @ head.t()
    kw = rules_case("f32", 4, 5, V, seed=3)[1]
    got = dfl().process_logits(logits, rows_per_seq=5, **rules_dev(kw))
    rules_check("f32", logits.cpu(), kw, 5, got)
