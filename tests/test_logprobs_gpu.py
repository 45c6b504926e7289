"""Log probabilities of tokens and their gradient on the GPU against fp64, at the vocabularies, strides, masks and values
where they can go wrong."""
import numpy as np
import pytest
import torch

from oracle import trees

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
U = 2.0 ** -24


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


def rows_of(dtype, rows, vocab, seed, scale=3.0):
    x = scale * torch.randn((rows, vocab), generator=torch.Generator().manual_seed(seed))
    return x.to(DT[dtype])


def tokens_of(x, n, seed):
    """Likely and unlikely tokens, the same one twice and padding."""
    rng = np.random.default_rng(seed)
    rows, vocab = x.shape
    t = rng.integers(0, vocab, (rows, n))
    t[:, 0] = host(x.float()).argmax(1) if rows else 0
    if n > 2:
        t[:, 1], t[:, 2] = t[:, 0], rng.choice([-1, vocab, 0, vocab - 1], rows)
    return t


def bounds(x, temperature):
    """(relative error of the sum of exponentials, mean |z|, mean z^2) a row, z = (x - max) / T.
    Of a term: z is off by 3 u |z| (difference, inverse temperature, product), 2^z's function by 2^-22; a running maximum's
    moves add up to the range of z and one exponential a tile of 4096 tokens; a sum of n terms is off by n u, where a
    thread adds vocab / 256 at most and the threads' are joined in 64 steps; terms below e^-100 count for nothing."""
    x = x.astype(np.float64)
    x = np.where(np.isnan(x) | np.isposinf(x), -np.inf, x)  # (rows of NaN are compared as they are, whatever the bound)
    best = x.max(1, keepdims=True)
    z = (x - np.where(np.isfinite(best), best, 0)) / temperature
    p = np.exp(z)
    p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
    z = np.where(np.isfinite(z), z, 0)
    spread = np.minimum(np.abs(z).max(1), 100.0)
    rel = 3 * U * spread + (x.shape[1] / 4096 + 8) * 2.0 ** -21 + (x.shape[1] / 256 + 64) * U
    z = np.abs(np.maximum(z, -700))
    return rel, (p * z).sum(1), (p * z * z).sum(1)


def check(x, tokens, top, got, temperature=1.0):
    x = host(x.float())
    logprobs, ranks, entropy, lse, top_ids, top_logprobs = trees.token_logprobs(x, tokens, top, temperature)
    rel, a1, a2 = bounds(x, temperature)

    def near(g, w, tol, name):
        g = host(g).astype(np.float64)
        fine = np.isfinite(w)
        np.testing.assert_array_equal(np.where(fine, 0, g), np.where(fine, 0, w), err_msg=name)
        err = np.abs(np.where(fine, g, 0) - np.where(fine, w, 0))
        assert (err <= tol).all(), (name, float((err / tol).max()))

    best = np.where(np.isfinite(x), x, -np.inf).max(1)
    best = np.abs(np.where(np.isfinite(best), best, 0)) / temperature
    log_l = rel + 4 * U * np.log(x.shape[1] + 1)
    fin = lambda a: np.abs(np.where(np.isfinite(a), a, 0))  # noqa: E731
    near(got.lse, lse, log_l + 3 * U * best + U * fin(lse), "lse")
    near(got.entropy, entropy, log_l + 2 * a1 * rel + 3 * U * a2 + 8 * U * a1, "entropy")
    near(got.logprobs, logprobs.reshape(got.logprobs.shape), (log_l[:, None] + 5 * U * (fin(logprobs) + 1)).reshape(got.logprobs.shape),
         "logprobs")
    np.testing.assert_array_equal(host(got.ranks), ranks.reshape(got.ranks.shape))
    if top:
        np.testing.assert_array_equal(host(got.top_ids), top_ids)
        near(got.top_logprobs, top_logprobs, log_l[:, None] + 5 * U * (fin(top_logprobs) + 1), "top")
    else:
        assert got.top_ids is None and got.top_logprobs is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,n,top", [(1, 1, 1, 1), (3, 2, 2, 5), (1, 31, 1, 32), (2, 33, 3, 32), (5, 1000, 1, 0), (2, 4096, 4, 20),
                                              (3, 4101, 1, 20), (1, 151936, 1, 20), (4, 128257, 8, 5), (300, 5003, 2, 3), (2500, 700, 1, 4)])
def test_token_logprobs(dtype, rows, vocab, n, top):
    x = rows_of(dtype, rows, vocab, seed=rows + vocab)
    t = tokens_of(x, n, seed=n)
    check(x, t, top, dfl().token_logprobs(x.cuda(), i32(t), top=top))


def test_token_logprobs_one_dimension_temperature_and_no_rows():
    x = rows_of("f32", 6, 3001, seed=1)
    t = tokens_of(x, 1, seed=2)
    for temperature in (0.05, 0.7, 30.0):
        got = dfl().token_logprobs(x.cuda(), i32(t[:, 0]), top=7, temperature=temperature)
        assert got.logprobs.shape == got.ranks.shape == (6,)
        check(x, t, 7, got, temperature)
    got = dfl().token_logprobs(torch.zeros((0, 50), device="cuda"), i32(np.zeros((0, 2))), top=3)
    assert got.logprobs.shape == (0, 2) and got.top_ids.shape == (0, 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset,ld", [(0, 5003), (1, 5004), (3, 5007), (0, 5120), (8, 5016)])
def test_token_logprobs_of_rows_that_begin_anywhere(dtype, offset, ld):
    x = rows_of(dtype, 5, 5003, seed=3)
    store = torch.full((offset + 5 * ld + 64,), 99.0, dtype=DT[dtype], device="cuda")
    view = store.as_strided((5, 5003), (ld, 1), offset)
    view.copy_(x)
    t = tokens_of(x, 3, seed=4)
    got = dfl().token_logprobs(view, i32(t), top=11)
    check(x, t, 11, got)
    # the gradient, between views that lie alike and ones that do not
    rng = np.random.default_rng(5)
    g, h = rng.standard_normal((5, 3)).astype(np.float32), rng.standard_normal(5).astype(np.float32)
    want = trees.token_logprobs_grad(host(x.float()), t, g, h)
    for off, l in ((offset, ld), (offset + 2, ld), (offset, 5200)):
        out = torch.full((off + 5 * l + 64,), 55.0, dtype=DT[dtype], device="cuda")
        o = out.as_strided((5, 5003), (l, 1), off)
        back = dfl().token_logprobs_grad(view, i32(t), got.lse, torch.from_numpy(g).cuda(), entropy=got.entropy,
                                         grad_entropy=torch.from_numpy(h).cuda(), out=o)
        grad_check(dtype, x, t, g, h, back, want)
        keep = torch.ones_like(out, dtype=torch.bool)
        keep.as_strided((5, 5003), (l, 1), off).fill_(False)
        assert (out[keep] == 55.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["ascending", "descending", "equal", "two values", "zeros of both signs", "late peak", "blocks"])
@pytest.mark.parametrize("vocab", [5000, 70001])
def test_token_logprobs_in_any_order(dtype, kind, vocab):
    """Rows in the orders that fill the list of candidates, and ties: the lower id first."""
    v = np.arange(vocab)
    x = {"ascending": v * (20.0 / vocab), "descending": v * (-20.0 / vocab), "equal": np.full(vocab, 1.25), "two values": (v % 3 == 1) * 1.0,
         "zeros of both signs": np.where(v % 2, -0.0, 0.0), "late peak": np.where(v < vocab - 40, 0.0, v * 1e-3),
         "blocks": (v // 300) * 0.25}[kind]
    x = torch.from_numpy(np.stack([x, np.roll(x, 17)])).to(DT[dtype])
    t = np.array([[0, vocab - 1, vocab // 2], [5, 16, 17]])
    for top in (1, 20, 32):
        check(x, t, top, dfl().token_logprobs(x.cuda(), i32(t), top=top))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_logprobs_of_masked_rows(dtype):
    """-inf for all but a few, one and no tokens; the type's lowest value; infinities and NaN."""
    vocab = 9000
    low = torch.finfo(DT[dtype]).min
    x = rows_of(dtype, 10, vocab, seed=6).float()
    some = x[0].clone()
    x[0], x[1], x[2] = float("-inf"), float("-inf"), float("-inf")
    x[0, 4000:4005] = some[4000:4005]
    x[1, vocab - 1] = -7.0
    x[3, :] = low
    x[4, 10:] = low
    x[5, 77] = float("inf")
    x[6, 8191] = float("nan")
    x[7, :] = float("nan")
    x[8, 1:] = float("-inf")
    x = x.to(DT[dtype])
    t = np.array([[4001, 3, -1], [vocab - 1, 0, 5], [1, 2, vocab], [8, 0, 8], [2, 11, 9], [77, 1, -1], [0, 8191, 3], [0, 1, 2], [0, 0, 1], [4, 5, 6]])
    got = dfl().token_logprobs(x.cuda(), i32(t), top=9)
    rows = np.array([r for r in range(10) if r != 3])
    pick = type(got)(*(y[torch.from_numpy(rows).cuda()] for y in got))
    check(x[torch.from_numpy(rows)], t[rows], 9, pick)
    # a row of the lowest value alone is uniform (its lse is that value: ln vocab is far below its last digit)
    assert float(got.lse[3]) == float(low) and abs(float(got.entropy[3]) - np.log(vocab)) < 1e-4
    np.testing.assert_allclose(host(got.logprobs[3]), -np.log(vocab), atol=1e-4)
    assert host(got.top_ids[3]).tolist() == list(range(9)) and host(got.ranks[3]).tolist() == [8, 0, 8]
    assert host(got.top_ids[2]).tolist() == [-1] * 9 and float(got.entropy[2]) == 0 and np.isneginf(float(got.lse[2]))


def test_token_logprobs_twice_and_in_a_graph():
    """The same bits each time, two captured calls on one stream, and another stream beside them."""
    x = rows_of("bf16", 40, 128256, seed=9).cuda()
    t = i32(tokens_of(x.cpu(), 2, seed=1))
    want = dfl().token_logprobs(x, t, top=20)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = dfl().token_logprobs(x, t, top=20)
        b = dfl().token_logprobs(x, t, top=20)
    with torch.cuda.stream(s):
        c = dfl().token_logprobs(x, t, top=20)
    g.replay()
    torch.cuda.synchronize()
    for got in (a, b, c):
        assert all(torch.equal(p, q) for p, q in zip(got, want))


# ------------------------------------------------------------------------------------------------------ gradient
def grad_check(dtype, x, tokens, g, h, got, want, temperature=1.0):
    """ln p = x / T - lse is off by one rounding of each and of lse before (u each), and by the bound of lse itself; p's
    function by 2^-22; the sums of a row's g by n u; the result is rounded once to its type."""
    x = host(x.float()).astype(np.float64)
    rel, a1, _ = bounds(x, temperature)
    best = np.where(np.isfinite(x.max(1, keepdims=True)), x.max(1, keepdims=True), 0)
    z = (x - best) / temperature
    lse = np.log(np.maximum(np.exp(z).sum(1, keepdims=True), 1e-300))
    logp = np.where(np.isfinite(z), z - lse, 0)
    p = np.where(np.isfinite(z), np.exp(z - lse), 0)
    off = (rel + 4 * U * 12)[:, None] + U * (4 * np.abs(best / temperature + lse) + 4 * np.abs(np.where(np.isfinite(z), z, 0))) + 2.0 ** -22
    off = np.minimum(off, 1.0)
    real = (tokens >= 0) & (tokens < x.shape[1])
    G = np.abs(np.where(real, g, 0)).sum(1, keepdims=True)
    H = np.abs(h)[:, None]
    tol = p * (G * (off + 64 * U) + H * (np.abs(logp) + a1[:, None] + 20) * (2 * off + 8 * U)) + 64 * U * G * (want != 0)
    tol = tol / temperature + HALF[dtype] * np.abs(want) * (1 + 8 * U) + 4 * U * np.abs(want) + 1e-30
    err = np.abs(host(got.float()).astype(np.float64) - want)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,n,entropy,temperature", [(1, 1, 1, True, 1.0), (2, 7, 3, True, 1.0), (3, 4099, 1, False, 1.0),
                                                              (40, 5000, 32, True, 0.6), (2, 128257, 8, True, 1.0), (700, 900, 1, False, 2.0)])
def test_token_logprobs_grad(dtype, rows, vocab, n, entropy, temperature):
    x = rows_of(dtype, rows, vocab, seed=rows)
    t = tokens_of(x, n, seed=3)
    rng = np.random.default_rng(4)
    g = rng.standard_normal((rows, n)).astype(np.float32)
    h = rng.standard_normal(rows).astype(np.float32) if entropy else np.zeros(rows, np.float32)
    f = dfl().token_logprobs(x.cuda(), i32(t), temperature=temperature)
    kw = dict(entropy=f.entropy, grad_entropy=torch.from_numpy(h).cuda()) if entropy else {}
    got = dfl().token_logprobs_grad(x.cuda(), i32(t), f.lse, torch.from_numpy(g).cuda(), temperature=temperature, **kw)
    want = trees.token_logprobs_grad(host(x.float()), t, g, h, temperature)
    grad_check(dtype, x, t, g, h, got, want, temperature)
    y = x.cuda().clone()
    back = dfl().token_logprobs_grad(y, i32(t), f.lse, torch.from_numpy(g).cuda(), temperature=temperature, out=y, **kw)
    assert back is y and torch.equal(y, got)  # in place


def test_token_logprobs_grad_against_differences():
    """Of the forward operator itself: a central difference of step d is off by d^2 / 6 times the third derivative (below 2 for
    these, whose gradients by any logit are below one) and by the rounding of the loss over d."""
    x = rows_of("f32", 1, 50, seed=12, scale=1.0).cuda()
    t, g, h = i32([[3, 40, 3]]), torch.tensor([[0.5, -0.25, 0.125]], device="cuda"), torch.tensor([0.5], device="cuda")

    def loss(y):
        f = dfl().token_logprobs(y, t)
        return float((f.logprobs.double() * g).sum() + (f.entropy.double() * h).sum())

    f = dfl().token_logprobs(x, t)
    got = host(dfl().token_logprobs_grad(x, t, f.lse, g, entropy=f.entropy, grad_entropy=h))[0]
    d = 2.0 ** -6
    for v in range(50):
        up, down = x.clone(), x.clone()
        up[0, v] += d
        down[0, v] -= d
        assert abs((loss(up) - loss(down)) / (2 * d) - got[v]) < 2 * d * d / 6 + 8 * 2.0 ** -21 / d


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_logprobs_grad_of_masked_and_padded_rows(dtype):
    vocab = 6000
    x = rows_of(dtype, 6, vocab, seed=13).float()
    x[0, 50:] = float("-inf")
    x[1] = float("-inf")
    x[2, 9] = float("nan")
    x[3, 9] = float("nan")
    x[4, ::2] = torch.finfo(DT[dtype]).min
    x = x.to(DT[dtype])
    t = np.array([[3, 60], [7, -1], [5, 6], [-1, vocab], [1, 0], [-1, 2]])
    g = np.array([[1.0, 0.5], [2.0, 3.0], [1.0, 1.0], [4.0, 5.0], [1.0, -1.0], [7.0, 0.0]], np.float32)
    h = np.array([0.5, 0.5, 0.0, 0.0, -1.0, 0.0], np.float32)
    f = dfl().token_logprobs(x.cuda(), i32(t))
    got = dfl().token_logprobs_grad(x.cuda(), i32(t), f.lse, torch.from_numpy(g).cuda(), entropy=f.entropy, grad_entropy=torch.from_numpy(h).cuda())
    for r in (0, 1, 4, 5):
        want = trees.token_logprobs_grad(host(x[r:r + 1].float()), t[r:r + 1], g[r:r + 1], h[r:r + 1])
        grad_check(dtype, x[r:r + 1], t[r:r + 1], g[r:r + 1], h[r:r + 1], got[r:r + 1], want)
    assert torch.isnan(got[2]).all()                               # a row that holds NaN
    assert (got[3] == 0).all() and (got[5] == 0).all()             # rows without a gradient, whatever they hold
    assert float(got[1, 7]) == 2.0 and float(got[1].float().abs().sum()) == 2.0


def test_a_loss_and_its_gradient():
    """A policy-gradient step on a block of sampled tokens (log probabilities, their alternatives among the tokens, an entropy
    bonus): the operators' gradient is that of the same loss in fp64."""
    x = rows_of("f32", 16, 2000, seed=14).cuda()
    t = i32(tokens_of(x.cpu(), 1, seed=5))
    f = dfl().token_logprobs(x, t, top=4)
    names = torch.cat([t, f.top_ids], 1)
    adv = torch.randn((16, 5), generator=torch.Generator().manual_seed(1)).cuda() / 16
    f2 = dfl().token_logprobs(x, names)
    bonus = torch.full((16,), 0.01, device="cuda")
    got = dfl().token_logprobs_grad(x, names, f2.lse, adv, entropy=f2.entropy, grad_entropy=bonus)
    y = x.double().requires_grad_()
    logp = torch.log_softmax(y, 1)
    loss = (logp.gather(1, names.long().clamp(min=0)) * (names >= 0) * adv).sum() + 0.01 * -(logp.exp() * logp).sum()
    loss.backward()
    grad_check("f32", x.cpu(), host(names), host(adv), host(bonus), got, host(y.grad))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 3.0])
def test_token_logprobs_grad_of_rows_of_any_size(dtype, temperature):
    """From lse_parts: a row all of the type's lowest value is uniform, and rows far from 0 are as exact as others."""
    vocab = 5000
    x = rows_of(dtype, 6, vocab, seed=15).float()
    x[0] = torch.finfo(DT[dtype]).min
    x[1] += 1e5 if dtype == "f32" else 500.0
    x[2] = float("-inf")
    x[2, 5] = torch.finfo(DT[dtype]).min
    x[3] = float("-inf")
    x[4, 9] = float("nan")
    x = x.to(DT[dtype])
    t = np.array([[3, 60], [7, -1], [5, 6], [2, vocab - 1], [1, 0], [4, 2]])
    rng = np.random.default_rng(3)
    g, h = rng.standard_normal((6, 2)).astype(np.float32), rng.standard_normal(6).astype(np.float32)
    two = torch.empty((6, 2), device="cuda")
    f = dfl().token_logprobs(x.cuda(), i32(t), temperature=temperature, lse_parts=two)
    got = dfl().token_logprobs_grad(x.cuda(), i32(t), two, torch.from_numpy(g).cuda(), entropy=f.entropy, grad_entropy=torch.from_numpy(h).cuda(),
                                    temperature=temperature)
    assert torch.isnan(got[4]).all() and torch.isnan(two[4]).all()
    rows = [0, 1, 2, 3, 5]
    xs = host(x.float())[rows]
    best = xs.max(1)
    np.testing.assert_array_equal(host(two)[rows, 0], best)
    y = np.where(np.isneginf(xs), -np.inf, xs.astype(np.float64) - np.where(np.isneginf(best), 0, best)[:, None])  # (rows from 0: the same law)
    want = trees.token_logprobs_grad(y, t[rows], g[rows], h[rows], temperature)
    grad_check(dtype, torch.from_numpy(np.where(np.isneginf(y), -np.inf, np.maximum(y, -1e30))), t[rows], g[rows], h[rows], got[rows], want, temperature)


def test_parts_of_lse_make_lse():
    x = rows_of("f32", 4, 3001, seed=16)
    t = tokens_of(x, 1, seed=2)
    two = torch.empty((4, 2), device="cuda")
    f = dfl().token_logprobs(x.cuda(), i32(t), temperature=0.7, lse_parts=two)
    want = host(two).astype(np.float64)
    want = want[:, 0] * np.float32(1 / 0.7) + want[:, 1]
    # one rounding
    np.testing.assert_allclose(host(f.lse), want, rtol=U, atol=0)
    with pytest.raises(ValueError, match="lse_parts"):
        dfl().token_logprobs(x.cuda(), i32(t), lse_parts=torch.empty((4, 1), device="cuda"))
    with pytest.raises(ValueError, match="lse_parts"):
        dfl().token_logprobs_grad(x.cuda(), i32(t), torch.empty((4, 3), device="cuda"), f.logprobs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 7])
@pytest.mark.parametrize("vocab", [30, 157, 4099, 9001])
def test_ranks_of_masked_tokens_anywhere(dtype, n, vocab):
    """Tokens at -inf before the first aligned vector, behind the last one and at the ends of the CTAs' slices, behind elements
    that are none."""
    for offset in (0, 1, 5):
        x = torch.full((vocab, vocab + 9), float("-inf"))
        x[:, :vocab] = rows_of("f32", vocab, vocab, seed=vocab)
        x[torch.rand(x.shape, generator=torch.Generator().manual_seed(offset)) < 0.9] = float("-inf")
        x = x[:min(vocab, 200)].to(DT[dtype])
        rows = len(x)
        t = np.random.default_rng(n).integers(0, vocab, (rows, n))
        t[:, 0] = vocab - 1 - np.arange(rows) % min(vocab, 9)
        t[:, -1] = np.arange(rows) % vocab
        y = torch.empty(rows * (vocab + 9) + 5, dtype=DT[dtype], device="cuda")[offset:offset + rows * (vocab + 9)].view(rows, vocab + 9)
        y.copy_(x)
        got = dfl().token_logprobs(y[:, :vocab], i32(t))
        z, ids = host(x.float())[:, None, :vocab], np.arange(vocab)
        xt = np.take_along_axis(z[:, 0], t, 1)[:, :, None]
        np.testing.assert_array_equal(host(got.ranks), ((z > xt) | ((z == xt) & (ids < t[:, :, None]))).sum(2))


def test_ranks_and_order_are_those_of_the_logits_themselves():
    """Neighbours of 1e5 that a product with 1 / T rounded to fp32 would make equal, and logits whose product is beyond fp32."""
    step = 2.0 ** -7  # of fp32 at 1e5
    x = np.full((2, 6000), 9e4, np.float32)
    x[0, [10, 4000, 20, 5999]] = 1e5 + step * np.array([0, 1, 2, 3])
    assert len(set((x[0, [10, 4000, 20, 5999]] * np.float32(1 / 3.0)).tolist())) < 4
    x[1, :50], x[1, 50:] = 2e38, -2e38
    t = np.array([[10, 4000, 20], [49, 0, 60]])
    got = dfl().token_logprobs(torch.from_numpy(x).cuda(), i32(t), top=4, temperature=3.0)
    assert host(got.ranks).tolist() == [[3, 2, 1], [49, 0, 60]]
    assert host(got.top_ids).tolist() == [[5999, 20, 4000, 10], [0, 1, 2, 3]]
    got = dfl().token_logprobs(torch.from_numpy(x[1:]).cuda(), i32(t[1:]), top=4, temperature=0.25)
    assert np.isposinf(host(got.lse)).all() and abs(float(got.entropy) - np.log(50)) < 1e-5
    np.testing.assert_allclose(host(got.logprobs)[0, :2], -np.log(50), rtol=1e-6)
    assert np.isneginf(host(got.logprobs)[0, 2])  # (-4e38 / 0.25 lies beyond fp32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("temperature", [0.7, 3.0, 2.0 ** -20, 2.0 ** 20])
def test_log_probabilities_of_rows_far_from_zero(dtype, temperature):
    """The difference to the largest logit comes before the scale: check()'s bound of logprobs has no term of the logits' size."""
    x = rows_of("f32", 4, 9001, seed=21)
    x[1] += 1e5 if dtype == "f32" else 500.0
    x[2] -= 1e6 if dtype == "f32" else 900.0
    x[3] *= 1e-3
    x = x.to(DT[dtype])
    t = tokens_of(x, 3, seed=22)
    two = torch.empty((4, 2), device="cuda")
    f = dfl().token_logprobs(x.cuda(), i32(t), top=6, temperature=temperature, lse_parts=two)
    check(x, t, 6, f, temperature)
    np.testing.assert_array_equal(host(two)[:, 0], host(x.float()).max(1))
    # and the gradient from the parts, whose law is that of the rows from 0
    rng = np.random.default_rng(5)
    g, h = rng.standard_normal((4, 3)).astype(np.float32), rng.standard_normal(4).astype(np.float32)
    got = dfl().token_logprobs_grad(x.cuda(), i32(t), two, torch.from_numpy(g).cuda(), entropy=f.entropy, grad_entropy=torch.from_numpy(h).cuda(),
                                    temperature=temperature)
    y = host(x.float()).astype(np.float64)
    y -= y.max(1, keepdims=True)
    grad_check(dtype, torch.from_numpy(y), t, g, h, got, trees.token_logprobs_grad(y, t, g, h, temperature), temperature)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 151936), (7, 33003), (300, 4099), (5, 40)])
@pytest.mark.parametrize("n", [5, 9, 16, 31, 32])
def test_ranks_of_up_to_32_tokens(dtype, rows, vocab, n):
    """Likely and unlikely ones, tokens at -inf, the same token twice, padding among them, in every lane."""
    x = rows_of("f32", rows, vocab, seed=vocab + n)
    x[::2][torch.rand(x[::2].shape, generator=torch.Generator().manual_seed(n)) < 0.5] = float("-inf")
    x = x.to(DT[dtype]).cuda()
    rng = np.random.default_rng(n)
    t = rng.integers(0, vocab, (rows, n))
    likely = host(x.float().topk(min(40, vocab), 1)[1])
    for r in range(rows):
        some = rng.permutation(n)[:n // 2]
        t[r, some] = rng.choice(likely[r], len(some))
    t[:, n // 3], t[::3, n - 1] = t[:, 0], -1
    t[1::3, n // 2] = vocab
    got = dfl().token_logprobs(x, i32(t), top=3)
    z, ids = x.double(), torch.arange(vocab, device="cuda")
    for i in range(n):
        real = (t[:, i] >= 0) & (t[:, i] < vocab)
        at = torch.from_numpy(np.where(real, t[:, i], 0)).cuda()[:, None]
        xt = z.gather(1, at)
        want = host(((z > xt) | ((z == xt) & (ids < at))).sum(1))
        np.testing.assert_array_equal(host(got.ranks)[:, i], np.where(real, want, -1))
        np.testing.assert_array_equal(host(got.logprobs)[~real, i], 0)


def test_rows_that_begin_behind_2_31_elements():
    rows, vocab, ld = 10, 5000, (1 << 28) + 8
    store = [torch.empty((rows - 1) * ld + vocab, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x, out = (s.as_strided((rows, vocab), (ld, 1)) for s in store)
    y = rows_of("bf16", rows, vocab, seed=30)
    x.copy_(y)
    out.fill_(7.0)
    t = tokens_of(y, 3, seed=31)
    got = dfl().token_logprobs(x, i32(t), top=5)
    check(y, t, 5, got)
    rng = np.random.default_rng(32)
    g, h = rng.standard_normal((rows, 3)).astype(np.float32), rng.standard_normal(rows).astype(np.float32)
    want = trees.token_logprobs_grad(host(y.float()), t, g, h)
    kw = dict(entropy=got.entropy, grad_entropy=torch.from_numpy(h).cuda())
    dfl().token_logprobs_grad(x, i32(t), got.lse, torch.from_numpy(g).cuda(), out=out, **kw)
    grad_check("bf16", y, t, g, h, out, want)
    dfl().token_logprobs_grad(x, i32(t), got.lse, torch.from_numpy(g).cuda(), out=x, **kw)  # in place
    assert torch.equal(x, out)
