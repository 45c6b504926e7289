"""Sessions behind one shared prefix (dflash_prefill_shared), with logit rules
(dflash_set_logit_rules) and with token masks (dflash_set_token_masks), against
the fp64 oracle on the whole prompts / the rules applied token by token."""
import numpy as np
import pytest

import synth
from synth import configs
from oracle import model as om, serving, spec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_ctx_gb300 import build
    build.build()


def _session(w, **kw):
    from block_diffusion_speculative_ctx_gb300 import Session
    return Session(w, **kw)


def _prompts(w, prefix_len, lens, seed):
    toks = synth.uniform_ints(seed, 0x70, prefix_len + sum(lens), w.vocab).astype(np.int32)
    own, at = [], prefix_len
    for n in lens:
        own.append(toks[at:at + n])
        at += n
    return toks[:prefix_len], own


def _rel(a, b):
    return float(np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-30))


# The bounds are those of the parity tests: fp32 logits 1e-3 and caches 1e-5; bf16 logits 5e-2 (tokens equal
# but where the oracle's top two lie closer), caches 2e-2.
@pytest.mark.parametrize("name,prefix_len,lens,schedule", [
    ("tiny_f32_b3", 64, (7, 1, 30), None),            # a prefix of exactly one page
    ("tiny_f32_b3", 150, (5, 60, 12), (4, 2, 1, 3)),  # two pages and 22 tokens, changing block sizes
    ("small_f32", 300, (37, 100), None),
    ("small_bf16", 130, (37, 100), None),
    ("small_bf16", 1000, (3, 400), (16, 8)),
    ("small_bf16_llama", 200, (64, 5, 130, 33), None),
    ("tiny_f32_b3", 1100, (5, 60, 12), (4, 2, 1, 3)),  # 17 shared pages: the rounds attend to them once
    ("small_bf16_long8k", 1100, (3, 40), None),
])
def test_prefill_shared_and_rounds(name, prefix_len, lens, schedule):
    w = configs.get(name)
    w = w.with_(batch=len(lens), prompt_lens=tuple(prefix_len + n for n in lens))
    bf16 = w.dtype == "bf16"
    tol = 5e-2 if bf16 else 1e-3
    m = om.Model(w)
    prefix, own = _prompts(w, prefix_len, lens, 31)
    states = [spec.prefill(m, np.concatenate([prefix, p])) for p in own]
    rounds = 4
    sess = _session(w, keep_logits=True, max_seq_len=max(w.prompt_lens) + (rounds + 2) * w.block_size + 8)
    try:
        first = sess.prefill_shared(prefix, own)
        plog = sess.logits("prefill")
        alive = [True] * len(states)
        for s, st in enumerate(states):
            assert np.abs(plog[s] - st.first_logits).max() <= tol
            if int(first[s]) != st.anchor:
                assert bf16 and spec.top2_margin(st.first_logits[None])[0] < tol
                alive[s] = False
            for l in range(w.draft_layers):
                assert _rel(sess.cache("draft", "k", s, l), st.dcache.k[l]) < (2e-2 if bf16 else 1e-5)
                assert _rel(sess.cache("draft", "v", s, l), st.dcache.v[l]) < (2e-2 if bf16 else 1e-5)
        compared = 0
        for r in range(rounds):
            B = schedule[r % len(schedule)] if schedule else w.block_size
            mr = spec.at_block_size(m, B) if schedule else m
            if schedule:
                sess.set_block_size(B)
            sess.draft_block()
            dlog = sess.logits("draft") if B > 1 else None
            props = []
            for s, st in enumerate(states):
                if not alive[s]:
                    props.append(np.zeros(B - 1, np.int64))
                    continue
                d, odl = spec.draft(mr, st)
                if B > 1:
                    assert np.abs(dlog[s] - odl).max() <= tol, f"round {r} sequence {s}"
                props.append(np.asarray(d))
            prop = np.stack(props).astype(np.int32) if B > 1 else np.zeros((len(states), 1), np.int32)
            acc, bonus = sess.verify(prop)
            vlog = sess.logits("verify")
            for s, st in enumerate(states):
                if not alive[s]:
                    continue
                rd = spec.verify(mr, st, prop[s][:B - 1].astype(np.int64), keep_logits=True)
                assert np.abs(vlog[s] - rd.verify_logits).max() <= tol, f"round {r} sequence {s}"
                if (int(acc[s]), int(bonus[s])) != (rd.accepted, rd.bonus):
                    assert bf16 and spec.top2_margin(rd.verify_logits).min() < tol
                    alive[s] = False
                    continue
                assert int(sess.lengths()[s]) == st.committed
                compared += 1
        assert compared >= 2
    finally:
        sess.close()


@pytest.mark.parametrize("prefix_len", [900, 2200])  # rounds sequence by sequence; rounds on the shared keys
def test_prefill_shared_runs_in_several_chunks(prefix_len):
    """A prefix longer than one prefill chunk and more suffix rows than one (a sequence split over two), against a
    plain prefill of the whole prompts by the same library; then graph replays equal eager rounds bit for bit."""
    w = configs.get("small_bf16")
    lens = (700, 3, 900, 1200, 64)
    w = w.with_(batch=len(lens), prompt_lens=tuple(prefix_len + n for n in lens), target_layers=2, ctx_layer_ids=(0, 1), draft_layers=1)
    prefix, own = _prompts(w, prefix_len, lens, 5)
    out = {}
    for mode in ("plain", "shared", "eager"):
        sess = _session(w, keep_logits=True, max_seq_len=max(w.prompt_lens) + 200, graphs=mode != "eager")
        try:
            if mode == "plain":
                sess.prefill([np.concatenate([prefix, p]) for p in own])
            else:
                sess.prefill_shared(prefix, own)
            pl = sess.logits("prefill")
            v = []
            for r in range(4):
                sess.draft_block()
                prop = synth.uniform_ints(r, 0x7A, len(lens) * (w.block_size - 1), w.vocab).reshape(len(lens), -1).astype(np.int32)
                sess.verify(prop)
                v.append(sess.logits("verify"))
            out[mode] = (pl, v)
        finally:
            sess.close()
    # bf16 storage on both sides, sums in another order: the parity tests' bound, each side's
    assert np.abs(out["plain"][0] - out["shared"][0]).max() <= 2 * 5e-2
    assert np.abs(out["plain"][1][0] - out["shared"][1][0]).max() <= 2 * 5e-2
    np.testing.assert_array_equal(out["shared"][0], out["eager"][0])
    for a, b in zip(out["shared"][1], out["eager"][1]):
        np.testing.assert_array_equal(a, b)


def test_prefill_shared_pages_are_shared_and_errors():
    from block_diffusion_speculative_ctx_gb300 import DFLASH_E_CAPACITY, DFLASH_E_INVAL, DFlashError
    w = configs.get("tiny_f32_b3")
    prefix, own = _prompts(w, 640, (10, 20, 30), 3)
    w = w.with_(prompt_lens=tuple(640 + len(p) for p in own))
    # ten shared pages and one own page each: 13 pages hold what 33 would without sharing
    sess = _session(w, max_seq_len=760, kv_pool_tokens=13 * 64)
    try:
        with pytest.raises(DFlashError) as e:
            sess.prefill([np.concatenate([prefix, p]) for p in own])
        assert e.value.status == DFLASH_E_CAPACITY
        first = sess.prefill_shared(prefix, own)
        sess.verify(sess.draft_block())
        with pytest.raises(DFlashError) as e:
            sess.prefill_shared(prefix, [np.concatenate([p, prefix[:100]]) for p in own])
        assert e.value.status == DFLASH_E_CAPACITY
        bad = prefix.copy()
        bad[3] = w.vocab
        with pytest.raises(DFlashError) as e:
            sess.prefill_shared(bad, own)
        assert e.value.status == DFLASH_E_INVAL
        with pytest.raises(DFlashError):
            sess.prefill_shared(prefix, [own[0], own[1][:0], own[2]])
        # a prefix below one page is a plain prefill; an empty one too; and the session is reusable
        np.testing.assert_array_equal(sess.prefill_shared(prefix[:20], own), sess.prefill([np.concatenate([prefix[:20], p]) for p in own]))
        np.testing.assert_array_equal(sess.prefill_shared(prefix[:0], own), sess.prefill(own))
        np.testing.assert_array_equal(sess.prefill_shared(prefix, own), first)
    finally:
        sess.close()


# ---------------------------------------------------------------------------------------------- logit rules
RULES = dict(repetition=[1.3, 1.0, 2.0], presence=[0.5, 0.0, -0.25], frequency=[0.2, 0.4, 0.0],
             bias=[{5: 3.0, 900: -1e9, 7: 2.5}, {}, {11: 4.0}])


def _ruled(lg, history, prompt_len, s):
    bias = RULES["bias"][s]
    ids, vals = np.array([list(bias.keys()) or [-1]]), np.array([list(bias.values()) or [0.0]])
    f = lambda k: np.float32([RULES[k][s]])  # noqa: E731
    return serving.process_logits(lg[None], 1, history=np.array([history]), hist_lens=[len(history)], prompt_lens=[prompt_len],
                                  repetition=f("repetition"), presence=f("presence"), frequency=f("frequency"),
                                  bias_ids=ids, bias_values=vals.astype(np.float32))[0]


def _ruled_stream(m, prompt, n, s, mask=None):
    """Token by token under the rules: (tokens, their top-two margins)."""
    st = spec.prefill(m, prompt)
    cache = st.tcache.copy()
    hist, out, margins = [int(t) for t in prompt], [], []
    lg = st.first_logits
    while len(out) < n:
        z = _ruled(lg, hist, len(prompt), s)
        if mask is not None:
            z = np.where(mask(len(out)), z, -np.inf)
        t = int(np.argmax(z))
        margins.append(float(np.diff(np.sort(z[np.isfinite(z)])[-2:])[0]))
        out.append(t)
        hist.append(t)
        lg = m.target_forward([t], cache)[0][0]
    return np.array(out), np.array(margins)


def _same_stream(got, stream, n):
    """Equal up to the first difference, which may only be at a near-tie (both sides' logits agree to 1e-3, so the
    top two of the oracle lie within 2e-3); returns how many tokens were compared."""
    toks, margins = stream
    for i in range(n):
        if got[i] != toks[i]:
            assert margins[i] < 2e-3, (i, got[i], toks[i], margins[i])
            return i
    return n


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("planted", [False, True])
def test_ruled_rounds_emit_the_token_by_token_stream(shared, planted):
    """fp32: the speculative stream under penalties and biases equals decoding token by token under them, with the
    drafter's own proposals and with planted ones (accepted drafts, which later rows must count)."""
    w = configs.get("tiny_f32_b3")
    m = om.Model(w)
    prefix, own = _prompts(w, 70, (20, 7, 19), 9)
    prompts = [np.concatenate([prefix, p]) for p in own]
    n = 26
    streams = [_ruled_stream(m, p, n + w.block_size, s) for s, p in enumerate(prompts)]
    assert any(len(set(streams[s][0].tolist())) < n for s in range(3))   # tokens do repeat
    w = w.with_(prompt_lens=tuple(len(p) for p in prompts))
    sess = _session(w, max_seq_len=max(w.prompt_lens) + n + 4 * w.block_size)
    try:
        sess.set_logit_rules(**RULES)
        first = sess.prefill_shared(prefix, own) if shared else sess.prefill(prompts)
        got = [[int(first[s])] for s in range(3)]
        rounds = 0
        while min(len(g) for g in got) < n:
            drafts = sess.draft_block()
            if planted:   # true tokens, then a wrong one, 0..B-1 of them right
                for s in range(3):
                    right = (rounds + s) % w.block_size
                    nxt = streams[s][0][len(got[s]):len(got[s]) + w.block_size - 1]
                    drafts[s] = (streams[s][0][0] + 1) % w.vocab
                    drafts[s][:min(right, len(nxt))] = nxt[:right]
            acc, bonus = sess.verify(drafts)
            for s in range(3):
                got[s] += [int(t) for t in drafts[s][:acc[s]]] + [int(bonus[s])]
            rounds += 1
        assert sum(_same_stream(got[s], streams[s], n) for s in range(3)) >= 2 * n
        if planted:
            assert rounds < n - 1   # drafts were accepted
        # off again: the plain greedy stream
        sess.set_logit_rules()
        first = sess.prefill(prompts)
        for s in range(3):
            assert int(first[s]) == spec.prefill(m, prompts[s]).anchor
    finally:
        sess.close()


def test_ruled_sampled_round_at_top_1_is_the_greedy_one():
    """top-k 1 keeps one token of each ruled law: the sampled round emits the ruled greedy stream."""
    w = configs.get("tiny_f32_b3")
    m = om.Model(w)
    prompts = synth.prompts(w)
    n = 14
    streams = [_ruled_stream(m, p, n + w.block_size, s) for s, p in enumerate(prompts)]
    sess = _session(w, max_seq_len=max(w.prompt_lens) + n + 4 * w.block_size)
    rng = np.random.default_rng(0)
    try:
        sess.set_logit_rules(**RULES)
        sess.set_sampling_filter(top_k=1)
        first = sess.prefill(prompts)
        got = [[int(first[s])] for s in range(3)]
        while min(len(g) for g in got) < n:
            d = sess.draft_block_sampled(1.3, rng.random((3, w.block_size - 1)).astype(np.float32))
            acc, emit = sess.verify_sampled(1.3, d, rng.random((3, w.block_size)).astype(np.float32))
            for s in range(3):
                got[s] += [int(t) for t in d[s][:acc[s]]] + [int(emit[s])]
        assert sum(_same_stream(got[s], streams[s], n) for s in range(3)) >= 2 * n
    finally:
        sess.close()


def _pack(allowed):
    V = allowed.shape[-1]
    pad = np.zeros((allowed.shape[0], (V + 31) // 32 * 32), np.uint64)
    pad[:, :V] = allowed
    return (pad.reshape(allowed.shape[0], -1, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)


@pytest.mark.parametrize("device", [False, True])
def test_masked_rounds_emit_the_masked_stream(device):
    """A grammar by position: token k of a sequence must be k modulo 3.  With masks (one per state) on the first
    tokens and on every verify, the emitted stream is the masked token-by-token one."""
    import torch
    w = configs.get("tiny_f32_b3")
    m = om.Model(w)
    prompts = synth.prompts(w)
    V, n, B = w.vocab, 12, w.block_size
    states = np.stack([np.arange(V) % 3 == k for k in range(3)])
    saved = {k: RULES[k] for k in RULES}
    streams = [_ruled_stream(m, p, n + B, s, mask=lambda k: states[k % 3]) for s, p in enumerate(prompts)]
    assert RULES == saved
    masks = _pack(states)
    if device:
        masks = torch.from_numpy(masks.view(np.int32)).cuda()
    put = lambda i: torch.as_tensor(np.asarray(i), dtype=torch.int32).cuda() if device else np.asarray(i, np.int32)  # noqa: E731
    sess = _session(w, max_seq_len=max(w.prompt_lens) + 6 * n + 4 * B)
    try:
        sess.set_logit_rules(**RULES)
        sess.set_token_masks(masks, put([0, 0, 0]))
        first = sess.prefill(prompts)
        got = [[int(first[s])] for s in range(3)]
        while min(len(g) for g in got) < n:
            drafts = sess.draft_block()
            for s in range(3):
                nxt = streams[s][0][len(got[s]):len(got[s]) + B - 1]
                drafts[s][:len(nxt)] = nxt
                drafts[s][s:] = 0   # some right, the rest wrong or right by chance
            sess.set_token_masks(masks, put([[(len(got[s]) + j) % 3 for j in range(B)] for s in range(3)]).reshape(-1))
            acc, bonus = sess.verify(drafts)
            for s in range(3):
                got[s] += [int(t) for t in drafts[s][:acc[s]]] + [int(bonus[s])]
        assert sum(_same_stream(got[s], streams[s], n) for s in range(3)) >= 2 * n
    finally:
        sess.close()


def test_masks_that_leave_nothing_and_bad_masks():
    from block_diffusion_speculative_ctx_gb300 import DFLASH_E_DEVICE_CHECK, DFLASH_E_INVAL, DFlashError
    w = configs.get("tiny_f32_b3")
    prompts = synth.prompts(w)
    words = (w.vocab + 31) // 32
    none, some = np.zeros((1, words), np.uint32), np.full((1, words), 3, np.uint32)
    B = w.block_size
    sess = _session(w)
    try:
        sess.set_token_masks(none, [-1, 0, -1])
        with pytest.raises(DFlashError) as e:
            sess.prefill(prompts)
        assert e.value.status == DFLASH_E_DEVICE_CHECK and "without a token" in str(e.value)
        sess.set_token_masks(some, [0, 0])
        with pytest.raises(DFlashError) as e:   # set for two rows, the prefill has three
            sess.prefill(prompts)
        assert e.value.status == DFLASH_E_INVAL
        sess.set_token_masks()
        plain = sess.prefill(prompts)
        for bad in ((none, [0] * 3), (none, [1] * (3 * B)), (np.zeros((1 + 3 * B, words), np.uint32), [0] * (3 * B))):
            d = sess.draft_block() if sess.lengths()[0] == len(prompts[0]) and bad[1] == [0] * 3 else d
            with pytest.raises(DFlashError) as e:
                sess.set_token_masks(*bad)
            assert e.value.status == DFLASH_E_INVAL
        sess.set_token_masks(none, [-1] * (3 * B - 1) + [0])
        with pytest.raises(DFlashError) as e:
            sess.verify(d)
        assert e.value.status == DFLASH_E_DEVICE_CHECK
        np.testing.assert_array_equal(sess.prefill(prompts), plain)   # masks are for one pass; the session goes on
        for kw in (dict(repetition=0.0), dict(repetition=float("nan")), dict(presence=float("inf")), dict(bias={w.vocab: 1.0}),
                   dict(bias={1: float("nan")})):
            with pytest.raises(DFlashError) as e:
                sess.set_logit_rules(**kw)
            assert e.value.status == DFLASH_E_INVAL
    finally:
        sess.close()


def test_a_device_mask_index_behind_the_masks_means_no_mask():
    """Masks of an earlier call still lie in the session's buffer behind a later, shorter list: a device index that
    points there leaves the row as it is, as does one far outside."""
    import torch
    w = configs.get("tiny_f32_b3")
    prompts = synth.prompts(w)
    words, B = (w.vocab + 31) // 32, w.block_size
    only = np.zeros((3, words), np.uint32)   # mask k allows token k alone
    only[:, 0] = [1, 2, 4]
    dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    sess = _session(w, max_seq_len=max(w.prompt_lens) + 8 * B)
    try:
        plain = sess.prefill(prompts)
        sess.set_token_masks(dev(only.view(np.int32)), dev([0, 1, 2]))
        np.testing.assert_array_equal(sess.prefill(prompts), [0, 1, 2])
        sess.set_token_masks(dev(only[2:].view(np.int32)), dev([0, 1, 2]))   # one mask: 1 and 2 lie behind it
        np.testing.assert_array_equal(sess.prefill(prompts), [2, plain[1], plain[2]])
        sess.set_token_masks(dev(only[2:].view(np.int32)), dev([1 << 30, -(1 << 31), 0]))
        np.testing.assert_array_equal(sess.prefill(prompts), [plain[0], plain[1], 2])
        # the same in verified rows
        d = sess.draft_block()
        sess.set_token_masks(dev(only[:1].view(np.int32)), dev([0] + [1] * (3 * B - 1)))
        acc, bonus = sess.verify(d)
        assert d[0][0] != 0 and (int(acc[0]), int(bonus[0])) == (0, 0)
        sess.set_token_masks(dev(only[2:].view(np.int32)), dev([1, 1, 0]))
        sess.prefill(prompts)
        np.testing.assert_array_equal(sess.draft_block(), d)
        a2, b2 = sess.verify(d)   # without masks: the rows above that were not masked
        np.testing.assert_array_equal(a2[1:], acc[1:])
        np.testing.assert_array_equal(b2[1:], bonus[1:])
    finally:
        sess.close()


@pytest.mark.parametrize("filtered", [False, True])
def test_masked_sampled_rounds_emit_open_tokens_alone(filtered):
    """Masks and -inf biases in sampled rounds, with proposals from any law: no closed token is accepted or emitted,
    filtered or not."""
    w = configs.get("tiny_f32_b3")
    prompts = synth.prompts(w)
    V, B, n = w.vocab, w.block_size, 10
    states = np.stack([np.arange(V) % 3 == k for k in range(3)])
    masks = _pack(states)
    banned = 9
    rng = np.random.default_rng(4)
    sess = _session(w, keep_logits=True, max_seq_len=max(w.prompt_lens) + (n + 2) * B)
    tested = 0
    try:
        sess.set_logit_rules(bias={banned: -np.inf})
        if filtered:
            sess.set_sampling_filter(top_k=5)
        sess.set_token_masks(masks, [0, 1, 2])
        anchor = sess.prefill(prompts)
        assert [int(t) % 3 for t in anchor] == [0, 1, 2] and banned not in anchor
        for r in range(n):
            u = rng.random((3, B - 1)).astype(np.float32)
            d = sess.draft_block_sampled(1.0, u)
            dlog = sess.logits("draft")
            state = rng.integers(0, 3, (3, B))
            for s in range(3):
                # proposals that the drafter's own filtered law does not have (its least likely tokens), open ones and
                # closed ones in turn
                for j in range(B - 1):
                    want = states[state[s, j]] if (r + s + j) % 2 else ~states[state[s, j]]
                    d[s, j] = np.flatnonzero(want)[np.argmin(dlog[s, j + 1][want])]
            if r % 3 == 2:
                d[:, 0], state[:, 0] = banned, 0
            sess.set_token_masks(masks, state.reshape(-1))
            acc, emit = sess.verify_sampled(1.0, d, (0.999 * rng.random((3, B))).astype(np.float32))
            for s in range(3):
                row = np.arange(int(acc[s]) + 1)
                out = np.append(d[s][:acc[s]], emit[s])
                assert (out % 3 == state[s, row]).all() and banned not in out, (r, s, out, state[s])
                tested += len(out)
    finally:
        sess.close()
    assert tested >= 3 * n


def test_a_proposal_outside_the_drafters_law_is_accepted_where_the_target_has_it():
    """A mask that leaves one token: p is 1 there.  Proposed although the drafter's top-1 law lacks it, it is accepted
    (and every closed one refused)."""
    w = configs.get("tiny_f32_b3")
    V, B = w.vocab, w.block_size
    sess = _session(w, keep_logits=True, max_seq_len=max(w.prompt_lens) + 4 * B)
    try:
        sess.set_sampling_filter(top_k=1)
        sess.prefill(synth.prompts(w))
        d = sess.draft_block_sampled(1.0, np.full((3, B - 1), 0.5, np.float32))
        only = np.zeros((3 * B, V), bool)
        tok = np.zeros((3, B), np.int64)
        for s in range(3):
            for j in range(B):
                tok[s, j] = (int(d[s, min(j, B - 2)]) + 1 + j) % V   # not the drafter's
                only[s * B + j, tok[s, j]] = True
        sess.set_token_masks(_pack(only), np.arange(3 * B))
        prop = tok[:, :B - 1].astype(np.int32)
        prop[1, 1] = (prop[1, 1] + 1) % V                            # closed
        prop[2, 0] = d[2, 0]                                         # the drafter's own, closed
        acc, emit = sess.verify_sampled(1.0, prop, np.full((3, B), 0.5, np.float32))
        assert acc.tolist() == [B - 1, 1, 0]
        assert emit.tolist() == [tok[0, B - 1], tok[1, 1], tok[2, 0]]
    finally:
        sess.close()


def test_refused_masks_leave_those_set_before():
    """Masks set for a verify or a prefill, then refused ones: the pass runs under the first."""
    from block_diffusion_speculative_ctx_gb300 import DFLASH_E_INVAL, DFlashError
    w = configs.get("tiny_f32_b3")
    prompts = synth.prompts(w)
    words, B = (w.vocab + 31) // 32, w.block_size
    only = np.zeros((2, words), np.uint32)
    only[:, 0] = [1 << 5, 1 << 6]

    def refused(sess, rows):
        for bad in ((only, [2] + [0] * (rows - 1)), (only, [0] * (rows + 1) if rows != 3 else []),
                    (np.zeros((3 * B + 1, words), np.uint32), [0] * rows)):
            with pytest.raises(DFlashError) as e:
                sess.set_token_masks(*bad)
            assert e.value.status == DFLASH_E_INVAL

    sess = _session(w, max_seq_len=max(w.prompt_lens) + 8 * B)
    try:
        sess.set_token_masks(only, [0, 1, 0])
        refused(sess, 3)
        assert sess.prefill(prompts).tolist() == [5, 6, 5]
        d = np.full_like(sess.draft_block(), 7)
        sess.set_token_masks(only, [0, 1, 1] * B)
        refused(sess, 3 * B)
        with pytest.raises(DFlashError):   # a refused verify keeps them too
            sess.verify(np.full_like(d, w.vocab))
        acc, bonus = sess.verify(d)
        assert acc.tolist() == [0, 0, 0] and bonus.tolist() == [[5, 6, 6][(s * B) % 3] for s in range(3)]
    finally:
        sess.close()


def test_a_prefill_drops_the_masks_of_the_verify_it_takes_the_place_of():
    """Masks set after a draft belong to its verify: a prefill instead runs without them, whether or not their number
    of rows is its batch, and a refused prefill leaves them."""
    from block_diffusion_speculative_ctx_gb300 import DFlashError
    w = configs.get("tiny_f32_b3")
    prompts = synth.prompts(w)
    words, B = (w.vocab + 31) // 32, w.block_size
    only = np.zeros((1, words), np.uint32)
    only[0, 0] = 1 << 5
    sess = _session(w, max_seq_len=max(w.prompt_lens) + 8 * B)
    try:
        plain = sess.prefill(prompts)
        assert 5 not in plain
        for block in (B, 1):   # 3 B rows, then 3: as many as the prefill has
            sess.set_block_size(block)
            sess.draft_block()
            sess.set_token_masks(only, [0] * (3 * block))
            np.testing.assert_array_equal(sess.prefill(prompts), plain)
            d = sess.draft_block()
            sess.set_token_masks(only, [0] * (3 * block))
            with pytest.raises(DFlashError):
                sess.prefill([prompts[0][:0], prompts[1], prompts[2]])
            acc, bonus = sess.verify(d)
            assert acc.tolist() == [0, 0, 0] and bonus.tolist() == [5, 5, 5]
            np.testing.assert_array_equal(sess.prefill(prompts), plain)
    finally:
        sess.close()


def test_host_masks_are_the_callers_again_after_the_call():
    """Page-locked masks and indices are overwritten as soon as the call returns, while the session's stream is still
    busy with what was queued before."""
    import torch
    w = configs.get("tiny_f32_b3")
    prompts = synth.prompts(w)
    words = (w.vocab + 31) // 32
    sess = _session(w)
    try:
        sess.prefill(prompts)
        masks = torch.zeros((3, words), dtype=torch.int32).pin_memory()
        masks[:, 0] = torch.tensor([1 << 5, 1 << 6, 1 << 7])
        index = torch.tensor([2, 0, 1], dtype=torch.int32).pin_memory()
        torch.cuda._sleep(50_000_000)
        sess.set_token_masks(masks, index)
        masks.fill_(1 << 9)
        index.fill_(-1)
        assert sess.prefill(prompts).tolist() == [7, 5, 6]
    finally:
        sess.close()


def test_repetition_penalties_without_a_normal_reciprocal_are_refused():
    from block_diffusion_speculative_ctx_gb300 import DFLASH_E_INVAL, DFlashError
    w = configs.get("tiny_f32")
    sess = _session(w)
    try:
        for r in (2.0 ** -127, 2.0 ** -149, 2.0 ** 127, float("inf"), 0.0, -1.0):
            with pytest.raises(DFlashError) as e:
                sess.set_logit_rules(repetition=r)
            assert e.value.status == DFLASH_E_INVAL
        for r in (2.0 ** -126, 2.0 ** 126):
            sess.set_logit_rules(repetition=r)
    finally:
        sess.close()


def test_growing_bias_lists_give_the_old_ones_back():
    """A bias map that grows token by token: the session holds one pair of lists, and tokens follow the new one (the kept
    logits are those before the rules)."""
    w = configs.get("tiny_f32_b3")
    prompts = synth.prompts(w)
    sess = _session(w, keep_logits=True, max_seq_len=max(w.prompt_lens) + 8 * w.block_size)
    bias = np.zeros(w.vocab, np.float32)
    try:
        held = []
        for n in range(1, 30):
            bias[19 + n] = 50.0 + 19 + n
            sess.set_logit_rules(bias={t: 50.0 + t for t in range(20, 20 + n)})
            first = sess.prefill(prompts)
            np.testing.assert_array_equal(first, (sess.logits("prefill") + bias).argmax(-1))
            acc, bonus = sess.verify(sess.draft_block())
            best = (sess.logits("verify") + bias).argmax(-1)
            assert bonus.tolist() == [best[s, acc[s]] for s in range(3)]
            assert all(20 <= t < 20 + n for t in (*first, *bonus))
            held.append(len(sess.alloc.live))
        assert len(set(held)) == 1, held
        sess.set_logit_rules(bias={30: 99.0})   # shorter again: the lists stay
        assert sess.prefill(prompts).tolist() == [30] * 3 and len(sess.alloc.live) == held[0]
    finally:
        sess.close()
        assert not sess.alloc.live


def test_a_failed_allocation_leaves_nothing_behind():
    """The allocator refuses each of the shared prefix's, the rules' and the masks' buffers in turn: E_NOMEM, nothing more
    held than before, and the call succeeds once it can."""
    from block_diffusion_speculative_ctx_gb300 import DFLASH_E_NOMEM, DFlashError
    from block_diffusion_speculative_ctx_gb300 import session as sm
    left = [1 << 30]
    real = sm._TorchAllocator

    class Allocator(real):
        def _alloc(self, nbytes, user):
            left[0] -= 1
            return None if left[0] < 0 else super()._alloc(nbytes, user)

    w = configs.get("tiny_f32_b3")
    prefix, own = _prompts(w, 70, (20, 7, 19), 9)
    w = w.with_(prompt_lens=tuple(70 + len(p) for p in own))
    sm._TorchAllocator = Allocator
    try:
        sess = _session(w, max_seq_len=max(w.prompt_lens) + 8 * w.block_size)
    finally:
        sm._TorchAllocator = real
    try:
        masks = np.full((1, (w.vocab + 31) // 32), 0xFFFFFFFF, np.uint32)
        steps = [lambda: sess.prefill_shared(prefix, own),
                 lambda: sess.set_logit_rules(repetition=1.1) or sess.prefill(own),
                 lambda: sess.set_token_masks(masks, [0, 0, 0])]
        for step, buffers in zip(steps, (5, 6, 2)):
            before = len(sess.alloc.live)
            for k in range(buffers):
                left[0] = k
                with pytest.raises(DFlashError) as e:
                    step()
                assert e.value.status == DFLASH_E_NOMEM and len(sess.alloc.live) == before, k
            left[0] = 1 << 30
            step()
            assert len(sess.alloc.live) == before + buffers
    finally:
        left[0] = 1 << 30
        sess.close()


@pytest.mark.parametrize("prefix_len", [960, 1024, 2048])   # rounds sequence by sequence; rounds on the shared keys
def test_bf16_rounds_behind_shared_keys_are_as_exact_as_others(prefix_len):
    """The rms error of a bf16 session's logits against 64 bits, behind a shared prefix and on the same prompts without
    sharing.  Both make the same kinds of roundings, in another order: over 2 x 16 rows of logits the two rms values agree to
    some percent (their spread is 1 / sqrt(2 n) of n independent errors).  A weight rounded to one bf16 would add a rounding of
    the size of the attention output's own, a fifth more in all; the bound lies half way."""
    w = configs.get("small_bf16")
    lens = (37, 100)
    w = w.with_(batch=2, prompt_lens=tuple(prefix_len + n for n in lens))
    m = om.Model(w)
    prefix, own = _prompts(w, prefix_len, lens, 31)
    prompts = [np.concatenate([prefix, p]) for p in own]
    states = [spec.prefill(m, p) for p in prompts]
    prop = synth.uniform_ints(3, 4, 2 * (w.block_size - 1), w.vocab).reshape(2, -1).astype(np.int32)
    want = [m.target_forward(np.concatenate([[st.anchor], p.astype(np.int64)]), st.tcache.copy())[0] for st, p in zip(states, prop)]
    rms = {}
    for shared in (False, True):
        sess = _session(w, keep_logits=True, max_seq_len=prefix_len + 300)
        try:
            first = sess.prefill_shared(prefix, own) if shared else sess.prefill(prompts)
            assert [int(t) for t in first] == [st.anchor for st in states]
            sess.draft_block()
            sess.verify(prop)
            err = sess.logits("verify") - np.stack(want)
            rms[shared] = float(np.sqrt((err ** 2).mean()))
        finally:
            sess.close()
    assert rms[True] <= 1.1 * rms[False], rms
