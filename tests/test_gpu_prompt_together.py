"""The prompt's calls together, as a program uses them: pages reserved, rotated keys placed, attention over the chunk,
log-probabilities of the tokens that follow and their gradient; captured and replayed, on another stream, through the C
marshalling and without it, and at offsets beyond 32 bits.

Where two ways to the same rows are compared in float32, each is within its bound of the exact result: scores and
weights are off by (d + 3 + 9 + n + 64) u relative to sums of magnitudes below 100 here, so 1e-4 covers the difference of two
(u = 2^-24, d = 64, n <= 400: 3e-5 each).
"""
import math

import pytest
import torch

import gated_delta_rule_75_amd as kda
from test_gpu_prefill import BF16, DEV, F32, attention64, bits, check, cu_of, queries
from test_gpu_prompt import turn64
from test_gpu_serving import Cache, counts, gen, i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


class Layer:
    """One attention layer with its projections, and the logits behind it."""

    def __init__(self, hq=8, hkv=2, d=64, width=48, vocab=997, page=16, dtype=F32, seed=3):
        g = gen(seed)
        self.hq, self.hkv, self.d, self.page, self.dtype = hq, hkv, d, page, dtype
        self.wq, self.wk, self.wv = (torch.randn(width, h * d, generator=g) / width ** 0.5 for h in (hq, hkv, hkv))
        self.wo = torch.randn(hq * d, vocab, generator=g) / (hq * d) ** 0.5 * 4
        self.embed = torch.randn(vocab, width, generator=g)
        self.freqs = kda.rotary_frequencies(d, scaling="smooth", factor=4.0, original_length=256)
        for name in ("wq", "wk", "wv", "wo", "embed"):
            setattr(self, name, getattr(self, name).to(dtype).to(DEV))

    def rows(self, tokens):
        x = self.embed[tokens.long()]
        return [(x @ w).view(len(tokens), -1, self.d) for w in (self.wq, self.wk, self.wv)]


class Serving:
    """Sequences' pages of one layer."""

    def __init__(self, layer, n, n_pages, width):
        self.layer = layer
        self.table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
        self.lengths = torch.zeros(n, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        shape = (n_pages, layer.hkv, layer.page, layer.d)
        self.kp, self.vp = (torch.full(shape, float("nan"), dtype=layer.dtype, device=DEV) for _ in range(2))

    def run(self, tokens, new):
        """Attention outputs [T, Hq d] of the packed new tokens."""
        L = self.layer
        copies, granted = kda.cache_reserve(self.table, self.lengths, self.refs, i32(new), L.page)
        assert granted.tolist() == list(new)
        kda.pages_copy([self.kp, self.vp], copies)
        q, k, v = L.rows(tokens)
        cu = cu_of(new)
        q = kda.rotary_append(q, k, v, self.kp, self.vp, self.table, self.lengths - i32(new), L.freqs, cu_seqlens=cu,
                              q_out=q)
        return kda.paged_prefill(q, self.kp, self.vp, self.table, self.lengths, cu).flatten(1)


def exact(layer, tokens):
    """The layer's outputs for one sequence from its first token on, in fp64."""
    x = layer.embed.cpu().double()[tokens.long().cpu()]
    q, k, v = ((x @ w.cpu().double()).view(len(tokens), -1, layer.d) for w in (layer.wq, layer.wk, layer.wv))
    pos = torch.arange(len(tokens))
    q, k = (turn64(y, pos, layer.freqs, "half")[0] for y in (q, k))
    return attention64(k, v, q, 0, layer.d ** -0.5)[0].flatten(1)


def test_a_prompt_in_chunks_of_any_cut_and_one_token_at_a_time():
    L = Layer()
    tokens = torch.randint(0, 997, (130,), generator=gen(1), dtype=torch.int32).to(DEV)
    want = exact(L, tokens)
    for cut in ([130], [1, 60, 5, 64], [127, 1, 1, 1]):
        s, got, at = Serving(L, 1, 12, 9), [], 0
        for m in cut:
            got.append(s.run(tokens[at:at + m], [m]))
            at += m
        # (the projections are products of the library's in fp32 on values below 40)
        assert float((torch.cat(got).cpu().double() - want).abs().max()) <= 1e-3, cut
    # and the serving calls for one token: rotary, cache_append, paged_decode
    s = Serving(L, 1, 12, 9)
    s.run(tokens[:100], [100])
    for t in range(100, 130):
        kda.cache_reserve(s.table, s.lengths, s.refs, i32([1]), L.page)
        q, k, v = L.rows(tokens[t:t + 1])
        q, k = kda.rotary(q, k, i32([t]), L.freqs)
        kda.cache_append(k, v, s.kp, s.vp, s.table, s.lengths - 1)
        one = kda.paged_decode(q, s.kp, s.vp, s.table, s.lengths).flatten(1)
        assert float((one.cpu().double() - want[t]).abs().max()) <= 1e-3


def test_drafted_tokens_are_scored_behind_a_shared_prompt():
    """Two drafts after one prompt whose pages they share: each is scored as a sequence of its own would be, and the
    shared pages stay as they were."""
    L = Layer()
    prompt = torch.randint(0, 997, (77,), generator=gen(2), dtype=torch.int32).to(DEV)
    drafts = torch.randint(0, 997, (2, 6), generator=gen(3), dtype=torch.int32).to(DEV)
    s = Serving(L, 1, 30, 9)
    s.run(prompt, [77])
    held = s.kp[s.table[0, :4].long()].clone()
    s.table, s.lengths = kda.cache_fork(s.table, s.lengths, s.refs, i32([0, 0]))
    out = s.run(drafts.flatten(), [6, 6])
    assert torch.equal(bits(s.kp[s.table[0, :4].long()]), bits(held)) and torch.equal(s.table[0, :4], s.table[1, :4])
    logits = out @ L.wo
    nxt = torch.cat([drafts[:, 1:], i32([[-1], [5]])], 1).flatten()
    lp, lse, ent, best, which = kda.token_logprobs(logits, nxt, top=2, entropy=True)
    for n in range(2):
        x = exact(L, torch.cat([prompt, drafts[n]]))[77:] @ L.wo.cpu().double()
        p = torch.log_softmax(x, 1)
        mine = slice(6 * n, 6 * n + 6)
        t = nxt[mine].long().cpu()
        want = torch.where(t >= 0, p.gather(1, t.clamp(min=0)[:, None])[:, 0], torch.zeros(6).double())
        assert float((lp[mine].cpu().double() - want).abs().max()) <= 1e-2
        assert float((ent[mine].cpu().double() + (p.exp() * p).sum(1)).abs().max()) <= 1e-2
        assert float((best[mine].cpu().double() - torch.sort(p, 1, descending=True)[0][:, :2]).abs().max()) <= 1e-2
    # each draft's score as a sampler accepts it: within the row's best
    assert bool((lp <= best[:, 0] + 1e-5).logical_or(nxt < 0).all())


def test_the_loss_and_its_gradient_through_the_rotation():
    """Mean of -log p plus an entropy bonus of logits q . k' over rotated queries: the gradient of the queries through
    token_logprobs_grad and the inverse rotation against autograd in fp64."""
    R, H, d, V = 9, 2, 64, 501
    g = gen(5)
    q, w = torch.randn(R, H, d, generator=g).to(DEV), torch.randn(H * d, V, generator=g).to(DEV) / 4
    pos, tokens = i32(list(range(100, 100 + R))), torch.randint(0, V, (R,), generator=g, dtype=torch.int32).to(DEV)
    tokens[4] = -1
    f = kda.rotary_frequencies(48)
    turned, _ = kda.rotary(q, None, pos, f, layout="interleaved", amplitude=1.2)
    logits = turned.flatten(1) @ w
    lp, lse, h, _, _ = kda.token_logprobs(logits, tokens, entropy=True)
    d_lp = torch.full((R,), -1.0 / R, device=DEV)
    d_h = torch.full((R,), -0.1, device=DEV)
    d_logits = kda.token_logprobs_grad(logits, tokens, lse, d_lp, entropy=h, d_entropy=d_h)
    back, _ = kda.rotary((d_logits @ w.T).view(R, H, d), None, pos, f, layout="interleaved", amplitude=1.2, inverse=True)
    x = q.cpu().double().requires_grad_()
    a = pos.cpu().double()[:, None, None] * f.cpu()
    even, odd, rest = x[..., 0:48:2], x[..., 1:48:2], x[..., 48:]
    y = torch.stack([even * a.cos() - odd * a.sin(), even * a.sin() + odd * a.cos()], -1).flatten(2) * 1.2
    p = torch.log_softmax(torch.cat([y, rest], 2).flatten(1) @ w.cpu().double(), 1)
    t = tokens.long().cpu()
    loss = -(p.gather(1, t.clamp(min=0)[:, None])[:, 0] * (t >= 0)).sum() / R + 0.1 * (p.exp() * p).sum()
    loss.backward()
    mine = -lp.double().sum() / R - 0.1 * h.double().sum()
    assert abs(float(mine) - float(loss.detach())) <= 1e-4 * max(1.0, abs(float(loss.detach())))
    assert float((back.cpu().double() - x.grad).abs().max()) <= 1e-4 * max(1.0, float(x.grad.abs().max()))


def workload(dtype=BF16, seed=41):
    """Ragged sequences whose keys are split, and scores whose rows are."""
    new, past = [4, 2, 6, 1], [3500, 40, 900, 2100]
    cache = Cache([a + b for a, b in zip(new, past)], 2, 64, 32, dtype, seed=seed, extra_cols=6, spare=30)
    x = dict(table=cache.table.clone(), lengths=i32(past), refs=i32(counts(cache.table.tolist(), cache.kp.shape[0])),
             kp=cache.kp.clone(), vp=cache.vp.clone(), q=queries(13, 8, 64, dtype), k=queries(13, 2, 64, dtype, seed=2),
             v=queries(13, 2, 64, dtype, seed=3),
             logits=(torch.randn(13, 40000, generator=gen(7)) * 3).to(dtype).to(DEV),
             tokens=torch.randint(0, 40000, (13,), generator=gen(8), dtype=torch.int32).to(DEV),
             d=torch.randn(13, generator=gen(9)).to(DEV))
    return new, x


def steps(new, freqs, prefill_ws=None, score_ws=None):
    cu, fresh = cu_of(new), i32(new)

    def step(x):
        copies, granted = kda.cache_reserve(x["table"], x["lengths"], x["refs"], fresh, 32)
        kda.pages_copy([x["kp"], x["vp"]], copies)
        q = kda.rotary_append(x["q"], x["k"], x["v"], x["kp"], x["vp"], x["table"], x["lengths"] - fresh, freqs, cu_seqlens=cu)
        out, lse = kda.paged_prefill(q, x["kp"], x["vp"], x["table"], x["lengths"], cu, lse=True, workspace=prefill_ws)
        lp, row_lse, h, best, which = kda.token_logprobs(x["logits"], x["tokens"], top=3, entropy=True, workspace=score_ws)
        grad = kda.token_logprobs_grad(x["logits"], x["tokens"], row_lse, x["d"], entropy=h, d_entropy=x["d"])
        back, _ = kda.rotary(out, None, x["tokens"], freqs, inverse=True)
        return dict(granted=granted, q=q, out=out, lse=lse, lp=lp, row_lse=row_lse, h=h, best=best, which=which, grad=grad,
                    back=back)
    return step


def changed(x, replay):
    fresh = {a: b.clone() for a, b in x.items()}
    g = gen(100 + replay)
    for a in ("q", "k", "logits"):
        fresh[a] = (torch.randn(x[a].shape, generator=g) * 2).to(x[a].dtype).to(DEV)
    # other lengths give other parts
    fresh["lengths"] -= i32([37 * replay, 3 * replay, 700 * (replay % 2), 5])
    return fresh


def captured(step, held):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step({a: b.clone() for a, b in held.items()})
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held)
    return graph, got


def same(got, want, where):
    for a in want:
        assert torch.equal(bits(got[a]), bits(want[a])), (where, a)


def test_calls_are_captured_and_replayed():
    new, x = workload()
    step = steps(new, kda.rotary_frequencies(64))
    held = {a: b.clone() for a, b in x.items()}
    graph, got = captured(step, held)
    for replay in range(4):
        fresh = changed(x, replay)
        for a, b in fresh.items():
            held[a].copy_(b)
        graph.replay()
        want = step(fresh)  # eager work between the replays
        torch.cuda.synchronize()
        same(got, want, replay)
        same(held, fresh, replay)


def test_two_graphs_share_their_workspaces():
    """Graphs of different batches with the same scratch, replayed in turn."""
    ws = [torch.full((1 << 24,), 255, dtype=torch.uint8, device=DEV) for _ in range(2)]
    freqs = kda.rotary_frequencies(64)
    pairs = []
    for seed in (41, 43):
        new, x = workload(seed=seed, dtype=BF16 if seed == 41 else F32)
        step = steps(new, freqs, *ws)
        held = {a: b.clone() for a, b in x.items()}
        pairs.append((x, held, steps(new, freqs), *captured(step, held), step))  # (a graph's inputs live as long)
    for replay in range(3):
        wants = []
        for x, held, eager, graph, got, _ in pairs:
            fresh = changed(x, replay)
            wants.append(eager(fresh))
            for a, b in changed(x, replay).items():
                held[a].copy_(b)
        for x, held, eager, graph, got, _ in pairs:
            graph.replay()
        torch.cuda.synchronize()
        for want, (x, held, eager, graph, got, _) in zip(wants, pairs):
            same(got, want, replay)


def test_calls_run_on_the_current_stream():
    """On a side stream behind a long fill, the calls see what the stream wrote before them."""
    new, x = workload()
    step = steps(new, kda.rotary_frequencies(64))
    want = step({a: b.clone() for a, b in x.items()})
    late = {a: torch.zeros_like(b) for a, b in x.items()}
    big = torch.zeros(1 << 28, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(4):
            big.add_(1.0)
        for a in x:
            late[a].copy_(x[a])
        got = step(late)
    side.synchronize()
    same(got, want, "side")


def test_two_streams_at_once():
    """Two batches in flight on two streams, each with scratch of its own, do not disturb one another."""
    freqs = kda.rotary_frequencies(64)
    work = [workload(seed=s) for s in (41, 43)]
    fs = [steps(new, freqs) for new, _ in work]
    wants = [f({a: b.clone() for a, b in x.items()}) for f, (_, x) in zip(fs, work)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    copies = [[{a: b.clone() for a, b in x.items()} for _ in range(4)] for _, x in work]
    torch.cuda.synchronize()
    gots = [[], []]
    for i in range(4):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                gots[j].append(fs[j](copies[j][i]))
    torch.cuda.synchronize()
    for j in range(2):
        for got in gots[j]:
            same(got, wants[j], j)


def test_debug_check_of_tables_and_segments(monkeypatch):
    cache = Cache([40, 40], 1, 64, 16, BF16, seed=61)
    q, k = queries(5, 2, 64, BF16), queries(5, 1, 64, BF16)
    f = kda.rotary_frequencies(64)
    monkeypatch.setenv("KDA_DEBUG_CHECK", "1")
    kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, i32([0, 2, 5]))
    kda.rotary_append(q, k, k, cache.kp, cache.vp, cache.table, i32([3, 4]), f, cu_seqlens=i32([0, 2, 5]))
    with pytest.raises(kda.KdaError, match=r"lengths\[1\]"):
        kda.paged_prefill(q, cache.kp, cache.vp, cache.table, i32([40, 49]), i32([0, 2, 5]))
    for cu in ([0, 3, 2], [0, 6, 5], [1, 2, 5], [0, 2, 4]):
        with pytest.raises(kda.KdaError):
            kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, i32(cu))
        with pytest.raises(kda.KdaError):
            kda.rotary_append(q, k, k, cache.kp, cache.vp, cache.table, i32([3, 4]), f, cu_seqlens=i32(cu))
    cache.table[0, 1] = cache.kp.shape[0]
    with pytest.raises(kda.KdaError, match=r"page_table\[0, 1\]"):
        kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, i32([0, 2, 5]))


def test_the_marshalling_module_serves_the_usual_calls(monkeypatch):
    """The calls of a plain program go through the C marshalling; with it taken away the results are the same, and
    what it does not know goes the Python way and is refused there."""
    from gated_delta_rule_75_amd import prompt, serving

    new, x = workload()
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    freqs = kda.rotary_frequencies(64)
    cu, past = cu_of(new), x["lengths"] - 50

    def everything():
        kp, vp, q, k, logits = (x[a].clone() for a in ("kp", "vp", "q", "k", "logits"))
        lengths = past + i32(new)
        res = [*kda.rotary(q, k, x["tokens"], freqs), kda.rotary(q, None, x["tokens"], freqs)[0]]
        res += kda.rotary(q, k, x["tokens"], freqs[:20].contiguous(), layout="interleaved", amplitude=1.1, inverse=True,
                          q_out=torch.empty_like(q), k_out=torch.empty_like(k))
        res.append(kda.rotary_append(q, k, x["v"], kp, vp, x["table"], past, freqs, cu_seqlens=cu))
        res.append(kda.rotary_append(q[:4], k[:4], x["v"][:4], kp, vp, x["table"], past, freqs, layout="interleaved",
                                     amplitude=0.9, q_out=torch.empty_like(q[:4])))
        res.append(kda.paged_prefill(q, kp, vp, x["table"], lengths, cu))
        res += kda.paged_prefill(q, kp, vp, x["table"], lengths, cu, scale=0.2, window=900, sinks=2, max_length=5000,
                                 lse=True, workspace=ws, out=torch.empty_like(q))
        res += kda.paged_prefill(q, kp, vp, x["table"], lengths, cu, lse=torch.empty(13, 8, device=DEV))
        lp, lse, none, no_best, no_which = kda.token_logprobs(logits, x["tokens"])
        assert none is None and no_best is None and no_which is None
        res += [lp, lse, *kda.token_logprobs(logits, x["tokens"], top=4, entropy=True, workspace=ws)]
        lp, lse, h, _, _ = kda.token_logprobs(logits, None, entropy=True)
        assert lp is None
        res += [lse, h, kda.token_logprobs_grad(logits, x["tokens"], lse, x["d"]),
                kda.token_logprobs_grad(logits, None, lse, d_lse=x["d"], entropy=h, d_entropy=x["d"], out=logits)]
        return res + [kp, vp, logits]

    first = everything()
    assert serving._M is not None
    for name in ("rotary", "rotary_append", "paged_prefill", "token_logprobs", "token_logprobs_grad"):
        assert hasattr(serving._M, name)
    calls = []
    real = prompt._run
    monkeypatch.setattr(prompt, "_run", lambda *a: calls.append(a) or real(*a))
    scratch = prompt._run_scratch
    monkeypatch.setattr(prompt, "_run_scratch", lambda *a: calls.append(a) or scratch(*a))
    everything()
    assert not calls  # nothing went the Python way
    monkeypatch.setattr(serving, "_M", None)
    for a, b in zip(first, everything()):
        assert a.dtype == b.dtype and torch.equal(bits(a), bits(b))
    assert calls
    monkeypatch.undo()
    q, kp, vp, table = x["q"], x["kp"], x["vp"], x["table"]
    with pytest.raises(kda.KdaError, match="sinks"):
        kda.paged_prefill(q, kp, vp, table, past, cu, sinks=3)
    with pytest.raises(ValueError, match="window"):
        kda.paged_prefill(q, kp, vp, table, past, cu, window=2 ** 32)
    with pytest.raises(ValueError, match="lengths"):
        kda.paged_prefill(q, kp, vp, table, past[:1], cu)
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.paged_prefill(q, kp, vp, table, past, cu[:3])
    with pytest.raises(ValueError, match="torch.int32"):
        kda.rotary(q, None, x["tokens"].long(), freqs)
    with pytest.raises(ValueError, match="float64"):
        kda.rotary(q, None, x["tokens"], freqs.float())
    with pytest.raises(ValueError, match="freqs"):
        kda.rotary(q, None, x["tokens"], kda.rotary_frequencies(66))
    with pytest.raises(ValueError, match="layout"):
        kda.rotary(q, None, x["tokens"], freqs, layout="other")
    with pytest.raises(ValueError, match="top"):
        kda.token_logprobs(x["logits"], x["tokens"], top=-1)
    with pytest.raises(kda.KdaError, match="top"):
        kda.token_logprobs(x["logits"], x["tokens"], top=65)
    with pytest.raises(ValueError, match="tokens"):
        kda.token_logprobs_grad(x["logits"], None, x["d"], x["d"])


def test_timed_kernels_have_names():
    new, x = workload()
    with kda.kernel_timing() as t:
        steps(new, kda.rotary_frequencies(64))(x)
    names = [n for n, _ in t.records]
    for name in ("kda_rotary", "kda_paged_prefill", "kda_prefill_join", "kda_logprob_scan", "kda_logprob_join",
                 "kda_logprob_grad"):
        assert name in names, names


def test_offsets_beyond_32_bits():
    """Pages whose element offset passes 2^32, in a pool reserved but mostly untouched."""
    page, hkv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * hkv * d) + 700
    kp = torch.empty(n_pages, hkv, page, d, dtype=BF16, device=DEV)
    vp = torch.empty(n_pages, hkv, page, d, dtype=BF16, device=DEV)
    cache = Cache([180], hkv, d, page, BF16, seed=27, spare=0)
    far = [n_pages - 1, n_pages - 600, 5]
    for j, p in enumerate(far):
        old = int(cache.table_cpu[0, j])
        kp[p], vp[p] = cache.kp[old], cache.vp[old]
        cache.table[0, j] = p
    cache.kp, cache.vp = kp, vp
    for m in (3, 100):
        check(cache, queries(m, 16, d, BF16), [m])
    q, k, v = queries(1, 16, d, BF16), queries(1, hkv, d, BF16, seed=2), queries(1, hkv, d, BF16, seed=3)
    f = kda.rotary_frequencies(d)
    got = kda.rotary_append(q, k, v, kp, vp, cache.table, i32([100]), f)
    want_q, want_k = kda.rotary(q, k, i32([100]), f)
    assert torch.equal(got, want_q)
    assert torch.equal(kp[far[1], :, 36], want_k[0]) and torch.equal(vp[far[1], :, 36], v[0])


def test_rows_beyond_32_bits():
    """Tokens and logits whose element offset passes 2^32: the last ones are what they are alone."""
    T, H, d = 530000, 64, 128
    q = torch.empty(T, H, d, dtype=BF16, device=DEV)
    q[-3:] = queries(3, H, d, BF16)
    q[0] = queries(1, H, d, BF16, seed=2)[0]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    f = kda.rotary_frequencies(d)
    want, _ = kda.rotary(q[-3:].clone(), None, pos[-3:].clone(), f)
    first, _ = kda.rotary(q[:1].clone(), None, pos[:1].clone(), f)
    kda.rotary(q, None, pos, f, q_out=q)
    assert torch.equal(bits(q[-3:]), bits(want)) and torch.equal(bits(q[:1]), bits(first))
    x = q.view(-1)[:33000 * 131072].view(33000, 131072)
    x.zero_()
    x[-2:] = (torch.randn(2, 131072, generator=gen(5)) * 3).to(BF16).to(DEV)
    tokens = torch.arange(33000, dtype=torch.int32, device=DEV)
    got = kda.token_logprobs(x, tokens, top=2, entropy=True)
    alone = kda.token_logprobs(x[-2:].clone(), tokens[-2:].clone(), top=2, entropy=True)
    # (rows alone are split and joined: a few units in the last place)
    for a, b in zip(got, alone):
        assert float((a[-2:].double() - b.double()).abs().max()) <= 2e-5
    assert float((got[1][:-2] - math.log(131072)).abs().max()) <= 2e-5
    assert got[4][0].tolist() == [0, 1]
    d_lp = torch.ones(33000, device=DEV)
    want = kda.token_logprobs_grad(x[-2:].clone(), tokens[-2:].clone(), got[1][-2:].clone(), d_lp[-2:].clone())
    kda.token_logprobs_grad(x, tokens, got[1], d_lp, out=x)
    assert torch.equal(bits(x[-2:]), bits(want)) and float(x[5, 5]) == 1.0 and float(x[5, 6]) == -2.0 ** -17


def test_sizes_that_32_bits_do_not_hold_are_refused():
    """They would reach the library cut to their lower bits (2^32 + 5 logits as 5).  No tensor here has an element, so
    that none of these calls has anything to launch."""
    big = 2 ** 32

    def f(*shape, dtype=F32):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    def i(*shape):
        return f(*shape, dtype=torch.int32)

    freqs, none, pages = kda.rotary_frequencies(64), i(0), f(2, 1, 16, 64)
    cu = i32([0])
    calls = [
        ("V", lambda: kda.token_logprobs(f(0, big + 5), none, top=3)),
        ("V", lambda: kda.token_logprobs_grad(f(0, big + 5, dtype=BF16), none, f(0), f(0))),
        ("H_q", lambda: kda.rotary(f(0, big + 8, 64), None, none, freqs)),
        ("H_k", lambda: kda.rotary(f(0, 8, 64), f(0, big + 1, 64), none, freqs)),
        ("d", lambda: kda.rotary(f(0, 8, big + 64), None, none, freqs)),
        ("H_q", lambda: kda.rotary_append(f(0, big + 8, 64), f(0, 1, 64), f(0, 1, 64), pages, pages.clone(), i(0, 4), none, freqs)),
        ("P", lambda: kda.rotary_append(f(0, 8, 64), f(0, 1, 64), f(0, 1, 64), pages, pages.clone(), i(0, big + 4), none, freqs)),
        ("H_q", lambda: kda.paged_prefill(f(0, big + 8, 64), pages, pages, i(0, 4), none, cu)),
        ("P", lambda: kda.paged_prefill(f(0, 8, 64), pages, pages, i(0, big + 4), none, cu)),
        ("H_q", lambda: kda.paged_decode(f(0, big + 8, 64), pages, pages, i(0, 4), none)),
        ("P", lambda: kda.cache_append(f(0, 1, 64), f(0, 1, 64), pages, pages.clone(), i(0, big + 4), none)),
        ("P", lambda: kda.cache_fork(i(0, big + 4), none, i(3), none)),
        ("P", lambda: kda.cache_free(i(0, big + 4), none, i(3), none)),
        ("P", lambda: kda.cache_reserve(i(0, big + 4), none, i(3), none, 16)),
        ("P", lambda: kda.cache_compact(i(0, big + 4), i(3))),
        ("n_pages", lambda: kda.pages_copy(f(big + 2, 0), i(0, 2))),
        ("V", lambda: kda.beam_select(f(0, 2, big + 5), f(0, 2))),
        ("K", lambda: kda.beam_reorder(f(0, 4), i(0, big + 2))),
    ]
    for at, (name, call) in enumerate(calls):
        print(f"call {at}: {name}", flush=True)
        with pytest.raises(ValueError, match=f"{name} must be a 32-bit whole number"):
            call()


@pytest.mark.parametrize("marshalled", [True, False])
def test_tensors_that_calls_write_to_count_as_modified(monkeypatch, marshalled):
    """A value that autograd has saved and a call overwrites makes the backward fail instead of using what is there now;
    what the calls return requires no gradient; tensors of inference mode are written without a count."""
    from gated_delta_rule_75_amd import serving

    freqs = kda.rotary_frequencies(64)
    kda.rotary(queries(1, 1, 64, F32), None, i32([0]), freqs)
    if not marshalled:
        monkeypatch.setattr(serving, "_M", None)
    cache = Cache([40], 1, 64, 16, F32, seed=71)
    q, k = queries(3, 2, 64, F32), queries(3, 1, 64, F32)
    pos, cu, start = i32([5, 6, 7]), i32([0, 3]), i32([37])
    x, tokens = torch.randn(3, 90, generator=gen(1)).to(DEV), i32([1, 2, 3])
    lse, d = torch.logsumexp(x, 1), torch.ones(3, device=DEV)

    def writes(shape, call):
        leaf = torch.randn(shape, device=DEV, requires_grad=True)
        saved = leaf.exp()  # its backward needs its own result
        call(saved.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.sum().backward()

    writes(q.shape, lambda y: kda.rotary(q, k, pos, freqs, q_out=y))
    writes(k.shape, lambda y: kda.rotary(q, k, pos, freqs, k_out=y))
    writes(q.shape, lambda y: kda.rotary(y, None, pos, freqs, q_out=y))
    writes(q.shape, lambda y: kda.rotary_append(q, k, k, cache.kp, cache.vp, cache.table, start, freqs, cu_seqlens=cu,
                                                q_out=y))
    writes(cache.kp.shape, lambda y: kda.rotary_append(q, k, k, y, cache.vp, cache.table, start, freqs, cu_seqlens=cu))
    writes(cache.vp.shape, lambda y: kda.rotary_append(q, k, k, cache.kp, y, cache.table, start, freqs, cu_seqlens=cu))
    writes(q.shape, lambda y: kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu, out=y))
    writes((3, 2), lambda y: kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu, lse=y))
    writes(x.shape, lambda y: kda.token_logprobs_grad(x, tokens, lse, d, out=y))
    writes(x.shape, lambda y: kda.token_logprobs_grad(y, tokens, lse, d, out=y))
    z = q.clone().requires_grad_()
    for got in (*kda.rotary(z, k, pos, freqs), kda.paged_prefill(z, cache.kp, cache.vp, cache.table, cache.len, cu),
                kda.token_logprobs(x.clone().requires_grad_(), tokens)[0]):
        assert not got.requires_grad
    want = kda.rotary(q, None, pos, freqs)[0]
    with torch.inference_mode():
        y = q.clone()
        assert torch.equal(kda.rotary(y, None, pos, freqs, q_out=y)[0], want)
