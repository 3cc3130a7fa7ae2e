"""Attention of a chunk of new tokens over pages on the GPU against plain 64-bit code.

Tolerances (u = 2^-24; a rounding to bf16 is off by 2^-8 of the value at most): those of the one-token attention
(test_gpu_serving.py) with two more roundings for bf16.  A score is off by ds <= (d + 3) u scale sum|q k|, a weight by
the factor 1 +- (2 ds + w), w = 9 u; sums of n terms add (n + 64) u: |out - exact| <= vmax (4 ds + 2 w + 2 (n + 64) u).
With bf16 every weight enters the product rounded, which adds 2^-8 sum p |v|, and the output is rounded to bf16.
|lse - exact| <= 2 ds + w + (n + 64) u + 4 u |lse|.
"""
import math

import pytest
import torch

import gated_delta_rule_75_amd as kda
from test_gpu_serving import Cache, counts, gen, i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
STEP = {BF16: 2.0 ** -8, F32: U}
DEV = "cuda"


def bits(x):
    return x.contiguous().view(torch.uint8)


def queries(t, hq, d, dtype, seed=1, scale=2.0):
    return (torch.randn(t, hq, d, generator=gen(seed)) * scale).to(dtype).to(DEV)


def cu_of(new):
    return i32([sum(new[:i]) for i in range(len(new) + 1)])


def attention64(k, v, q, first, scale, window=0, sinks=0, absent=(), page=1, most=None):
    """Queries q [m,Hq,d] at positions first .. over k, v [t,Hkv,d], in fp64: out, lse, and their bounds without the
    output's rounding."""
    rounded = q.dtype == BF16
    m, hq, d = q.shape
    t, hkv = k.shape[:2]
    group = hq // hkv
    pos, at = torch.arange(t), first + torch.arange(m)
    seen = pos[None] <= at[:, None]
    if most is not None:
        seen &= pos[None] < most
    if window:
        seen &= (pos[None] > at[:, None] - window) | (pos[None] < sinks)
    for a in absent:
        seen &= (pos // page != a)[None]
    k, v, q = k.double(), v.double(), q.double()
    out, lse, tol, tol_lse = (torch.zeros(m, hq, *x).double() for x in ((d,), (), (d,), ()))
    for h in range(hkv):
        qs = q[:, h * group:(h + 1) * group].reshape(m * group, d)
        s = (qs @ k[:, h].T).view(m, group, t) * scale
        size = ((qs.abs() @ k[:, h].abs().T).view(m, group, t) * abs(scale))
        s = torch.where(seen[:, None], s, torch.full_like(s, -math.inf))
        size = torch.where(seen[:, None], size, torch.zeros_like(size)).amax(2) if t else torch.zeros(m, group).double()
        L = torch.logsumexp(s, 2) if t else torch.full((m, group), -math.inf).double()
        p = torch.exp(s - torch.where(L == -math.inf, torch.zeros_like(L), L)[..., None])
        n = seen.sum(1).double()[:, None]
        vv = torch.where(seen.any(0)[:, None], v[:, h], torch.zeros_like(v[:, h])) if t else v[:, h]
        mine = slice(h * group, (h + 1) * group)
        out[:, mine] = p @ vv
        lse[:, mine] = L
        ds, w, acc = (d + 3) * U * size, 9 * U, (n + 64) * U
        vmax = float(vv.abs().max()) if t else 0.0
        tol[:, mine] = (vmax * (4 * ds + 2 * w + 2 * acc))[..., None]
        if rounded:
            tol[:, mine] += p @ vv.abs() * 2.0 ** -8
        tol_lse[:, mine] = 2 * ds + w + acc + 4 * U * torch.where(L == -math.inf, torch.zeros_like(L), L).abs()
    return out, lse, tol, tol_lse


def check(cache, q, new, scale=None, window=0, sinks=0, absent=(), **kw):
    """The call for the last new[n] tokens of each sequence of the cache."""
    T, hq, d = q.shape
    dt = q.dtype
    out, lse = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu_of(new), scale=scale, window=window,
                                 sinks=sinks, lse=True, **kw)
    torch.cuda.synchronize()
    assert out.dtype == dt and out.shape == q.shape and lse.shape == (T, hq)
    at, worst = 0, 0.0
    for n, m in enumerate(new):
        if not m:
            continue
        qn = q[at:at + m].cpu()
        want, wlse, tol, tol_lse = attention64(cache.k[n], cache.v[n], qn, cache.lengths[n] - m,
                                               d ** -0.5 if scale is None else scale, window, sinks, absent, cache.page)
        tol = tol + STEP[dt] * (want.abs() + tol)
        got, got_lse = out[at:at + m].cpu().double(), lse[at:at + m].cpu().double()
        assert bool(got.isfinite().all()), n
        err = (got - want).abs()
        assert bool((err <= tol).all()), (n, m, cache.lengths[n], float((err / tol.clamp(min=1e-30)).max()))
        none = wlse == -math.inf
        assert torch.equal(got_lse == -math.inf, none) and not got[none].any()
        assert bool(((got_lse - wlse).abs()[~none] <= tol_lse[~none]).all()), n
        if (~none).any():
            worst = max(worst, float((err / tol)[~none].max()))
        at += m
    print(f"  worst error {worst:.3f} of the bound", flush=True)
    return out, lse


# dtype, hq, hkv, d, page, new tokens, earlier tokens
SHAPES = [
    (BF16, 8, 2, 128, 64, [5, 1, 16, 3], [100, 0, 63, 700]),          # few rows: keys split over waves
    (BF16, 4, 4, 64, 16, [1, 1, 1, 1, 1], [0, 15, 16, 300, 31]),      # one token, one head
    (BF16, 32, 1, 128, 16, [1, 2], [40, 200]),
    (BF16, 6, 2, 256, 48, [4, 9], [30, 500]),
    (BF16, 8, 2, 128, 64, [40, 100, 1, 129], [0, 7, 500, 64]),        # many rows: rows split over waves
    (BF16, 4, 4, 64, 32, [200, 33, 0, 64], [100, 0, 9, 1000]),
    (BF16, 14, 2, 64, 16, [65, 20], [3, 333]),                        # seven heads to one
    (BF16, 35, 5, 128, 256, [50], [77]),
    (BF16, 4, 2, 256, 16, [130, 17], [20, 450]),
    (BF16, 66, 2, 64, 64, [3, 70], [500, 0]),                         # 33 to one
    (BF16, 512, 1, 64, 64, [3, 1], [90, 31]),                         # more heads than a tile's rows
    (F32, 8, 2, 128, 64, [5, 1, 16, 3], [100, 0, 63, 700]),
    (F32, 4, 4, 64, 16, [1, 1, 1, 1, 1], [0, 15, 16, 300, 31]),
    (F32, 6, 2, 256, 48, [4, 9], [30, 500]),
    (F32, 8, 2, 128, 64, [40, 100, 1, 129], [0, 7, 500, 64]),
    (F32, 20, 4, 64, 32, [90, 33], [0, 900]),
    (F32, 4, 2, 256, 16, [130, 17], [20, 450]),
]


@pytest.mark.parametrize("dtype,hq,hkv,d,page,new,past", SHAPES)
def test_paged_prefill_matches_fp64(dtype, hq, hkv, d, page, new, past):
    print(f"prefill {dtype} hq={hq} hkv={hkv} d={d} page={page} new={new} past={past}", flush=True)
    cache = Cache([a + b for a, b in zip(new, past)], hkv, d, page, dtype, seed=hq + d)
    check(cache, queries(sum(new), hq, d, dtype), new)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,past", [([6], [9000]), ([3, 2], [200, 5000]), ([150], [4000])])
def test_paged_prefill_of_few_rows_is_split_and_joined(dtype, d, new, past):
    print(f"split {dtype} d={d} new={new} past={past}", flush=True)
    cache = Cache([a + b for a, b in zip(new, past)], 1, d, 64, dtype, seed=3)
    q = queries(sum(new), 4, d, dtype, scale=1.0)
    need = kda._lib.load().kda_paged_prefill_workspace(len(new), sum(new), 4, 1, d, int(dtype == BF16),
                                                       cache.table.shape[1] * 64, 0, 0)
    assert need > 0
    check(cache, q, new)
    check(cache, q, new, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [[1, 2, 3, 1, 5, 1], [60, 1, 100, 7, 90, 33]])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 1), (33, 4), (64, 64), (100, 17), (5000, 4), (700, 0),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)])
def test_paged_prefill_window_and_sinks(dtype, new, window, sinks):
    """Windows that begin inside a page, sinks that end inside one or reach into the window, windows longer than
    the sequence; every row has its own."""
    print(f"window {window} sinks {sinks} {dtype} new={new}", flush=True)
    cache = Cache([a + b for a, b in zip(new, [0, 62, 97, 700, 200, 1500])], 2, 64, 32, dtype, seed=window % 1000)
    check(cache, queries(sum(new), 8, 64, dtype), new, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [[2, 3, 2], [60, 100, 40]])
def test_paged_prefill_pages_given_back(dtype, new):
    """Entries without a page leave their tokens out, inside the sequence too; a sequence that has none left gives 0
    and -inf."""
    cache = Cache([300, 300, 40], 2, 128, 32, dtype, seed=5)
    cache.table[:, 1] = -1
    cache.table[:, 4] = cache.kp.shape[0]
    cache.table[:, 6] = -2147483648
    q = queries(sum(new), 4, 128, dtype)
    check(cache, q, new, absent=(1, 4, 6))
    cache.table[2] = -1
    out, lse = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu_of(new), lse=True)
    at = sum(new[:2])
    assert not out[at:].any() and bool(torch.isneginf(lse[at:]).all()) and bool(out[:at].any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [[3, 7], [70, 100]])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), -float("inf")])
def test_paged_prefill_never_uses_what_is_not_visible(dtype, d, new, garbage):
    """Keys and values behind a query (later tokens of its own chunk), before its window and behind the sequence hold
    NaN or infinities: each row is what it is without them."""
    cache = Cache([77 + new[0], 300 + new[1]], 2, d, 16, dtype, seed=9, garbage=garbage)
    q = queries(sum(new), 4, d, dtype)
    cu = cu_of(new)
    plain = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu, window=40, sinks=5, lse=True)
    first = [cache.lengths[n] - new[n] for n in range(2)]
    for n in range(2):  # before the first row's window, and the last tokens
        t = cache.lengths[n]
        for i in list(range(5, first[n] - 39)) + [t - 1, t - 2]:
            p = int(cache.table_cpu[n, i // 16])
            cache.kp[p, :, i % 16] = garbage
            cache.vp[p, :, i % 16] = garbage
    again = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu, window=40, sinks=5, lse=True)
    for a, b in zip(plain, again):
        at = 0
        for m in new:
            assert torch.equal(a[at:at + m - 2], b[at:at + m - 2])
            assert not bool(b[at + m - 1].isfinite().all())
            at += m


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [[4], [140]])
def test_paged_prefill_visible_values_that_are_not_finite(dtype, new):
    """They reach the rows that see them, in tiles with hidden keys and without, and no other row or channel."""
    cache = Cache([400], 1, 64, 16, dtype, seed=9)
    q = queries(sum(new), 2, 64, dtype, scale=0.3)
    for i in (3, 400 - new[0], 399):
        vp = cache.vp.clone()
        vp[int(cache.table_cpu[0, i // 16]), 0, i % 16, 17] = math.inf
        out = kda.paged_prefill(q, cache.kp, vp, cache.table, cache.len, cu_of(new))
        bad = ~out.isfinite()
        sees = torch.arange(400 - new[0], 400) >= i
        assert torch.equal(bad[..., 17].cpu(), sees[:, None].expand(-1, 2))
        bad[..., 17] = False
        assert not bad.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [[3, 3, 3], [90, 90, 90]])
def test_paged_prefill_extreme_scores(dtype, new):
    """One key far above the others early, late, and keys far below; every score of -inf."""
    cache = Cache([400, 400, 400], 1, 64, 16, dtype, seed=11)
    q = queries(sum(new), 4, 64, dtype)
    m = new[0]
    for n, (i, f) in enumerate([(5, 200.0), (310, 200.0), (3, -5000.0)]):
        cache.k[n][i] = (q[n * m, 0].cpu().float() * f).to(dtype)
        cache.kp[int(cache.table_cpu[n, i // 16]), :, i % 16] = cache.k[n][i].to(DEV)
    check(cache, q, new)
    kp = torch.full((2, 1, 16, 64), math.inf, dtype=dtype, device=DEV)
    out, lse = kda.paged_prefill(-torch.ones(m, 2, 64, dtype=dtype, device=DEV), kp, kp.clone().fill_(3.0), i32([[0, 1]]),
                                 i32([20]), i32([0, m]), lse=True)
    assert not out.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("new", [[7, 5, 3], [100, 20, 70]])
def test_paged_prefill_strided_queries_interleaved_pages_and_buffers(new):
    cache = Cache([70 + new[0], 3 + new[1], 129 + new[2]], 2, 128, 32, BF16, seed=21, interleaved=True)
    wide = queries(sum(new), 12, 128, BF16)
    table = torch.full((3, 40), -1, dtype=torch.int32, device=DEV)
    table[:, :cache.table.shape[1]] = cache.table
    cache.table = table[:, :cache.table.shape[1] + 3]
    out = torch.empty(sum(new), 8, 128, dtype=BF16, device=DEV)
    got, _ = check(cache, wide[:, 2:10], new, out=out)
    assert got.data_ptr() == out.data_ptr()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [[4, 9], [80, 120]])
def test_paged_prefill_scale(dtype, new):
    cache = Cache([200, 333], 2, 64, 16, dtype, seed=23)
    q = queries(sum(new), 4, 64, dtype)
    for scale in (-0.3, 0.0, 1e-30):
        check(cache, q, new, scale=scale)


@pytest.mark.parametrize("new", [[2, 5, 6, 1], [50, 70, 90, 40]])
def test_paged_prefill_lengths_that_cut(new):
    """max_length hides what lies behind it; new tokens before position 0 and sequences of no length see nothing; rows
    that belong to no sequence stay as they are."""
    cache = Cache([123, 300, 60, 60], 2, 64, 16, F32, seed=29)
    q = queries(sum(new) + 9, 4, 64, F32)
    cu = cu_of(new)
    out, lse = torch.full_like(q, 7.0), torch.full((q.shape[0], 4), 7.0, device=DEV)
    lengths = i32([123, 300, 4, -3])
    kda.paged_prefill(q, cache.kp, cache.vp, cache.table, lengths, cu, max_length=200, out=out, lse=lse)
    at = 0
    for n, m in enumerate(new):
        length = max(0, int(lengths[n]))
        want, wlse, tol, tol_lse = attention64(cache.k[n][:length], cache.v[n][:length], q[at:at + m].cpu(), length - m, 0.125,
                                               most=200)
        got, got_lse = out[at:at + m].cpu().double(), lse[at:at + m].cpu().double()
        assert bool(((got - want).abs() <= tol + 1e-30).all()), n
        none = wlse == -math.inf
        assert torch.equal(got_lse == -math.inf, none) and not got[none].any()
        assert bool(((got_lse - wlse).abs()[~none] <= tol_lse[~none]).all())
        at += m
    assert bool((out[at:] == 7).all()) and bool((lse[at:] == 7).all())
    none = kda.paged_prefill(q[:0], cache.kp, cache.vp, cache.table, lengths, i32([0, 0, 0, 0, 0]))
    assert none.shape == (0, 4, 64)
    out.fill_(7.0)
    kda.paged_prefill(q, cache.kp, cache.vp, cache.table, lengths, i32([0, 0, 0, 0, 0]), out=out)
    assert bool((out == 7).all())


def test_paged_prefill_many_sequences():
    """More sequences than a wave's lanes, empty ones among them, decode steps and prompts in one batch."""
    new = [(7 * i) % 3 if i % 50 else 40 for i in range(700)]
    past = [(13 * i) % 90 for i in range(700)]
    cache = Cache([a + b for a, b in zip(new, past)], 1, 64, 16, BF16, seed=31)
    check(cache, queries(sum(new), 2, 64, BF16), new)


def test_paged_prefill_is_the_one_token_attention_for_one_token():
    for dtype in (BF16, F32):
        cache = Cache([1, 77, 500, 3000], 2, 128, 32, dtype, seed=33)
        q = queries(4, 8, 128, dtype)
        one, lse1 = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, window=100, sinks=3, lse=True)
        out, lse = check(cache, q, [1, 1, 1, 1], window=100, sinks=3)
        assert float((out.float() - one).abs().max()) <= (2.0 ** -6 if dtype == BF16 else 2e-5)
        assert float((lse - lse1).abs().max()) <= 2e-5


def test_paged_prefill_chunks_do_not_depend_on_their_cut():
    """A prompt in one piece, in three and token by token: the same rows within the bounds of each."""
    cache = Cache([150], 2, 64, 16, F32, seed=35)
    q = queries(150, 4, 64, F32)
    whole = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, i32([0, 150]))
    for cut in ([0, 1, 66, 150], list(range(151))):
        parts = [kda.paged_prefill(q[a:b], cache.kp, cache.vp, cache.table, i32([b]), i32([0, b - a]))
                 for a, b in zip(cut, cut[1:])]
        assert float((torch.cat(parts) - whole).abs().max()) <= 1e-4


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged_prefill_repeats_bit_for_bit(dtype):
    new = [3, 200, 50]
    cache = Cache([900, 260, 4000], 2, 64, 16, dtype, seed=37)
    q = queries(sum(new), 4, 64, dtype)
    a = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu_of(new), lse=True)
    for _ in range(3):
        b = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu_of(new), lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 2, 17, 63, 64, 65, 100])
def test_paged_prefill_of_uneven_sequences(dtype, n):
    """Lengths from one to thousands in a batch, whose shares go by the lengths up to 64 sequences and by their bound
    beyond; a table much wider than any of them."""
    new = [1 + (3 * i) % 6 for i in range(n)]
    past = [(2900 * (i % 5 == 0) + 53 * i) % 3300 for i in range(n)]
    past[0] = 3000
    cache = Cache([a + b for a, b in zip(new, past)], 1, 64, 32, dtype, seed=n, extra_cols=300)
    check(cache, queries(sum(new), 4, 64, dtype, scale=1.0), new)
    check(cache, queries(sum(new), 4, 64, dtype, scale=1.0), new, max_length=max(cache.lengths), window=1500, sinks=5)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged_prefill_of_a_long_chunk_behind_short_ones(dtype):
    """Many rows: one long sequence is split, the short ones are not; more key-value heads than one."""
    new = [3, 120, 1, 40]
    cache = Cache([9, 5000, 30, 700], 3, 64, 16, dtype, seed=91)
    check(cache, queries(sum(new), 6, 64, dtype, scale=1.0), new)


@pytest.mark.parametrize("dtype,d,n,m,past", [
    (BF16, 64, 70, 20, 2500), (F32, 64, 70, 20, 1300), (BF16, 256, 66, 20, 1500),   # shares by the bound of the lengths
    (F32, 64, 40, 190, 1100), (F32, 128, 33, 250, 700),                             # a round of row tiles, uneven lengths
    (BF16, 256, 3, 30, 2500), (F32, 256, 3, 30, 900)])
def test_paged_prefill_of_many_rows_is_split_and_joined(dtype, d, n, m, past):
    hkv = 4 if n in (33, 40) else 1
    new = [m + i % 3 for i in range(n)]
    cache = Cache([a + past * (1 + i % 4) // 4 for i, a in enumerate(new)], hkv, d, 32, dtype, seed=n + d)
    group = 1 if hkv == 4 else 2
    need = kda._lib.load().kda_paged_prefill_workspace(n, sum(new), hkv * group, hkv, d, int(dtype == BF16),
                                                       max(cache.lengths), 0, 0)
    assert need > 0
    print(f"many rows {dtype} d={d} n={n}", flush=True)
    check(cache, queries(sum(new), hkv * group, d, dtype, scale=1.0), new, max_length=max(cache.lengths))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("new", [[4], [140]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_paged_prefill_visible_values_that_are_not_finite_in_wide_heads(dtype, d, new, bad):
    """In each block of channels, in tiles with hidden keys and without: they reach the rows that see them, and no other
    row or channel.  (Rows whose sums are not finite are formed again with another reference, so that the others are within
    the bound of the exact ones, not bit for bit what they are without.)"""
    cache = Cache([400], 1, d, 16, dtype, seed=13)
    q = queries(sum(new), 2, d, dtype, scale=0.2)
    exact, _, tol, _ = attention64(cache.k[0], cache.v[0], q.cpu(), 400 - new[0], d ** -0.5)
    tol = tol + STEP[dtype] * (exact.abs() + tol)
    for i in (3, 400 - new[0], 399):
        vp = cache.vp.clone()
        channels = [5, 63, d - 40, d - 1]
        for c in channels:
            vp[int(cache.table_cpu[0, i // 16]), 0, i % 16, c] = bad
        out = kda.paged_prefill(q, cache.kp, vp, cache.table, cache.len, cu_of(new)).cpu().double()
        sees = torch.arange(400 - new[0], 400) >= i
        mask = torch.zeros(d, dtype=torch.bool)
        mask[channels] = True
        want = (sees[:, None, None] & mask).expand(-1, 2, -1)
        assert torch.equal(~out.isfinite(), want), i
        assert bool(((out - exact).abs() <= tol)[~want].all()), i


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [[4], [140]])
@pytest.mark.parametrize("key", [-math.inf, -8192.0])
def test_paged_prefill_values_that_are_not_finite_with_a_weight_of_0(dtype, d, new, key):
    """A score of -inf, or one so low that its weight is 0 in fp32: the value's product with it is NaN, in tiles with hidden
    keys and without, as in the one-token attention; no other row or channel changes, nor a log-sum."""
    m = new[0]
    cache = Cache([400], 1, d, 16, dtype, seed=15)
    q = torch.full((m, 2, d), 0.0625, dtype=dtype, device=DEV)
    for i in (3, 70, 400 - m, 399):
        kp, vp = cache.kp.clone(), cache.vp.clone()
        at = (int(cache.table_cpu[0, i // 16]), 0, i % 16)
        kp[at] = key  # a score of -512 d / sqrt(d): below -4096
        clean = kda.paged_prefill(q, kp, vp, cache.table, cache.len, cu_of(new), lse=True)
        assert bool(clean[0].isfinite().all()) and bool(clean[1].isfinite().all())
        for bad in (math.inf, math.nan):
            vp[at][d - 17] = bad
            out, lse = kda.paged_prefill(q, kp, vp, cache.table, cache.len, cu_of(new), lse=True)
            want = (torch.arange(400 - m, 400) >= i)[:, None].expand(-1, 2)
            assert torch.equal(out[..., d - 17].isnan().cpu(), want), (i, bad)
            out[..., d - 17], clean[0][..., d - 17] = 0.0, 0.0
            assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
            one = kda.paged_decode(q[-1:], kp, vp, cache.table, cache.len)
            assert bool(one[..., d - 17].isnan().all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,length,first,last", [(4, 20, 0, 20), (4, 400, 0, 400), (4, 9000, 1024, 7000), (9, 9000, 0, 9000),
                                                   (140, 400, 0, 400), (140, 4000, 1024, 3000)])
def test_paged_prefill_keys_that_are_all_nan(dtype, d, new, length, first, last):
    """A row that sees nothing but such keys, in all of a sequence or in whole parts of it, has NaN outputs and a NaN
    log-sum: -inf would say that it sees no key.  The sequence next to it is what it is without."""
    cache = Cache([length, 50], 1, d, 16, dtype, seed=17)
    q = queries(new + 2, 2, d, dtype)
    cu = cu_of([new, 2])
    clean = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu, lse=True)
    for j in range(first // 16, -(-last // 16)):
        cache.kp[int(cache.table_cpu[0, j])] = math.nan
    out, lse = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu, lse=True)
    assert bool(out[:new].isnan().all()) and bool(lse[:new].isnan().all())
    assert torch.equal(out[new:], clean[0][new:]) and torch.equal(lse[new:], clean[1][new:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [[2, 1], [70, 40]])
def test_a_bound_of_0_shows_nothing(dtype, new):
    """max_length hides what lies behind it: with 0, everything, in the one-token attention too; 1 shows one token."""
    cache = Cache([200, 90], 2, 256, 16, dtype, seed=19)
    q = queries(sum(new), 4, 256, dtype)
    out, lse = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu_of(new), lse=True, max_length=0)
    one, lse1 = kda.paged_decode(q[:2], cache.kp, cache.vp, cache.table, cache.len, lse=True, max_length=0)
    for o, l in ((out, lse), (one, lse1)):
        assert not o.any() and bool(torch.isneginf(l).all())
    out = kda.paged_prefill(q, cache.kp, cache.vp, cache.table, cache.len, cu_of(new), max_length=1)
    # out = fl(fl(w v) fl(1 / w)) with the one weight w = 2^(s - fl(s)) about 1: three roundings to fp32 (3 u of v, which a
    # rounding to bf16 takes back to v; the weight's own rounding to bf16 is 1, and two bf16 are w but for 2^-17)
    first = cache.v[0][0].to(DEV).repeat_interleave(2, 0).expand(new[0], 4, 256)
    assert bool(((out[:new[0]] - first).abs() <= (4 * U * first.abs() if dtype == F32 else 0.0)).all())
