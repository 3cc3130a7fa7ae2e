"""Paged-cache attention, page bookkeeping and beam search on the GPU against plain 64-bit code.

Tolerances (u = 2^-24, the fp32 unit roundoff).  Attention, per query with n visible tokens, every
bound worst-case: a score s is a sum of d exact (bf16) or once-rounded (fp32) products, so it is off
by ds <= (d + 3) u scale sum|q k|; a weight p = exp(s - m) is off by the factor 1 +- (2 ds + w), w =
u for a weight carried as three bf16 plus 8 u for the exponential and its argument's
rounding, |s - m| <= 2 S1 included in ds; sums of n terms and of rescaled partial sums add (n + 64) u.
So |out - exact| <= vmax (4 ds + 2 w + 2 (n + 64) u) and |lse - exact| <= 2 ds + w + (n + 64) u +
4 u |lse|.  Everything that is copied or counted is compared bit for bit.
"""
import math

import pytest
import torch

import gated_delta_rule_75_amd as kda

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


class Cache:
    """Pages, a table with the pages in random order, and the plain keys and values of each sequence."""

    def __init__(self, lengths, hkv, d, page, dtype, seed=0, spare=3, garbage=float("nan"), extra_cols=0,
                 interleaved=False):
        g = gen(seed)
        self.page, self.lengths = page, list(lengths)
        need = [-(-t // page) for t in lengths]
        n_pages = sum(need) + spare
        width = max(need + [1]) + extra_cols
        ids = torch.randperm(n_pages, generator=g).tolist()
        table = torch.full((len(lengths), width), -1, dtype=torch.int32)
        kp = torch.full((n_pages, hkv, page, d), garbage, dtype=dtype)
        vp = torch.full((n_pages, hkv, page, d), garbage, dtype=dtype)
        self.k, self.v = [], []
        for n, t in enumerate(lengths):
            k = torch.randn(t, hkv, d, generator=g).to(dtype)
            v = torch.randn(t, hkv, d, generator=g).to(dtype)
            self.k.append(k)
            self.v.append(v)
            for j in range(need[n]):
                p = ids.pop()
                table[n, j] = p
                m = min(page, t - j * page)
                kp[p, :, :m] = k[j * page:j * page + m].transpose(0, 1)
                vp[p, :, :m] = v[j * page:j * page + m].transpose(0, 1)
        self.table_cpu, self.table = table, table.to(DEV)
        if interleaved:  # keys and values of a page side by side in one pool
            pool = torch.stack([kp, vp], 1).to(DEV)
            self.kp, self.vp = pool[:, 0], pool[:, 1]
        else:
            self.kp, self.vp = kp.to(DEV), vp.to(DEV)
        self.len = i32(self.lengths)


def attention64(cache, n, q, scale, window=0, sinks=0, absent=()):
    """out [Hq,d], lse [Hq] in fp64 and the error bounds of the module's docstring."""
    t = cache.lengths[n]
    hkv, d = cache.kp.shape[1], q.shape[1]
    near = max(0, t - window) if window else 0
    seen = [i for i in range(t) if (i >= near or i < sinks) and i // cache.page not in absent]
    if not seen:
        return torch.zeros(q.shape[0], d).double(), torch.full((q.shape[0],), -math.inf).double(), 0.0, 0.0
    k, v = cache.k[n][seen].double(), cache.v[n][seen].double()
    group = q.shape[0] // hkv
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)  # [n, Hq, d]
    qd = q.double()
    s = (k * qd[None]).sum(2) * scale  # [n, Hq]
    size = float(((k * qd[None]).abs().sum(2) * abs(scale)).max())
    lse = torch.logsumexp(s, 0)
    out = (torch.exp(s - lse)[..., None] * v).sum(0)
    ds = (d + 3) * U * size
    w = 9 * U
    acc = (len(seen) + 64) * U
    return (out, lse, float(v.abs().max()) * (4 * ds + 2 * w + 2 * acc),
            2 * ds + w + acc + 4 * U * float(lse.abs().max()))


def check_attention(cache, q, scale=None, window=0, sinks=0, absent=(), **kw):
    scale_used = q.shape[2] ** -0.5 if scale is None else scale
    out, lse = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, scale=scale, window=window,
                                sinks=sinks, lse=True, **kw)
    torch.cuda.synchronize()
    assert out.dtype == F32 and tuple(out.shape) == tuple(q.shape)
    worst = 0.0
    for n in range(q.shape[0]):
        want, want_lse, tol, tol_lse = attention64(cache, n, q[n].cpu(), scale_used, window, sinks, absent)
        got, got_lse = out[n].cpu().double(), lse[n].cpu().double()
        assert torch.isfinite(got).all(), n
        err = float((got - want).abs().max())
        assert err <= tol, (n, cache.lengths[n], err, tol)
        if math.isinf(float(want_lse[0])):
            assert torch.equal(got_lse, want_lse)
        else:
            assert float((got_lse - want_lse).abs().max()) <= tol_lse, (n, cache.lengths[n])
        worst = max(worst, err / tol if tol else 0.0)
    print(f"  worst error {worst:.3f} of the bound", flush=True)
    return out, lse


def queries(n, hq, d, dtype, seed=1, scale=2.0):
    return (torch.randn(n, hq, d, generator=gen(seed)) * scale).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype,hq,hkv,d,page,lengths", [
    (BF16, 8, 2, 128, 64, [1, 2, 15, 16, 17, 63, 64, 65, 127, 500]),
    (BF16, 4, 4, 64, 16, [31, 32, 33, 1, 0, 257]),      # one query head per key head; an empty sequence
    (BF16, 16, 1, 128, 16, [100, 700]),                 # all query heads share one key head
    (BF16, 20, 1, 256, 48, [1, 49, 333]),               # more than 16 heads to a key head; pages of 48
    (BF16, 35, 5, 64, 32, [95, 96, 97]),                # seven to one
    (BF16, 66, 2, 64, 16, [200, 5]),                    # 33 to one
    (BF16, 128, 1, 128, 64, [130]),
    (F32, 8, 2, 128, 64, [1, 2, 15, 16, 17, 63, 64, 65, 127, 500]),
    (F32, 5, 5, 64, 16, [31, 32, 33, 1, 0, 257]),
    (F32, 20, 1, 256, 48, [1, 49, 333]),
    (F32, 40, 2, 64, 128, [1000, 3]),
    (F32, 16, 1, 128, 4096, [600]),                     # one page holds everything
])
def test_paged_decode_matches_fp64(dtype, hq, hkv, d, page, lengths):
    print(f"paged decode {dtype} hq={hq} hkv={hkv} d={d} page={page} lengths={lengths}", flush=True)
    cache = Cache(lengths, hkv, d, page, dtype, seed=hq + d)
    check_attention(cache, queries(len(lengths), hq, d, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("length,n", [(20001, 1), (9000, 3)])
def test_paged_decode_long_sequences_are_split_and_joined(dtype, length, n):
    print(f"long {dtype} {length} x {n}", flush=True)
    cache = Cache([length - 4000 * i for i in range(n)], 2, 64, 64, dtype, seed=3)
    check_attention(cache, queries(n, 6, 64, dtype, scale=1.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 1), (33, 4), (64, 64), (100, 17), (5000, 4), (700, 0)])
def test_paged_decode_window_and_sinks(dtype, window, sinks):
    """Windows that begin inside a page, sinks that end inside one, sequences shorter than the window, and
    sinks that reach into the window."""
    print(f"window {window} sinks {sinks} {dtype}", flush=True)
    cache = Cache([1, 30, 64, 65, 99, 101, 118, 700, 1500], 2, 64, 32, dtype, seed=window)
    check_attention(cache, queries(9, 8, 64, dtype), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)])
def test_paged_decode_largest_windows_and_sinks(dtype, window, sinks):
    """The largest 32-bit window and sinks: every token is visible, without a sum that leaves 32 bits."""
    print(f"window {window} sinks {sinks} {dtype}", flush=True)
    cache = Cache([0, 1, 5, 6, 64, 700], 2, 64, 32, dtype, seed=13)
    check_attention(cache, queries(6, 8, 64, dtype), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged_decode_pages_given_back(dtype):
    """Entries without a page (-1, or beyond the pool) leave their tokens out, inside the sequence too; a
    sequence that has none left gives 0 and -inf."""
    cache = Cache([300, 300, 40], 2, 128, 32, dtype, seed=5)
    cache.table[:, 1] = -1
    cache.table[:, 4] = cache.kp.shape[0]
    cache.table[:, 6] = -2147483648
    q = queries(3, 4, 128, dtype)
    check_attention(cache, q, absent=(1, 4, 6))
    cache.table[2] = -1
    out, lse = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, lse=True)
    assert not out[2].any() and bool(torch.isneginf(lse[2]).all()) and bool(out[:2].any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), -float("inf")])
def test_paged_decode_never_uses_what_is_not_visible(dtype, garbage):
    """Slots behind the sequence, before the window and between sinks and window hold NaN or infinities."""
    cache = Cache([77, 500], 2, 64, 16, dtype, seed=9, garbage=garbage)
    q = queries(2, 8, 64, dtype)
    plain = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, window=40, sinks=5)
    for n, t in enumerate(cache.lengths):
        for i in range(5, t - 40):
            p = int(cache.table_cpu[n, i // 16])
            cache.kp[p, :, i % 16] = garbage
            cache.vp[p, :, i % 16] = garbage
    check_attention(cache, q, window=40, sinks=5)
    again = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, window=40, sinks=5)
    assert torch.equal(plain, again)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged_decode_extreme_scores(dtype):
    """One key far above the others in a late tile, scores of +-1e4, a score of -inf, a visible NaN."""
    cache = Cache([400, 400, 400, 400], 1, 64, 16, dtype, seed=11)
    q = queries(4, 4, 64, dtype)
    for n, (i, f) in enumerate([(333, 200.0), (3, -5000.0)]):
        cache.k[n][i] = (q[n, 0].cpu().float() * f).to(dtype)
        cache.kp[int(cache.table_cpu[n, i // 16]), :, i % 16] = cache.k[n][i].to(DEV)
    big = torch.zeros(64)
    big[0] = math.inf  # q[0] * inf: +-inf by the sign of the query
    p = int(cache.table_cpu[2, 10])
    q[2, :, 0] = -1.0
    cache.kp[p, 0, 4] = big.to(dtype).to(DEV)
    cache.k[2] = torch.cat([cache.k[2][:164], cache.k[2][165:]])
    cache.v[2] = torch.cat([cache.v[2][:164], cache.v[2][165:]])
    cache.kp[int(cache.table_cpu[3, 7]), 0, 3] = math.nan
    out, lse = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, lse=True)
    assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(lse[3]).all())
    for n in (0, 1):
        want, want_lse, tol, _ = attention64(cache, n, q[n].cpu(), 0.125)
        assert float((out[n].cpu().double() - want).abs().max()) <= tol
    cache.lengths[2] = 399  # the token at -inf has no weight
    cache.page = 10 ** 6
    want, want_lse, tol, _ = attention64(cache, 2, q[2].cpu(), 0.125)
    # its products with the other components of q are 0 * q: only the infinite one counts
    assert float((out[2].cpu().double() - want).abs().max()) <= tol
    all_out = torch.full((1, 64), math.inf, dtype=dtype, device=DEV)
    kp = all_out.expand(1, 1, 16, 64).contiguous()
    o, l = kda.paged_decode(-torch.ones(1, 2, 64, dtype=dtype, device=DEV), kp, kp.clone().fill_(3.0), i32([[0]]),
                            i32([9]), lse=True)
    assert not o.any() and bool(torch.isneginf(l).all())  # every visible score is -inf


def test_paged_decode_strided_queries_and_interleaved_pages():
    """q as a slice of a wider projection, keys and values side by side in one pool, a table that is a
    view of a wider one, and an out buffer."""
    cache = Cache([70, 3, 129], 2, 128, 32, BF16, seed=21, interleaved=True)
    wide = queries(3, 12, 128, BF16)
    q = wide[:, 2:10]
    table = torch.full((3, 40), -1, dtype=torch.int32, device=DEV)
    table[:, :cache.table.shape[1]] = cache.table
    cache.table = table[:, :cache.table.shape[1] + 3]
    out = torch.empty(3, 8, 128, device=DEV)
    got, _ = check_attention(cache, q, out=out)
    assert got.data_ptr() == out.data_ptr()


def test_paged_decode_max_length_and_scale():
    """max_length sizes the launch and cuts longer sequences; scale may be negative or zero."""
    cache = Cache([500, 200], 2, 64, 16, F32, seed=23)
    q = queries(2, 4, 64, F32)
    a = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len)
    b = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, max_length=500)
    assert float((a - b).abs().max()) <= 1e-5
    for scale in (-0.3, 0.0):
        check_attention(cache, q, scale=scale)
    cache.lengths, cache.k, cache.v = [123, 123], [k[:123] for k in cache.k], [v[:123] for v in cache.v]
    check_attention(cache, q, max_length=123)
    cache.len = i32([0, -5])
    out, lse = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, max_length=0, lse=True)
    assert not out.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged_decode_is_deterministic_and_does_not_depend_on_the_workspace(dtype):
    cache = Cache([9001, 40, 3000], 2, 128, 64, dtype, seed=25)
    q = queries(3, 16, 128, dtype)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)  # NaN bits
    first = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, workspace=ws, lse=True)
    ws.fill_(1)
    again = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, workspace=ws, lse=True)
    fresh = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, lse=True)
    for x, y, z in zip(first, again, fresh):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged_decode_may_read_one_pool_as_keys_and_values(dtype):
    cache = Cache([90, 33], 2, 64, 16, dtype, seed=26)
    cache.v, cache.vp = cache.k, cache.kp
    check_attention(cache, queries(2, 4, 64, dtype), workspace=torch.empty(1 << 10, 1 << 10, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,hkv,group", [(64, 3, 5), (128, 2, 40), (256, 1, 17)])
def test_paged_decode_every_length_around_tiles_and_parts(dtype, d, hkv, group):
    """Lengths 0 .. 70 and around the ends of steps and parts of a longer batch, in one call."""
    lengths = list(range(71)) + [127, 128, 129, 255, 256, 257, 511, 513, 1023, 1025, 2047, 2048, 2049, 2303]
    cache = Cache(lengths, hkv, d, 16, dtype, seed=d)
    q = queries(len(lengths), hkv * group, d, dtype)
    check_attention(cache, q)
    check_attention(cache, q, window=37, sinks=3)


def test_paged_decode_table_without_columns():
    q = queries(3, 4, 64, F32)
    pages = torch.zeros(2, 2, 16, 64, device=DEV)
    out, lse = kda.paged_decode(q, pages, pages, torch.zeros(3, 0, dtype=torch.int32, device=DEV), i32([0, 5, 9]), lse=True)
    assert not out.any() and bool(torch.isneginf(lse).all())
    out = kda.paged_decode(q[:0], pages, pages, torch.zeros(0, 3, dtype=torch.int32, device=DEV), i32([]))
    assert tuple(out.shape) == (0, 4, 64)


def test_paged_decode_offsets_beyond_32_bits():
    """Pages whose byte offset (and element offset) passes 2^32, in a pool reserved but mostly untouched."""
    page, hkv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * hkv * d) + 700  # elements beyond 2^32
    kp = torch.empty(n_pages, hkv, page, d, dtype=BF16, device=DEV)
    vp = torch.empty(n_pages, hkv, page, d, dtype=BF16, device=DEV)
    cache = Cache([150], hkv, d, page, BF16, seed=27, spare=0)
    far = [n_pages - 1, n_pages - 600, 5]
    for j, p in enumerate(far):
        old = int(cache.table_cpu[0, j])
        kp[p], vp[p] = cache.kp[old], cache.vp[old]
        cache.table[0, j] = p
    cache.kp, cache.vp = kp, vp
    check_attention(cache, queries(1, 16, d, BF16))
    k, v = queries(1, hkv, d, BF16, seed=2), queries(1, hkv, d, BF16, seed=3)
    kda.cache_append(k, v, kp, vp, cache.table, i32([100]))
    assert torch.equal(kp[far[1], :, 36], k[0]) and torch.equal(vp[far[1], :, 36], v[0])
    kda.pages_copy([kp, vp], i32([[far[1], 9]]))
    assert torch.equal(kp[9], kp[far[1]]) and torch.equal(vp[9], vp[far[1]])


# ------------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------------
def append_plain(kp, vp, table, start, k, v, cu, page):
    for n in range(len(start)):
        for i in range(cu[n + 1] - cu[n]):
            pos = start[n] + i
            if pos < 0 or pos // page >= table.shape[1]:
                continue
            p = int(table[n, pos // page])
            if 0 <= p < kp.shape[0]:
                kp[p, :, pos % page] = k[cu[n] + i]
                vp[p, :, pos % page] = v[cu[n] + i]


@pytest.mark.parametrize("dtype,hkv,d,page,start,new", [
    (BF16, 2, 128, 64, [0, 5, 63, 64, 100], [1, 0, 2, 130, 28]),
    (BF16, 3, 64, 16, [0, 17, 3], [50, 1, 33]),
    (F32, 1, 256, 48, [40, 0], [20, 97]),
    (F32, 8, 64, 32, [0, 31, 2], [300, 1, 0]),
    (BF16, 128, 256, 16, [3], [20]),
])
def test_cache_append_segments(dtype, hkv, d, page, start, new):
    """Packed segments, empty ones among them; only the slots of the new tokens change."""
    print(f"append {dtype} hkv={hkv} d={d} page={page} start={start} new={new}", flush=True)
    total = [a + b for a, b in zip(start, new)]
    cache = Cache(total, hkv, d, page, dtype, seed=d, garbage=7.0)
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    g = gen(4)
    k, v = (torch.randn(cu[-1], hkv, d, generator=g).to(dtype) for _ in range(2))
    kp, vp = cache.kp.cpu(), cache.vp.cpu()
    append_plain(kp, vp, cache.table_cpu, start, k, v, cu, page)
    kda.cache_append(k.to(DEV), v.to(DEV), cache.kp, cache.vp, cache.table, i32(start), cu_seqlens=i32(cu))
    assert torch.equal(cache.kp.cpu(), kp) and torch.equal(cache.vp.cpu(), vp)


def test_cache_append_one_token_each_from_a_fused_projection():
    cache = Cache([1, 64, 65, 300], 2, 128, 64, BF16, seed=31, garbage=1.0)
    qkv = queries(4, 8, 128, BF16)  # queries, keys and values side by side
    k, v = qkv[:, 4:6], qkv[:, 6:8]
    start = [0, 63, 64, 299]
    kp, vp = cache.kp.cpu(), cache.vp.cpu()
    append_plain(kp, vp, cache.table_cpu, start, k.cpu(), v.cpu(), list(range(5)), 64)
    kda.cache_append(k, v, cache.kp, cache.vp, cache.table, i32(start))
    assert torch.equal(cache.kp.cpu(), kp) and torch.equal(cache.vp.cpu(), vp)


def test_cache_append_drops_positions_without_a_page():
    """Before 0, behind the table, entries that name no page: nothing else is written."""
    cache = Cache([64, 64, 64], 2, 64, 16, BF16, seed=33, garbage=1.0)
    cache.table[1, 2] = -1
    cache.table[2, 0] = cache.kp.shape[0]
    table = cache.table.cpu()
    start, new = [-3, 20, 0], [6, 60, 20]
    cu = [0, 6, 66, 86]
    k, v = queries(86, 2, 64, BF16, seed=5), queries(86, 2, 64, BF16, seed=6)
    kp, vp = cache.kp.cpu(), cache.vp.cpu()
    append_plain(kp, vp, table, start, k.cpu(), v.cpu(), cu, 16)
    kda.cache_append(k, v, cache.kp, cache.vp, cache.table, i32(start), cu_seqlens=i32(cu))
    assert torch.equal(cache.kp.cpu(), kp) and torch.equal(cache.vp.cpu(), vp)
    kda.cache_append(k[:0], v[:0], cache.kp, cache.vp, cache.table, i32(start), cu_seqlens=i32([0, 0, 0, 0]))
    kda.cache_append(k, v, cache.kp, cache.vp, cache.table, i32(start), cu_seqlens=i32([0, 0, 0, 0]))  # all behind
    assert torch.equal(cache.kp.cpu(), kp)


# ------------------------------------------------------------------------------------------------
# pages
# ------------------------------------------------------------------------------------------------
def counts(table, n_pages):
    refs = [0] * n_pages
    for row in table:
        for e in row:
            if 0 <= e < n_pages:
                refs[e] += 1
    return refs


def reserve_plain(table, lengths, refs, new, page):
    """include/kda.h's words, one sequence after another."""
    free = [p for p, r in enumerate(refs) if r == 0]
    before = list(refs)
    copies, granted, taken = [], [], 0
    for n, add in enumerate(new):
        copies.append([-1, -1])
        granted.append(0)
        if add <= 0:
            continue
        cols = list(range(lengths[n] // page, (lengths[n] + add - 1) // page + 1))
        if cols[-1] >= len(table[n]):
            continue
        want = [j for j in cols if not 0 <= table[n][j] < len(refs) or before[table[n][j]] > 1]
        taken += len(want)
        if taken > len(free):
            continue
        for j, p in zip(want, free[taken - len(want):taken]):
            old = table[n][j]
            table[n][j] = p
            refs[p] = 1
            if 0 <= old < len(refs):
                refs[old] -= 1
                if j == cols[0] and lengths[n] % page:
                    copies[n] = [old, p]
        lengths[n] += add
        granted[n] = add
    return copies, granted


def random_tables(rng, n, width, n_pages, page, share=0.4):
    """Tables whose sequences share random beginnings."""
    table, lengths, left = [], [], list(range(n_pages))
    rng.shuffle(left)
    for i in range(n):
        t = rng.randrange(0, width * page + 1)
        cols = -(-t // page)
        row = []
        if i and rng.random() < share:
            row = [e for e in table[rng.randrange(i)][:rng.randrange(width + 1)] if e >= 0][:cols]
        while len(row) < cols and left:
            row.append(left.pop())
        t = min(t, len(row) * page)
        lengths.append(t)
        table.append(row + [-1] * (width - len(row)))
    return table, lengths


@pytest.mark.parametrize("seed,n,width,n_pages,page", [(1, 5, 4, 40, 16), (2, 70, 9, 300, 16), (3, 33, 300, 9000, 48),
                                                       (4, 1, 1, 2, 64), (5, 20, 6, 60, 32), (6, 300, 70, 20000, 16),
                                                       (7, 12, 40, 8192, 16), (8, 12, 40, 8193, 16)])
def test_fork_reserve_free_match_a_plain_cache(seed, n, width, n_pages, page):
    """A life of a cache: forks (rows dropped, kept, repeated, moved, wrong indices), reservations until the
    pages run out, drops (rows named twice, wrong indices); tables, lengths and counts after each step."""
    import random

    print(f"cache life seed={seed} n={n} width={width} pages={n_pages} page={page}", flush=True)
    rng = random.Random(seed)
    table, lengths = random_tables(rng, n, width, n_pages, page)
    refs = counts(table, n_pages)
    T, L, R = i32(table), i32(lengths), i32(refs)
    for step in range(4):
        m = rng.randrange(1, 2 * n + 2)
        parents = [rng.choice([rng.randrange(-2, n + 2), i % n]) for i in range(m)]
        old, old_len = table, lengths
        table = [list(old[p]) if 0 <= p < n else [-1] * width for p in parents]
        lengths = [old_len[p] if 0 <= p < n else 0 for p in parents]
        before, after = counts(old, n_pages), counts(table, n_pages)
        refs = [r - b + a for r, b, a in zip(refs, before, after)]
        T, L = kda.cache_fork(T, L, R, i32(parents))
        assert T.tolist() == table and L.tolist() == lengths and R.tolist() == refs
        n = m
        new = [rng.choice([0, 1, 1, page, rng.randrange(-1, 3 * page)]) for _ in range(n)]
        copies, granted = reserve_plain(table, lengths, refs, new, page)
        C, G = kda.cache_reserve(T, L, R, i32(new), page)
        assert G.tolist() == granted and C.tolist() == copies
        assert T.tolist() == table and L.tolist() == lengths and R.tolist() == refs
        rows = [rng.randrange(-1, n + 1) for _ in range(max(1, n // 3))]
        rows += rows[:2]
        for r in set(rows):
            if 0 <= r < n:
                for e in table[r]:
                    if e >= 0:
                        refs[e] -= 1
                table[r], lengths[r] = [-1] * width, 0
        kda.cache_free(T, L, R, i32(rows))
        assert T.tolist() == table and L.tolist() == lengths and R.tolist() == refs
        assert refs == counts(table, n_pages)


def test_reserve_when_pages_or_columns_run_out():
    """Served in order while the pages last; a sequence that is not served is left as it was."""
    table = [[0, 1, -1], [0, 1, -1], [2, -1, -1], [3, 4, 5]]
    lengths, refs = [20, 20, 16, 48], counts([[0, 1], [0, 1], [2], [3, 4, 5]], 8)
    T, L, R = i32(table), i32(lengths), i32(refs)
    # free: 6, 7.  Sequence 0 needs a copy of page 1, sequence 1 one and another page, sequence 2 one,
    # sequence 3 has no column left
    new = [3, 13, 1, 1]
    want = reserve_plain(table, lengths, refs, new, 16)
    C, G = kda.cache_reserve(T, L, R, i32(new), 16)
    assert (C.tolist(), G.tolist()) == want == ([[1, 6], [-1, -1], [-1, -1], [-1, -1]], [3, 0, 0, 0])
    assert T.tolist() == table and L.tolist() == lengths and R.tolist() == refs
    assert T.tolist()[1] == [0, 1, -1] and L.tolist()[1] == 20


@pytest.mark.parametrize("n,width,n_pages", [(5, 9, 40), (5, 200, 600), (40, 200, 2500), (5, 200, 9000)])
def test_reserve_leaves_a_sequence_that_is_not_served_as_it_was(n, width, n_pages):
    """Entries that name no page (-1, other negative numbers, those of pages that there are and not, numbers
    beyond the pool) stand in the columns to come of every sequence, next to shared and own pages.  Two
    sequences are served, the third needs more pages than there are, so it and those behind it keep every
    entry; so does one whose row is too narrow.  One workgroup and two launches, columns behind the 64th."""
    page, half = 16, width // 2
    none = [-1, -2, -3, -2147483648, n_pages, 2147483647, -2 - (n_pages - 1), -7]
    free = 2 * width + 3
    own = list(range(free, n_pages))  # the others are in use: each row has two of its own, shared ones twice
    table, refs = [], [0] * n_pages
    for r in range(n):
        row = [none[(r + j) % len(none)] for j in range(width)]
        row[half], row[half + 1] = own[0], own[1 + r]
        table.append(row)
    for p in own:
        refs[p] = 1
    refs[own[0]] = n
    lengths = [3] * n
    new = [width * page - 3] * n  # every column: a sequence takes all but its own page
    new[1] = (width - 1) * page
    new[3] = width * page - 2  # one token too many for the row
    if n > 5:
        new[5:] = [page] * (n - 5)
    want_table, want_len, want_refs = [list(r) for r in table], list(lengths), list(refs)
    want_c, want_g = reserve_plain(want_table, want_len, want_refs, new, page)
    assert want_g[0] == new[0] and want_g[1:4] == [new[1], 0, 0] and not any(want_g[3:])
    assert want_table[2:] == table[2:]
    T, L, R = i32(table), i32(lengths), i32(refs)
    C, G = kda.cache_reserve(T, L, R, i32(new), page)
    assert C.tolist() == want_c and G.tolist() == want_g and L.tolist() == want_len
    assert T.tolist() == want_table and R.tolist() == want_refs


@pytest.mark.parametrize("n,free", [(4099, 10 ** 6), (70001, 60000), (70001, 10 ** 6), ((1 << 22) + 3, 5 * 10 ** 6)])
def test_reserve_for_many_sequences(n, free):
    """Up to millions of sequences of two columns, of which some ask for nothing and some for more than their
    row holds; pages for all, or for the first ones.  (The sums over the sequences before each one have to
    grow with the sequences, not with their square.)"""
    g = gen(n)
    n_pages = 9 * 10 ** 6
    refs = torch.ones(n_pages, dtype=torch.int32)
    refs[torch.randperm(n_pages, generator=g)[:free]] = 0
    new = torch.randint(-5, 40, (n,), generator=g, dtype=torch.int32)
    refs, new = refs.to(DEV), new.to(DEV)
    ids = torch.nonzero(refs == 0).flatten()
    need = torch.where((new > 0) & (new <= 32), (new + 15) // 16, 0).long()
    base = torch.cumsum(need, 0) - need
    served = (need > 0) & (base + need <= free)
    want = torch.full((n, 2), -1, dtype=torch.int32, device=DEV)
    for j in (0, 1):
        has = served & (need > j)
        want[has, j] = ids[(base + j)[has]].to(torch.int32)
    want_refs = refs.clone()
    want_refs[want[want >= 0].long()] = 1
    table = torch.full((n, 2), -1, dtype=torch.int32, device=DEV)
    lengths = torch.zeros(n, dtype=torch.int32, device=DEV)
    copies, granted = kda.cache_reserve(table, lengths, refs, new, 16)
    assert torch.equal(table, want) and torch.equal(refs, want_refs) and bool((copies == -1).all())
    assert torch.equal(granted, torch.where(served, new, 0)) and torch.equal(lengths, granted)


def test_cache_calls_leave_the_rest_of_wider_buffers_alone():
    wide = torch.full((4, 20), 77, dtype=torch.int32, device=DEV)
    T = wide[:, 4:9]
    T.copy_(i32([[0, -1, -1, -1, -1]] * 4))
    L, R = i32([3, 3, 3, 3]), i32([4, 0, 0, 0, 0, 0])
    out = torch.full((2, 30), 55, dtype=torch.int32, device=DEV)
    kda.cache_reserve(T, L, R, i32([1, 1, 0, 1]), 16)
    assert R.tolist() == [1, 1, 1, 1, 0, 0] and T[:, 0].tolist() == [1, 2, 0, 3]
    kda.cache_fork(T, L, R, i32([3, 3]), table_out=out[:, 1:6])
    assert R.tolist() == [0, 0, 0, 2, 0, 0]
    assert bool((wide[:, :4] == 77).all()) and bool((wide[:, 9:] == 77).all())
    assert bool((out[:, 0] == 55).all()) and bool((out[:, 6:] == 55).all())
    assert out[:, 1:6].tolist() == [[3, -1, -1, -1, -1]] * 2


@pytest.mark.parametrize("n_pages,live,rows,width", [(1, 1.0, 1, 1), (2, 0.5, 1, 3), (64, 0.5, 3, 20), (65, 0.9, 2, 40),
                                                     (4096, 0.3, 40, 40), (4097, 0.7, 7, 600), (20000, 0.05, 300, 7),
                                                     (9001, 1.0, 4, 3000), (777, 0.0, 3, 4), (300, 0.6, 60, 300),
                                                     (8192, 0.6, 3, 700), (8193, 0.6, 3, 700)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_matches_plain(n_pages, live, rows, width, in_place):
    import random

    rng = random.Random(n_pages + rows)
    pages = rng.sample(range(n_pages), int(n_pages * live))
    table = [[rng.choice(pages) if pages and rng.random() < 0.8 else -1 for _ in range(width)] for _ in range(rows)]
    refs = [0] * n_pages
    for p in pages:
        refs[p] = rng.randrange(1, 5)
    used = sum(r > 0 for r in refs)
    holes = [p for p in range(used) if refs[p] == 0]
    movers = [p for p in range(used, n_pages) if refs[p] > 0]
    to = dict(zip(movers, holes))
    T, R = i32(table), i32(refs)
    data = torch.randint(0, 100, (n_pages, 4, 8), dtype=torch.int32, generator=gen(1))
    pool = data.to(DEV)
    T2, R2, M = kda.cache_compact(T, R, **(dict(table_out=T, refcount_out=R) if in_place else {}))
    want = list(refs)
    for a, b in to.items():
        want[a], want[b] = 0, refs[a]
    assert M.tolist() == [[a, b] for a, b in to.items()] + [[-1, -1]] * (n_pages // 2 - len(to))
    assert T2.tolist() == [[to.get(e, e) for e in row] for row in table] and R2.tolist() == want
    if not in_place:
        assert T.tolist() == table and R.tolist() == refs
    kda.pages_copy(pool, M)
    got = pool.cpu()
    for a, b in to.items():
        assert torch.equal(got[b], data[a])
    for p in range(used):
        if refs[p]:
            assert torch.equal(got[p], data[p])


@pytest.mark.parametrize("shapes", [
    [((50, 2, 16, 64), BF16)],
    [((50, 3, 16, 128), F32), ((50, 16), torch.uint8), ((50, 5, 4096, 4), F32)],  # sizes apart, one above 64 KiB
    [((50, 4, 4), F32)] * 35,  # more buffers than one launch takes
])
def test_pages_copy(shapes):
    pools = [torch.randn(s, generator=gen(i)).mul(50).to(t).to(DEV) for i, (s, t) in enumerate(shapes)]
    pairs = [[3, 4], [-1, -1], [7, 49], [3, 0], [50, 1], [2, 50], [-5, 2], [10, 10], [7, 20], [5, -1]]
    want = [p.cpu().clone() for p in pools]
    for w in want:
        for a, b in ([3, 4], [7, 49], [3, 0], [7, 20]):
            w[b] = w[a]
    kda.pages_copy(pools, i32(pairs))
    for p, w in zip(pools, want):
        assert torch.equal(p.cpu(), w)
    kda.pages_copy(pools, i32(pairs)[:0])
    kda.pages_copy([], i32(pairs))


def test_pages_copy_of_strided_pools_and_states():
    """Pages of keys and values in one buffer, and recurrent states as pages."""
    pool = torch.randn(6, 2, 2, 16, 64, generator=gen(1)).to(BF16).to(DEV)
    want = pool.cpu().clone()
    want[5, 1] = want[0, 1]
    kda.pages_copy(pool[:, 1], i32([[0, 5]]))
    assert torch.equal(pool.cpu(), want)
    states = torch.randn(9, 4, 128, 128, generator=gen(2)).to(DEV)
    want = states.cpu().clone()
    want[8] = want[1]
    kda.pages_copy(states, i32([[1, 8], [-1, 3]]))
    assert torch.equal(states.cpu(), want)


def test_pages_copy_of_lists_longer_than_a_launch():
    """More than 2^26 workgroups of 64 threads, which is more than a grid holds: two slices of the list.  Pages of
    2 MiB are 512 pieces, so 2^20 + 9 pairs an eighth apart make 2^26 + 1024 workgroups."""
    pool = torch.randn(24, 1 << 19, generator=gen(3)).to(DEV)
    n = (1 << 20) + 9
    pairs = torch.full((n, 2), -1, dtype=torch.int32)
    apart = -(-n // 8)
    want = pool.clone()
    # the list's ends, and both sides of the slices' border in every eighth of it
    at = [0, n - 1] + [i * apart + x for i in range(8) for x in (((1 << 26) - 1) // 512 - 1, ((1 << 26) - 1) // 512)]
    at = sorted({x for x in at if x < n})
    assert len(at) == 16 and apart * 512 > (1 << 26) - 1
    for to, x in enumerate(at, start=6):
        pairs[x] = torch.tensor([to % 6, to], dtype=torch.int32)
        want[to] = want[to % 6]
    kda.pages_copy(pool, pairs.to(DEV))
    assert torch.equal(pool, want)


# ------------------------------------------------------------------------------------------------
# beam search
# ------------------------------------------------------------------------------------------------
def select_plain(logits, scores, n_out, finished=None, eos=-1):
    """include/kda.h's order: inside a beam by (logit, -token), over the beams by (c, -beam)."""
    B, K, V = logits.shape
    res = []
    for b in range(B):
        cand = []
        for k in range(K):
            x = logits[b, k].double()
            x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
            if finished is not None and finished[b, k]:
                x = torch.full_like(x, -math.inf)
                x[eos] = 0.0
                lse = torch.zeros(())
            else:
                lse = torch.logsumexp(x, 0)
            order = torch.sort(x + 0.0, descending=True, stable=True).indices[:n_out].tolist()
            for r, t in enumerate(order):
                c = float(scores[b, k].double() + x[t] - lse)
                cand.append((-(-math.inf if math.isnan(c) else c), k, r, t))
        cand.sort()
        res.append([(-c, k, t) for c, k, r, t in cand[:n_out]])
    return res


def check_select(logits, scores, n_out=None, finished=None, eos=-1):
    """Tokens and beams are compared exactly, but for the order of different beams whose c is closer than
    the log-sums can tell.  A log-sum is a running fp32 sum: with t = x - m, a term is off by the factor
    1 +- (2 |t| + 2) u (rounding of t and of its product with log2 e, one step of the exponential), where the
    terms' weighted mean of |t| is at most ln V < 17; a thread adds 16 terms a round and rescales
    once, V / 4096 rounds at most, and the joins add 64 u.  So it is off by less than tol = (19 V / 4096 +
    100) u, c adds 4 u |c| in the fp32 result, and two beams can change places only if their c are within 2
    tol.  Inside a beam the order is exact."""
    B, K, V = logits.shape
    n = K if n_out is None else n_out
    args = (logits.cpu(), scores.cpu(), None if finished is None else finished.cpu())
    want = select_plain(args[0], args[1], n, args[2], eos)
    every = None
    s, p, t, over = kda.beam_select(logits, scores, n_out=n_out, finished=finished, eos=eos)
    assert tuple(s.shape) == (B, n)
    sum_tol = (19 * V / 4096 + 100) * U
    for b in range(B):
        got = list(zip(p[b].tolist(), t[b].tolist()))
        assert len(set(got)) == n
        if got != [(k, x) for _, k, x in want[b]]:
            if every is None:  # all candidates that can take part, in exact order
                every = select_plain(args[0], args[1], K * n, args[2], eos)
            c_of = {(k, x): c for c, k, x in every[b]}
            for o, kx in enumerate(got):
                c, k, x = want[b][o]
                assert kx == (k, x) or (kx[0] != k and abs(c_of[kx] - c) <= 2 * sum_tol), (b, o, kx, want[b][o])
            for k in range(K):  # each beam's own best, in order
                mine = [x for kk, x in got if kk == k]
                assert mine == [x for _, kk, x in every[b] if kk == k][:len(mine)]
        for o in range(n):
            c, k, x = want[b][o]
            val = float(s[b, o])
            tol = 3 * sum_tol + 4 * U * abs(c) if math.isfinite(c) else 0.0
            assert val == c or abs(val - c) <= tol, (b, o, val, c)
            if finished is not None:
                assert bool(over[b, o]) == (bool(finished[b, got[o][0]]) or got[o][1] == eos)
    assert (over is None) == (finished is None)


@pytest.mark.parametrize("dtype,B,K,V,n_out", [
    (F32, 1, 1, 1, 1), (F32, 2, 3, 7, 3), (BF16, 1, 4, 5, 20), (F32, 3, 5, 1000, 5), (BF16, 3, 5, 1001, 10),
    (BF16, 2, 8, 4096, 8), (F32, 2, 8, 4097, 8), (F32, 1, 4, 32000, 4), (BF16, 4, 16, 50257, 32), (F32, 1, 64, 513, 64),
    (BF16, 1, 1, 300000, 64), (BF16, 1, 2, 4089, 2), (F32, 2, 64, 9000, 64), (BF16, 40, 2, 2047, 4),
])
def test_beam_select_matches_plain(dtype, B, K, V, n_out):
    print(f"select {dtype} B={B} K={K} V={V} n_out={n_out}", flush=True)
    g = gen(V + K)
    logits = (torch.randn(B, K, V, generator=g) * 3).to(dtype).to(DEV)
    scores = (torch.randn(B, K, generator=g) * 1.5 - 10).to(DEV)
    check_select(logits, scores, n_out)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_beam_select_ties_and_masks(dtype):
    """Equal logits (the lower token and beam), rows with fewer tokens above -inf than places, NaN,
    beams that do not take part, all of it -inf, infinities."""
    g = gen(3)
    flat = torch.zeros(2, 4, 9000, dtype=dtype, device=DEV)
    check_select(flat, torch.zeros(2, 4, device=DEV), 8)  # everything ties
    few = torch.full((3, 4, 5000), -math.inf, dtype=dtype)
    few[:, :, 4321] = 1.0
    few[:, 1, 77] = 2.0
    few[0, 2] = -math.inf  # a beam with nothing
    few[1, 3, 10] = math.nan
    few[2, 0, 4999] = math.inf
    scores = (torch.randn(3, 4, generator=g) - 3).to(DEV)
    for n_out in (4, 16, 64):
        check_select(few.to(DEV), scores, n_out)
    check_select(torch.full((2, 3, 700), math.nan, dtype=dtype, device=DEV), torch.zeros(2, 3, device=DEV), 5)
    first = torch.full((2, 8), -math.inf)
    first[:, 0] = 0.0  # the first step: one beam takes part
    logits = (torch.randn(2, 8, 20000, generator=g) * 2).to(dtype).to(DEV)
    check_select(logits, first.to(DEV), 8)
    steps = torch.arange(2 * 2 * 30000, dtype=F32).view(2, 2, 30000) * 1e-4  # ascending
    check_select(steps.to(dtype).to(DEV), torch.zeros(2, 2, device=DEV), 16)
    wild = (torch.randn(2, 4, 40000, generator=g) * 3).to(dtype)  # NaN and infinities here and there, huge values
    wild[0, 0, 12345], wild[0, 1, 7] = math.nan, -math.inf
    wild[0, 2, ::2] = math.nan
    wild[0, 3] = math.nan
    wild[0, 3, 39999] = -2.0
    wild[1, 0, 30000], wild[1, 1, 30001] = 3.2e38, math.inf
    wild[1, 2] = -3e38
    wild[1, 2, 5] = -2.9e38
    for n_out in (4, 40):
        check_select(wild.to(DEV), torch.tensor([[0.0, -1.0, 0.5, 0.2]] * 2, device=DEV), n_out)
    zeros = torch.where(torch.arange(8192) % 2 == 0, torch.tensor(-0.0), torch.tensor(0.0))
    check_select(zeros.expand(1, 2, 8192).contiguous().to(dtype).to(DEV), torch.zeros(1, 2, device=DEV), 4)


def far_rows(tops, V, g):
    """Rows that have their maximum at every hundredth token and values a few steps below it elsewhere."""
    m = torch.tensor(tops, dtype=F32).view(-1, 4, 1)
    below = m - m.abs() * torch.randint(1, 40, (1, 1, V), generator=g) * 2.0 ** -22
    assert bool((below < m).all())
    return torch.where(torch.arange(V) % 100 == 7, m, below)


def both_signs(n, e, g):
    return ((1 + torch.rand(n, generator=g)) * 2.0 ** e * torch.tensor([1.0, -1.0] * (n // 2))).tolist()


def test_beam_select_row_maxima_far_beyond_one():
    """Row maxima m of 2^20 .. 2^33 of both signs: m log2 e and its fp32 rounding then differ by 2^-5 .. 2^9, so
    a factor that makes up for the rounding leaves the range of the exponential (at 2119338368 and
    -1621624704 one of two factors is 0 and the other finite, and the log-sum -inf).  Bounds as in check_select:
    its fp64 sums of score, logit and log-sum are off by 6 * 2^-53 * 2^33 < 6e-6 at most, within its 3 tol."""
    g = gen(12)
    tops = [2119338368.0, -1621624704.0, 2.0 ** 24, -2.0 ** 24, 2.0 ** 24 - 1, 1.0 - 2.0 ** 24, 1e6, -1e6]
    for e in range(20, 33):
        tops += both_signs(8, e, g)
    logits = far_rows(tops, 300, g)
    scores = (torch.randn(logits.shape[0], 4, generator=g) - 3).to(DEV)
    check_select(logits.to(DEV), scores, 4)
    check_select(logits.to(BF16).to(DEV), scores, 4)


def test_beam_select_row_maxima_up_to_2_to_40():
    """As above for 2^28 .. 2^40, where a step of the logits is 64 or more: only the three maxima of a row have
    weight, and c = score - log 3 for each.  The fp64 sum score + m - (m + log 3) is off by 4 roundings of
    2^-53 |m|, the log of the fp32 sum by (100 + 2) u (check_select's tol without its rounds), the fp32 result
    by u |c|."""
    g = gen(13)
    tops = [1e10, -1e10, 2119338368.0, -1621624704.0]
    for e in range(28, 40):
        tops += both_signs(64, e, g)
    logits = far_rows(tops, 300, g)
    scores = torch.randn(logits.shape[0], 4, generator=g) - 3
    got = kda.beam_select(logits.to(DEV), scores.to(DEV))[0].cpu().double()
    top = torch.sort(scores.double(), dim=1, descending=True).values
    want = torch.stack([top[:, 0], top[:, 0], top[:, 0], top[:, 1]], 1) - math.log(3.0)
    far = logits.abs().amax((1, 2)).double()[:, None]
    tol = 4 * 2.0 ** -53 * far + 102 * U + U * want.abs()
    worst = float(((got - want).abs() / tol).max())
    assert worst <= 1, worst


@pytest.mark.parametrize("kind", [torch.uint8, torch.bool])
def test_beam_select_finished_beams(kind):
    g = gen(5)
    logits = (torch.randn(4, 6, 6000, generator=g) * 3).to(DEV)
    scores = (torch.randn(4, 6, generator=g) * 2 - 8).to(DEV)
    finished = (torch.rand(4, 6, generator=g) < 0.5)
    finished[0] = True  # all: their end tokens, then the first tokens at -inf
    finished[1] = False
    logits[2, :, 2] += 30.0  # the end token is what everybody wants
    done = finished.to(kind).to(DEV)
    for eos in (2, 0, 5999):
        check_select(logits, scores, 6, done, eos)
        check_select(logits, scores, 20, done, eos)
    logits[finished.to(DEV)] = math.nan  # not read
    check_select(logits, scores, 6, done, 2)


def test_beam_select_rows_of_a_padded_vocabulary():
    """Rows that are not 16-byte aligned, inside a wider buffer whose padding must not take part."""
    g = gen(6)
    for dtype, V, pad in ((BF16, 5001, 7), (F32, 12345, 2), (BF16, 8190, 1), (F32, 4099, 1)):
        wide = torch.full((2, 3, V + pad), 1e4)
        wide[:, :, 1:V + 1 if pad > 1 else V] = torch.randn(2, 3, V if pad > 1 else V - 1, generator=g)
        wide = wide.to(dtype).to(DEV)
        logits = wide[:, :, 1:V + 1] if pad > 1 else wide[:, :, 1:V]
        check_select(logits, torch.zeros(2, 3, device=DEV), 5)


@pytest.mark.parametrize("B,K,row", [(1, 1, (4,)), (3, 2, (2, 64, 64)), (5, 4, (4,)), (2, 8, (3, 128, 64)),
                                     (2, 16, (1028,)), (1, 32, (40, 100)), (2, 64, (33, 16))])
def test_beam_reorder(B, K, row):
    """In place, repeated and kept parents, wrong ones (the row stays); two states of different sizes."""
    g = gen(K)
    a = torch.randn(B * K, *row, generator=g).to(DEV)
    b = torch.randn(B * K, 8, generator=g).to(BF16).to(DEV)
    parents = torch.randint(-1, K + 1, (B, K), generator=g, dtype=torch.int32)
    at = [bb * K + (int(p) if 0 <= p < K else k) for bb in range(B) for k, p in enumerate(parents[bb])]
    want_a, want_b = a.cpu()[at], b.cpu()[at]
    kda.beam_reorder([a, b], parents.to(DEV))
    assert torch.equal(a.cpu(), want_a) and torch.equal(b.cpu(), want_b)
    kda.beam_reorder(a, torch.arange(K, dtype=torch.int32, device=DEV).expand(B, K).contiguous())
    assert torch.equal(a.cpu(), want_a)


def test_beam_reorder_of_more_groups_than_a_launch():
    """2^24 + 5 groups of two short rows: more workgroups of 256 threads than a grid holds."""
    B = (1 << 24) + 5
    a = torch.arange(4 * 2 * B, dtype=torch.int32, device=DEV).view(B, 2, 4)
    parents = torch.randint(-1, 3, (B, 2), generator=gen(4), dtype=torch.int32).to(DEV)
    keep = torch.arange(2, device=DEV)
    at = torch.where((parents >= 0) & (parents < 2), parents, keep).long()
    want = torch.gather(a, 1, at[:, :, None].expand(B, 2, 4))
    states = a.view(2 * B, 4).clone()
    kda.beam_reorder(states, parents)
    assert torch.equal(states.view(B, 2, 4), want)


# ------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------
class Hybrid:
    """A toy hybrid layer stack's serving state: one recurrent layer (states) and one attention layer (pages),
    with fixed random projections from tokens; fp32 throughout."""

    def __init__(self, B, K, V, seed):
        g = gen(seed)
        self.B, self.K, self.V, self.h, self.d = B, K, V, 2, 64
        self.emb = {n: torch.randn(V, self.h, self.d, generator=g) for n in ("q", "k", "v", "aq", "ak", "av")}
        for n in ("q", "k"):
            self.emb[n] = self.emb[n] / self.emb[n].norm(dim=-1, keepdim=True)
        self.emb["g"] = -0.1 * torch.rand(V, self.h, self.d, generator=g)
        self.emb["beta"] = torch.rand(V, self.h, generator=g)
        self.out = torch.randn(2 * self.h * self.d, V, generator=g) * 0.6


def test_beam_search_over_states_and_pages():
    """Beam search of a hybrid stack, step by step: append, attend, recurrent step, select, fork, reserve
    and copy, reorder.  The plain search keeps every beam's tokens and states in fp64 without pages; the
    chosen tokens and beams are the same, the scores within 1e-3 (fp32 layers, sums of 12 steps), and at the
    end no page is lost."""
    B, K, V, page, steps = 3, 4, 50, 16, 40
    m = Hybrid(B, K, V, 8)
    n, h, d = B * K, m.h, m.d
    e = {x: y.to(DEV) for x, y in m.emb.items()}
    proj = m.out.to(DEV)
    n_pages, width = 200, 8
    kp, vp = torch.zeros(n_pages, h, page, d, device=DEV), torch.zeros(n_pages, h, page, d, device=DEV)
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    lengths = torch.zeros(n, dtype=torch.int32, device=DEV)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    state = torch.zeros(n, h, d, d, device=DEV)
    ones = torch.ones(n, dtype=torch.int32, device=DEV)
    scores = torch.full((B, K), -math.inf, device=DEV)
    scores[:, 0] = 0.0
    finished = torch.zeros(B, K, dtype=torch.bool, device=DEV)
    token = torch.zeros(n, dtype=torch.long, device=DEV)
    base = (torch.arange(B, dtype=torch.int32, device=DEV) * K)[:, None]
    # the plain search
    em = {x: y.double() for x, y in m.emb.items()}
    plain = [[dict(s=0.0 if k == 0 else -math.inf, toks=[0], S=torch.zeros(h, d, d).double(), done=False)
              for k in range(K)] for _ in range(B)]

    def plain_step(beam):
        t = beam["toks"][-1]
        q, k, v = em["q"][t], em["k"][t], em["v"][t]
        S = torch.exp(em["g"][t])[:, :, None] * beam["S"]
        u = torch.einsum("hkv,hk->hv", S, k)
        beam["S"] = S + em["beta"][t][:, None, None] * k[:, :, None] * (v - u)[:, None, :]
        o1 = torch.einsum("hkv,hk->hv", beam["S"], q)
        ks, vs = em["ak"][beam["toks"]], em["av"][beam["toks"]]
        w = torch.softmax(torch.einsum("thd,hd->th", ks, em["aq"][t]) * d ** -0.5, 0)
        o2 = torch.einsum("th,thd->hd", w, vs)
        return torch.cat([o1.flatten(), o2.flatten()]) @ m.out.double()

    for step in range(steps):
        copies, granted = kda.cache_reserve(table, lengths, refs, ones, page)
        kda.pages_copy([kp, vp], copies)
        assert bool((granted == 1).all())
        kda.cache_append(e["ak"][token], e["av"][token], kp, vp, table, lengths - 1)
        o2 = kda.paged_decode(e["aq"][token], kp, vp, table, lengths)
        o1 = kda.decode_step(e["q"][token], e["k"][token], e["v"][token], e["g"][token], e["beta"][token], state)
        logits = torch.cat([o1.reshape(n, -1), o2.reshape(n, -1)], 1) @ proj
        scores, parents, chosen, finished = kda.beam_select(logits.view(B, K, V), scores, finished=finished, eos=1)
        kda.beam_reorder(state, parents)
        table, lengths = kda.cache_fork(table, lengths, refs, (parents + base).flatten())
        token = chosen.flatten().long()
        for b in range(B):
            lg = torch.stack([plain_step(x) for x in plain[b]])
            want = select_plain(lg[None], torch.tensor([[x["s"] for x in plain[b]]]).double(), K,
                                torch.tensor([[x["done"] for x in plain[b]]]), 1)[0]
            assert parents[b].tolist() == [k for _, k, _ in want], (step, b)
            assert chosen[b].tolist() == [t for _, _, t in want], (step, b)
            for o, (c, k, t) in enumerate(want):
                assert float(scores[b, o]) == c or abs(float(scores[b, o]) - c) < 1e-3
            plain[b] = [dict(s=c, toks=plain[b][k]["toks"] + [t], S=plain[b][k]["S"].clone(),
                             done=plain[b][k]["done"] or t == 1) for c, k, t in want]
        assert finished.tolist() == [[x["done"] for x in row] for row in plain]
    assert refs.tolist() == counts(table.tolist(), n_pages)
    # compaction between two steps changes nothing but the places
    before = kda.paged_decode(e["aq"][token], kp, vp, table, lengths)
    table, refs, moves = kda.cache_compact(table, refs)
    kda.pages_copy([kp, vp], moves)
    used = int((refs > 0).sum())
    assert not refs[used:].any()
    kp[used:], vp[used:] = math.nan, math.nan  # the freed end of the pool is not read
    assert torch.equal(before, kda.paged_decode(e["aq"][token], kp, vp, table, lengths))
    kda.cache_free(table, lengths, refs, torch.arange(n, dtype=torch.int32, device=DEV))
    assert not refs.any() and not lengths.any()


def test_calls_are_captured_and_replayed():
    """A serving step in a graph, replayed on changed inputs with eager work between, equals the eager step."""
    B, K, V, page, hkv, d = 2, 4, 6000, 32, 2, 64
    n = B * K
    cache = Cache([2500 + 37 * i for i in range(n)], hkv, d, page, BF16, seed=41, extra_cols=4, spare=40)
    refs0 = i32(counts(cache.table.tolist(), cache.kp.shape[0]))
    q, k, v = (queries(n, h, d, BF16, seed=s) for h, s in ((8, 1), (hkv, 2), (hkv, 3)))
    logits = (torch.randn(B, K, V, generator=gen(7)) * 3).to(BF16).to(DEV)
    scores = torch.randn(B, K, generator=gen(8)).to(DEV)
    state = torch.randn(n, 2, 64, 64, generator=gen(9)).to(DEV)
    base = (torch.arange(B, dtype=torch.int32, device=DEV) * K)[:, None]
    ones = torch.ones(n, dtype=torch.int32, device=DEV)
    inputs = dict(table=cache.table.clone(), lengths=cache.len.clone(), refs=refs0.clone(), kp=cache.kp.clone(),
                  vp=cache.vp.clone(), state=state.clone(), q=q, k=k, v=v, logits=logits, scores=scores)

    def step(x):
        copies, granted = kda.cache_reserve(x["table"], x["lengths"], x["refs"], ones, page)
        kda.pages_copy([x["kp"], x["vp"]], copies)
        kda.cache_append(x["k"], x["v"], x["kp"], x["vp"], x["table"], x["lengths"] - 1)
        out, lse = kda.paged_decode(x["q"], x["kp"], x["vp"], x["table"], x["lengths"], lse=True)
        s, p, t, _ = kda.beam_select(x["logits"], x["scores"])
        kda.beam_reorder(x["state"], p)
        table, lengths = kda.cache_fork(x["table"], x["lengths"], x["refs"], (p + base).flatten())
        table2, refs2, moves = kda.cache_compact(table, x["refs"])
        return dict(copies=copies, granted=granted, out=out, lse=lse, s=s, p=p, t=t, table=table, lengths=lengths,
                    table2=table2, refs2=refs2, moves=moves)

    warm = {a: b.clone() for a, b in inputs.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.current_stream().wait_stream(side)
    held = {a: b.clone() for a, b in inputs.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held)
    for replay in range(4):
        fresh = {a: b.clone() for a, b in inputs.items()}
        g = gen(100 + replay)
        fresh["q"] = torch.randn(q.shape, generator=g).to(BF16).to(DEV)
        fresh["logits"] = (torch.randn(B, K, V, generator=g) * 3).to(BF16).to(DEV)
        for a, b in fresh.items():
            held[a].copy_(b)
        graph.replay()
        want = step(fresh)  # eager work between the replays
        torch.cuda.synchronize()
        for a in want:
            assert torch.equal(got[a], want[a]), (replay, a)
        for a in fresh:
            assert torch.equal(held[a].view(torch.uint8), fresh[a].view(torch.uint8)), (replay, a)


def test_calls_run_on_the_current_stream():
    """On a side stream behind a long fill, the calls see what the stream wrote before them."""
    cache = Cache([200, 300], 2, 64, 32, BF16, seed=51)
    q = queries(2, 4, 64, BF16)
    want = kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len)
    kp, vp = torch.zeros_like(cache.kp), torch.zeros_like(cache.vp)
    big = torch.zeros(1 << 28, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(4):
            big.add_(1.0)
        kp.copy_(cache.kp)
        vp.copy_(cache.vp)
        got = kda.paged_decode(q, kp, vp, cache.table, cache.len)
    side.synchronize()
    assert torch.equal(got, want)


def test_debug_check_of_tables(monkeypatch):
    cache = Cache([40, 40], 1, 64, 16, BF16, seed=61)
    q = queries(2, 2, 64, BF16)
    monkeypatch.setenv("KDA_DEBUG_CHECK", "1")
    kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len)
    with pytest.raises(kda.KdaError, match=r"lengths\[1\]"):
        kda.paged_decode(q, cache.kp, cache.vp, cache.table, i32([40, 49]))
    cache.table[0, 1] = cache.kp.shape[0]
    with pytest.raises(kda.KdaError, match=r"page_table\[0, 1\]"):
        kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len)


def test_the_marshalling_module_serves_the_usual_calls(monkeypatch):
    """The calls of a plain program go through the C marshalling; with it taken away the results are the
    same, and what it does not know (strides, other types) goes the Python way and is refused there."""
    from gated_delta_rule_75_amd import serving

    cache = Cache([200, 70], 2, 64, 16, BF16, seed=71, extra_cols=3, spare=30)
    refs = i32(counts(cache.table.tolist(), cache.kp.shape[0]))
    q, k, v = queries(2, 8, 64, BF16), queries(2, 2, 64, BF16, seed=2), queries(2, 2, 64, BF16, seed=3)
    logits, scores = torch.randn(2, 3, 5000, generator=gen(4)).to(DEV), torch.zeros(2, 3, device=DEV)
    done = i32([[0, 1, 0], [0, 0, 0]]).to(torch.uint8)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)

    def everything():
        t, n, r, kp, vp = (x.clone() for x in (cache.table, cache.len, refs, cache.kp, cache.vp))
        state = torch.arange(6 * 8, device=DEV, dtype=F32).view(6, 8)
        res = []
        t2, n2 = kda.cache_fork(t, n, r, i32([0, 1, 0, 1, -1]))
        res += [t2, n2, *kda.cache_reserve(t2, n2, r, i32([1, 2, 3, 40, 5]), 16)]
        res += [*kda.cache_reserve(t2, n2, r, i32([1, 0, 0, 0, 5]), 16, workspace=ws)]
        kda.pages_copy([kp, vp], res[2])
        kda.pages_copy(kp, res[4])
        kda.cache_append(k, v, kp, vp, t, n - 1)
        kda.cache_append(k, v, kp, vp, t2, n2 - 1, cu_seqlens=i32([0, 1, 1, 2, 2, 2]))
        kda.cache_free(t2, n2, r, i32([1, 1]))
        res += [*kda.cache_compact(t2, r), *kda.cache_compact(t2, r, workspace=ws)]
        res.append(kda.paged_decode(q, kp, vp, t, n))
        res += kda.paged_decode(q, kp, vp, t, n, scale=0.2, window=9, sinks=2, max_length=250, lse=True, workspace=ws,
                                out=torch.empty(2, 8, 64, device=DEV))
        res += kda.paged_decode(q, kp, vp, t, n, lse=torch.empty(2, 8, device=DEV))
        a, b, c, d = kda.beam_select(logits, scores)
        assert d is None
        res += [a, b, c, *kda.beam_select(logits, scores, n_out=5, finished=done, eos=7, workspace=ws)]
        kda.beam_reorder([state], b)
        return res + [r, kp, vp, state]

    first = everything()
    assert serving._M is not None
    for name in ("cache_append", "paged_decode", "cache_fork", "cache_free", "cache_reserve", "cache_compact",
                 "pages_copy", "beam_select", "beam_reorder"):
        assert hasattr(serving._M, name)
    calls = []
    real = serving._run
    monkeypatch.setattr(serving, "_run", lambda *a: calls.append(a) or real(*a))
    everything()
    assert not calls  # nothing went the Python way
    monkeypatch.setattr(serving, "_M", None)
    for x, y in zip(first, everything()):
        assert x.dtype == y.dtype and torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert calls
    monkeypatch.undo()
    with pytest.raises(kda.KdaError, match="sinks"):
        kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, sinks=3)
    with pytest.raises(ValueError, match="window"):
        kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len, window=2 ** 32)
    with pytest.raises(ValueError, match="page_size"):
        kda.cache_reserve(cache.table, cache.len, refs, i32([1, 1]), 2 ** 32)
    with pytest.raises(ValueError, match="lengths"):
        kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len[:1])
    with pytest.raises(ValueError, match="torch.int32"):
        kda.cache_append(k, v, cache.kp, cache.vp, cache.table, cache.len.long())
    with pytest.raises(ValueError, match="expected|GPU tensor"):
        kda.cache_fork(cache.table, cache.len.cpu(), refs, i32([0]))
    with pytest.raises(ValueError, match="contiguous"):
        kda.paged_decode(q.transpose(1, 2).contiguous().transpose(1, 2), cache.kp, cache.vp, cache.table, cache.len)
    with pytest.raises(ValueError, match="must be"):
        kda.beam_reorder(torch.zeros(5, 4, device=DEV), i32([[0, 1, 2], [0, 1, 2]]))
    with pytest.raises(ValueError, match="must be"):
        kda.pages_copy([cache.kp, cache.vp[:3]], i32([[0, 1]]))
    with pytest.raises(kda.KdaError, match="multiples of 16"):
        kda.pages_copy(torch.zeros(5, 3, device=DEV), i32([[0, 1]]))


def test_kernel_timing_names_the_kernels():
    cache = Cache([4000, 40], 1, 64, 16, BF16, seed=63)
    q = queries(2, 2, 64, BF16)
    with kda.kernel_timing() as t:
        kda.cache_append(q[:, :1], q[:, 1:], cache.kp, cache.vp, cache.table, i32([3, 4]))
        kda.paged_decode(q, cache.kp, cache.vp, cache.table, cache.len)
        kda.beam_select(torch.zeros(1, 2, 5000, device=DEV), torch.zeros(1, 2, device=DEV))
    names = [n for n, _ in t.records]
    assert names[:2] == ["kda_cache_append", "kda_paged_decode"] and names[-2:] == ["kda_beam_scan", "kda_beam_join"]
