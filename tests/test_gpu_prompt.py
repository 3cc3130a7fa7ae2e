"""Rotary positions on the GPU against plain 64-bit code.

Tolerances (u = 2^-24, the fp32 unit roundoff; a rounding to bf16 is off by 2^-8 of the value at most).  Rotation:
the angle is reduced in fp64 and rounded to fp32 as a multiple of pi of at most 1, which moves it by pi u at most; its
cosine and sine are within two units in the last place, 2 u; the amplitude's product rounds once: 6.2 u in
all.  A product and a fused product and sum round twice more, so a rotated channel is within 9 u amplitude (|x| + |y|)
of the exact one, and one rounding to the type.  Copied channels are compared bit for bit.
"""
import math

import pytest
import torch

import gated_delta_rule_75_amd as kda

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
STEP = {BF16: 2.0 ** -8, F32: U}
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(dtype).to(DEV)


def bits(x):
    return x.contiguous().view(torch.uint8)


# ------------------------------------------------------------------------------------------------
# rotation
# ------------------------------------------------------------------------------------------------
def turn64(x, positions, freqs, layout, amplitude=1.0, inverse=False):
    """The rotation of x [T,H,d] in fp64, and |x| + |y| of every channel's pair (0 for the copied ones)."""
    x, r = x.double().cpu(), 2 * freqs.numel()
    a = positions.cpu().double()[:, None, None] * freqs.cpu()
    c, s = torch.cos(a) * amplitude, torch.sin(a) * amplitude * (-1 if inverse else 1)
    lo, hi = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    y, size = x.clone(), torch.zeros_like(x)
    y[..., lo], y[..., hi] = x[..., lo] * c - x[..., hi] * s, x[..., lo] * s + x[..., hi] * c
    size[..., lo] = size[..., hi] = (x[..., lo].abs() + x[..., hi].abs()) * abs(amplitude)
    return y, size


def check_turn(got, x, positions, freqs, layout, amplitude=1.0, inverse=False):
    want, size = turn64(x, positions, freqs, layout, amplitude, inverse)
    assert got.dtype == x.dtype and got.shape == x.shape
    err = (got.double().cpu() - want).abs()
    tol = 9 * U * size + STEP[x.dtype] * (want.abs() + 9 * U * size)
    assert bool((err <= tol).all()), float((err - tol).max())
    r = 2 * freqs.numel()
    assert torch.equal(bits(got[..., r:]), bits(x[..., r:]))


SHAPES = [  # T, H_q, H_k, d, rotary_dim
    (1, 1, 1, 64, 64), (3, 8, 2, 128, 128), (5, 4, 4, 256, 256), (2, 1, 0, 128, 64), (7, 3, 1, 64, 2), (4, 5, 1, 64, 40),
    (3, 6, 2, 128, 90), (3, 2, 1, 256, 254), (9, 7, 3, 8, 8), (9, 2, 1, 8, 6), (5, 3, 2, 24, 24), (5, 3, 2, 80, 80),
    (5, 3, 2, 80, 48), (2, 3, 2, 512, 512), (2, 300, 40, 64, 32), (5001, 2, 1, 64, 64), (33001, 1, 0, 16, 16),
    (6203, 2, 1, 24, 10), (40000, 3, 1, 64, 34)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hk,d,r", SHAPES)
def test_rotary_matches_fp64(dtype, layout, T, hq, hk, d, r):
    print(f"rotary {dtype} {layout} T={T} hq={hq} hk={hk} d={d} r={r}", flush=True)
    q = normal((T, hq, d), dtype, 1)
    k = normal((T, hk, d), dtype, 2) if hk else None
    positions = (torch.arange(T, dtype=torch.int32) * 7 + 1000 * (T % 5)).to(DEV)
    freqs = kda.rotary_frequencies(r)
    keep = q.clone()
    q_out, k_out = kda.rotary(q, k, positions, freqs, layout=layout, amplitude=1.25)
    torch.cuda.synchronize()
    assert torch.equal(bits(q), bits(keep))
    check_turn(q_out, q, positions, freqs, layout, 1.25)
    if hk:
        check_turn(k_out, k, positions, freqs, layout, 1.25)
    else:
        assert k_out is None


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout,r", [("half", 64), ("half", 36), ("interleaved", 64), ("interleaved", 38)])
def test_rotary_far_and_negative_positions(dtype, layout, r):
    """Positions to the ends of 32 bits: the angles are those of fp64."""
    positions = i32([0, 1, -1, 131071, 10 ** 6, 2 ** 31 - 1, -2 ** 31, 123456789])
    q = normal((8, 4, 64), dtype, 3)
    freqs = kda.rotary_frequencies(r, base=500000.0)
    out, _ = kda.rotary(q, None, positions, freqs, layout=layout)
    check_turn(out, q, positions, freqs, layout)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout,r", [("half", 128), ("half", 100), ("interleaved", 128), ("interleaved", 100)])
def test_rotary_in_place_on_slices_of_one_projection(dtype, layout, r):
    """q and k as slices of a fused projection, turned in place: the values between them stay as they are."""
    T, hq, hk, d = 37, 6, 2, 128
    qkv = normal((T, hq + 2 * hk, d), dtype, 4)
    before = qkv.clone()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    positions, freqs = i32(list(range(50, 50 + T))), kda.rotary_frequencies(r)
    q_out, k_out = kda.rotary(q, k, positions, freqs, layout=layout, q_out=q, k_out=k)
    assert q_out is q and k_out is k
    check_turn(q, before[:, :hq], positions, freqs, layout)
    check_turn(k, before[:, hq:hq + hk], positions, freqs, layout)
    assert torch.equal(bits(qkv[:, hq + hk:]), bits(before[:, hq + hk:]))
    # and back: the same as two separate calls into buffers of their own
    wide = torch.zeros(T, 2 * hq, d, dtype=dtype, device=DEV)
    kda.rotary(q, None, positions, freqs, layout=layout, inverse=True, q_out=wide[:, hq:])
    check_turn(wide[:, hq:], q, positions, freqs, layout, inverse=True)
    assert not wide[:, :hq].any()


def test_rotary_not_finite_values_stay_in_their_pairs():
    for layout, r in (("half", 32), ("half", 18), ("interleaved", 18)):
        q = normal((2, 2, 64), F32, 5)
        q[1, 0, 3], q[1, 0, 40] = math.nan, math.inf
        positions, freqs = i32([3, 9]), kda.rotary_frequencies(r)
        out, _ = kda.rotary(q, None, positions, freqs, layout=layout)
        hit = {3, 3 + r // 2} if layout == "half" else {2, 3}
        assert set(torch.nonzero(out[1, 0].isnan()).flatten().tolist()) == hit
        assert math.isinf(float(out[1, 0, 40])) and not out[0].isnan().any() and not out[1, 1].isnan().any()


@pytest.mark.parametrize("layout,r", [("half", 64), ("half", 20), ("interleaved", 48)])
def test_rotary_inverse_is_the_gradient(layout, r):
    """inverse=True on the outputs' gradients: the gradient of the fp64 formula, and of central differences of the
    call itself (which is linear: a difference of any width is exact up to rounding)."""
    T, h, d, amp = 6, 3, 64, 1.3
    q, g = normal((T, h, d), F32, 6), normal((T, h, d), F32, 7)
    positions, freqs = i32([5, 0, 77777, 3, 2, 100]), kda.rotary_frequencies(r)
    grad, _ = kda.rotary(g, None, positions, freqs, layout=layout, amplitude=amp, inverse=True)
    x = q.cpu().double().requires_grad_()
    rr = 2 * freqs.numel()
    a = positions.cpu().double()[:, None, None] * freqs.cpu()
    c, s = torch.cos(a) * amp, torch.sin(a) * amp
    lo, hi = (slice(0, rr // 2), slice(rr // 2, rr)) if layout == "half" else (slice(0, rr, 2), slice(1, rr, 2))
    loss = ((x[..., lo] * c - x[..., hi] * s) * g[..., lo].cpu().double()).sum() + (
        (x[..., lo] * s + x[..., hi] * c) * g[..., hi].cpu().double()).sum() + (x[..., rr:] * g[..., rr:].cpu().double()).sum()
    loss.backward()
    _, size = turn64(g, positions, freqs, layout, amp, True)
    assert bool(((grad.cpu().double() - x.grad).abs() <= 10 * U * size).all())
    v = normal((T, h, d), F32, 8)
    up, down = (kda.rotary(q + e * v, None, positions, freqs, layout=layout, amplitude=amp)[0].double() for e in (1, -1))
    # q +- v round by u; each channel of the two results by 10 u (|x| + |y|) amplitude
    slope = ((up - down) / 2 * g.double()).sum()
    _, s1 = turn64(q.abs() + v.abs(), positions, freqs, layout, amp)
    s1 = torch.where(s1 > 0, s1, (q.abs() + v.abs()).cpu().double())
    assert abs(float(slope - (v.double() * grad.double()).sum())) <= 24 * U * float((s1 * g.cpu().double().abs()).sum())


def test_rotary_without_tokens():
    q = torch.zeros(0, 4, 64, device=DEV)
    out, k = kda.rotary(q, q, i32([]), kda.rotary_frequencies(64))
    assert out.shape == q.shape and k.shape == q.shape


# ------------------------------------------------------------------------------------------------
# rotation into pages
# ------------------------------------------------------------------------------------------------
def pages(n_pages, hkv, page, d, dtype, seed=11):
    return normal((n_pages, hkv, page, d), dtype, seed), normal((n_pages, hkv, page, d), dtype, seed + 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout,hq,hkv,d,r,page,new,start", [
    ("half", 8, 2, 128, 128, 16, [1, 0, 17, 40], [0, 5, 31, 200]),
    ("half", 4, 4, 64, 64, 48, [3, 3, 3], [47, 48, 0]),
    ("half", 6, 1, 256, 100, 32, [33, 1], [7, 0]),
    ("interleaved", 8, 8, 64, 64, 64, [100], [3]),
    ("interleaved", 4, 2, 128, 90, 16, [0, 0, 5, 0, 1], [0, 9, 11, 2, 15]),
    ("half", 2, 1, 64, 64, 16, [1500, 2700, 900], [0, 3, 77]),
])
def test_rotary_append_is_rotary_and_append(dtype, layout, hq, hkv, d, r, page, new, start):
    """Bit for bit what the two calls give one after the other; other slots of the pages stay as they are."""
    N, T = len(new), sum(new)
    print(f"place {dtype} {layout} T={T} hq={hq} hkv={hkv} d={d} r={r}", flush=True)
    width = max(-(-(a + b) // page) for a, b in zip(new, start)) + 1
    n_pages = N * width + 2
    table = torch.randperm(n_pages, generator=gen(3))[:N * width].view(N, width).to(torch.int32).to(DEV)
    kp, vp = pages(n_pages, hkv, page, d, dtype)
    q, k, v = (normal((T, h, d), dtype, s) for h, s in ((hq, 21), (hkv, 22), (hkv, 23)))
    cu = i32([sum(new[:i]) for i in range(N + 1)])
    at = torch.cat([torch.arange(s, s + m) for s, m in zip(start, new)]).to(torch.int32).to(DEV)
    freqs = kda.rotary_frequencies(r)
    want_q, want_k = kda.rotary(q, k, at, freqs, layout=layout, amplitude=0.9)
    wkp, wvp = kp.clone(), vp.clone()
    kda.cache_append(want_k, v, wkp, wvp, table, i32(start), cu_seqlens=cu)
    got = kda.rotary_append(q, k, v, kp, vp, table, i32(start), freqs, cu_seqlens=cu, layout=layout, amplitude=0.9)
    assert torch.equal(bits(got), bits(want_q)) and torch.equal(bits(kp), bits(wkp)) and torch.equal(bits(vp), bits(wvp))


@pytest.mark.parametrize("layout,r", [("half", 64), ("half", 30), ("interleaved", 64)])
def test_rotary_append_one_token_per_sequence_in_place(layout, r):
    n, hq, hkv, d = 200, 4, 2, 64
    qkv = normal((n, hq + 2 * hkv, d), BF16, 31)
    before = qkv.clone()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    start = torch.randint(0, 64, (n,), generator=gen(5), dtype=torch.int32).to(DEV)
    table = torch.randperm(4 * n, generator=gen(6)).view(n, 4).to(torch.int32).to(DEV)
    pool = torch.zeros(4 * n, 2, hkv, 16, d, dtype=BF16, device=DEV)  # keys and values side by side
    freqs = kda.rotary_frequencies(r)
    out = kda.rotary_append(q, k, v, pool[:, 0], pool[:, 1], table, start, freqs, layout=layout, q_out=q)
    assert out is q
    check_turn(q, before[:, :hq], start, freqs, layout)
    assert torch.equal(bits(qkv[:, hq:]), bits(before[:, hq:]))
    ids = table.long().gather(1, (start.long() // 16)[:, None])[:, 0]
    check_turn(pool[ids, 0, :, start.long() % 16], before[:, hq:hq + hkv], start, freqs, layout)
    assert torch.equal(pool[ids, 1, :, start.long() % 16], before[:, hq + hkv:])
    assert int((pool != 0).any(4).sum()) == 2 * n * hkv


@pytest.mark.parametrize("layout,r", [("half", 64), ("half", 30), ("interleaved", 64)])
def test_rotary_append_drops_positions_without_a_page(layout, r):
    """Positions before 0, behind the table or at entries that name no page write nothing; their queries are
    turned.  Tokens that belong to no sequence are left as they were."""
    T, d = 12, 64
    q, k, v = (normal((T, h, d), F32, s) for h, s in ((2, 1), (1, 2), (1, 3)))
    kp, vp = torch.zeros(4, 1, 16, d, device=DEV), torch.zeros(4, 1, 16, d, device=DEV)
    table = i32([[0, -1], [1, 4], [2, -2147483648], [3, 3]])
    start, cu = i32([-2, 15, 31, 2147483646]), i32([1, 4, 6, 8, 10])
    freqs = kda.rotary_frequencies(r)
    q_out = torch.full_like(q, 7.0)
    kda.rotary_append(q, k, v, kp, vp, table, start, freqs, cu_seqlens=cu, layout=layout, q_out=q_out)
    at = torch.tensor([-2, -1, 0, 15, 16, 31, 32, 2147483646, 2147483647])
    check_turn(q_out[1:10], q[1:10], at, freqs, layout)
    assert bool((q_out[0] == 7).all()) and bool((q_out[10:] == 7).all())
    wrote = [(p, s) for p in range(4) for s in range(16) if bool(vp[p, 0, s].any())]
    assert wrote == [(0, 0), (1, 15)]
    assert torch.equal(vp[0, 0, 0], v[3, 0]) and torch.equal(vp[1, 0, 15], v[4, 0])
    check_turn(kp[0, 0, 0][None, None], k[3:4], torch.tensor([0]), freqs, layout)


def test_rotary_append_many_sequences():
    """More sequences than a wave's lanes, empty ones among them."""
    new = [(7 * i) % 3 for i in range(5000)]
    T, d = sum(new), 64
    q, k, v = (normal((T, 1, d), BF16, s) for s in (1, 2, 3))
    kp, vp = torch.zeros(5000, 1, 16, d, dtype=BF16, device=DEV), torch.zeros(5000, 1, 16, d, dtype=BF16, device=DEV)
    table = torch.arange(5000, dtype=torch.int32, device=DEV)[:, None]
    start = (torch.arange(5000) % 14).to(torch.int32)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(torch.tensor(new), 0)]).to(torch.int32).to(DEV)
    at = torch.cat([torch.arange(int(s), int(s) + m) for s, m in zip(start, new)])
    freqs = kda.rotary_frequencies(64)
    out = kda.rotary_append(q, k, v, kp, vp, table, start.to(DEV), freqs, cu_seqlens=cu)
    check_turn(out, q, at, freqs, "half")
    seq = torch.repeat_interleave(torch.arange(5000), torch.tensor(new)).to(DEV)
    assert torch.equal(vp[seq, :, at.to(DEV)], v) and int(vp.any(3).sum()) == T


# ------------------------------------------------------------------------------------------------
# frequencies
# ------------------------------------------------------------------------------------------------
def test_rotary_frequencies_on_the_device():
    f = kda.rotary_frequencies(128, base=10000.0)
    assert f.dtype == torch.float64 and f.is_cuda and tuple(f.shape) == (64,)
