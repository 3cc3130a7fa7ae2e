"""Token log-probabilities, entropy, best alternatives and their gradient on the GPU against plain 64-bit code.

Tolerances (u = 2^-24, the fp32 unit roundoff; a rounding to bf16 is off by 2^-8 of the value at most).  With p the
row's probabilities, S = sum p (|x - max| + 1) and S2 = sum p (|x - max| + 1)^2 (a thread's reference is at most 1 below
its maximum):
 * A weight exp(x - m) comes from an exponent z of one rounding and a constant that is off by 0.3 u: it is off by the
   factor 1 +- (2 |z| + 3) u.  Its sum has at most V / 1024 + 32 additions in a chain, and is moved to another
   reference a few times, each by a factor of 1/e at least, 8 u in all.  So |lse - exact| <= (2 S + V / 1024 + 64) u, and
   one rounding of the result; a log-probability is the difference in fp64, rounded once.
 * s = sum exp(x - m) (x - m) adds S2 and the same chain on S: |H - exact| <= (4 S2 + (V / 1024 + 70) (1 + S)) u, and one
   rounding.
 * Gradient: p from the given log-sum is off by (3 |log p| + 4) u, its factor by four roundings of its terms; then the sum
   with the token's share and one rounding to the type.  Weights below 2^-126 may be 0.
Tokens are compared exactly.
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


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rows(R, V, dtype, seed=0, scale=3.0, offset=0.0):
    return (torch.randn(R, V, generator=gen(seed)) * scale + offset).to(dtype).to(DEV)


def some_tokens(R, V, seed=0):
    t = torch.randint(0, V, (R,), generator=gen(seed + 77), dtype=torch.int32)
    t[::7] = V - 1
    if R > 3:
        t[1], t[2] = -100, V
    return t.to(DEV)


def plain64(x, tokens, top):
    """logprobs, lse, H, best, which, and the bounds' S and S2 (rows with a finite log-sum)."""
    x = x.double().cpu()
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
    V = x.shape[1]
    most = x.amax(1, keepdim=True)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    lp = torch.where(p > 0, x - lse[:, None], torch.zeros_like(x))
    h = -(p * lp).sum(1)
    far = torch.where(p > 0, most - x, torch.zeros_like(x)) + 1
    t = tokens.long().cpu()
    ok = (t >= 0) & (t < V)
    given = torch.where(ok, x.gather(1, t.clamp(0, V - 1)[:, None])[:, 0] - lse, torch.zeros_like(lse))
    y, at = torch.sort(x, dim=1, descending=True, stable=True)
    return given, lse, h, y[:, :top] - lse[:, None], at[:, :top], (p * far).sum(1), (p * far * far).sum(1)


def check(x, tokens, top, entropy=True, **kw):
    V = x.shape[1]
    keep = x.clone()
    got = kda.token_logprobs(x, tokens, top=top, entropy=entropy, **kw)
    torch.cuda.synchronize()
    assert torch.equal(x.contiguous().view(torch.uint8), keep.contiguous().view(torch.uint8))
    lp, lse, h, best, which, s, s2 = plain64(x, tokens, top)
    tol = U * (2 * s + V / 1024 + 64)
    worst = {}

    def near(name, a, b, t):
        a = a.double().cpu()
        assert a.shape == b.shape and bool(a.isfinite().all()), name
        e = (a - b).abs() / (t + U * b.abs())
        worst[name] = float(e.max()) if e.numel() else 0.0
        assert worst[name] <= 1, (name, worst[name], int(e.flatten().argmax()))

    near("logprobs", got[0], lp, tol)
    near("lse", got[1], lse, tol)
    if entropy:
        near("entropy", got[2], h, U * (4 * s2 + (V / 1024 + 70) * (1 + s)))
    else:
        assert got[2] is None
    if top:
        assert got[4].dtype == torch.int32 and torch.equal(got[4].long().cpu(), which)
        near("top", got[3], best, tol[:, None])
    else:
        assert got[3] is None and got[4] is None
    print("  of the bounds:", {k: round(v, 3) for k, v in worst.items()}, flush=True)
    return got


SHAPES = [(1, 1), (3, 7), (5, 64), (5, 1000), (2, 8185), (2, 8193), (4, 32003), (1, 131072), (70, 5000), (1030, 601),
          (260, 20000), (1100, 12289), (0, 50), (2, 300000)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,V", SHAPES)
@pytest.mark.parametrize("top", [0, 5])
def test_logprobs_match_fp64(dtype, R, V, top):
    print(f"logprobs {dtype} R={R} V={V} top={top}", flush=True)
    check(rows(R, V, dtype, seed=V), some_tokens(R, V), min(top, V), entropy=top > 0 or V % 2 == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,V,top", [(3, 64, 64), (3, 65, 64), (2, 9000, 64), (9, 40000, 33), (1200, 700, 17),
                                     (1050, 16400, 32), (1, 131072, 1), (30, 4096, 2)])
def test_best_alternatives(dtype, R, V, top):
    print(f"top {dtype} R={R} V={V} top={top}", flush=True)
    check(rows(R, V, dtype, seed=top, scale=1.0), some_tokens(R, V), top)


@pytest.mark.parametrize("R", [2, 1100])
@pytest.mark.parametrize("V", [3000, 20011])
@pytest.mark.parametrize("kind", ["flat", "ascending", "descending", "masked half", "masked end", "few", "steps"])
def test_best_alternatives_of_rows_that_fill_the_lists(kind, V, R):
    """Equal logits and finite masks before better ones: ties go to the lower token."""
    print(f"{kind} V={V} R={R}", flush=True)
    x = torch.randn(R, V, generator=gen(5))
    if kind == "flat":
        x[:] = 1.5
    elif kind == "ascending":
        x = (torch.arange(V, dtype=F32) / V * 4).expand(R, V).contiguous()
    elif kind == "descending":
        x = (-torch.arange(V, dtype=F32) / V * 4).expand(R, V).contiguous()
    elif kind == "masked half":
        x[:, :V // 2] = -1e4
    elif kind == "masked end":
        x[:, V // 2:] = torch.finfo(F32).min
    elif kind == "few":
        x[:] = -1e4
        x[:, 5::97] = torch.randn(R, len(range(5, V, 97)), generator=gen(6))
    else:
        x = (torch.arange(V) // 300 % 7).to(F32).expand(R, V).contiguous()
    for top in (1, 8, 64):
        check(x.to(DEV), some_tokens(R, V), top)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_any_stride_and_alignment(dtype):
    wide = rows(9, 9000, dtype, seed=3)
    for V, at in ((5001, 1), (5000, 3), (8999, 1), (17, 2)):
        x = wide[:, at:at + V]
        check(x, some_tokens(9, V), min(4, V))
        check(wide[:, :V], some_tokens(9, V), 3)


def test_logits_far_from_zero():
    """The weights depend on differences alone: rows around +-1e4, +-1e6 and 3e7 give what they give in fp64, and so do
    the lowest and highest finite values next to them."""
    for offset in (1e4, -1e4, 1e6, -1e6, 3e7, -3e7):
        check(rows(3, 5000, F32, seed=4, offset=offset), some_tokens(3, 5000), 5)
        check(rows(3, 50000, F32, seed=4, offset=offset), some_tokens(3, 50000), 5)
    x = rows(2, 3000, F32, seed=4)
    x[0, 100:] = torch.finfo(F32).min
    x[1, 7] = torch.finfo(F32).max
    check(x, some_tokens(2, 3000), 5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [700, 20001])
def test_masked_and_missing_logits(dtype, V):
    """-inf and NaN have probability 0; fewer finite logits than places; places at -inf go to the lowest tokens."""
    x = rows(6, V, dtype, seed=8)
    x[0, ::2] = -math.inf
    x[1, ::3] = math.nan
    x[2, 3:] = -math.inf
    x[2, 1] = math.nan
    x[3, :] = -math.inf
    x[3, V - 1] = 2.0
    x[4, :V - 40] = -math.inf
    tokens = torch.tensor([0, 0, 2, V - 1, V - 1, 5], dtype=torch.int32, device=DEV)
    lp, lse, h, best, which = kda.token_logprobs(x, tokens, top=6, entropy=True)
    assert math.isinf(float(lp[0])) and math.isinf(float(lp[1])) and float(lp[0]) < 0 and float(lp[1]) < 0
    wlp, wlse, wh, wbest, wwhich, s, s2 = plain64(x, tokens, 6)
    assert torch.equal(which.long().cpu(), wwhich)
    assert torch.equal(best.cpu().isinf(), wbest.isinf()) and not best.isnan().any()
    fine = wbest.isfinite()
    tol = U * (2 * s + V / 1024 + 64)
    assert bool(((best.cpu().double() - wbest).abs()[fine] <= (tol[:, None] + U * wbest.abs())[fine]).all())
    assert bool(((lse.cpu().double() - wlse).abs() <= tol + U * wlse.abs()).all())
    assert bool(((h.cpu().double() - wh).abs() <= U * (4 * s2 + (V / 1024 + 71) * (1 + s))).all())
    assert float(h[3]) == 0.0 and float(lp[3]) == 0.0
    assert bool(((lp.cpu().double() - wlp).abs()[2:] <= (tol + U * wlp.abs())[2:]).all())


@pytest.mark.parametrize("V", [700, 20001])
def test_rows_without_a_finite_log_sum(V):
    x = rows(4, V, F32, seed=9)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 5] = math.inf
    x[3, 5], x[3, 9], x[3, 2] = math.inf, math.inf, math.nan
    tokens = torch.tensor([3, 3, 5, 4], dtype=torch.int32, device=DEV)
    lp, lse, h, best, which = kda.token_logprobs(x, tokens, top=3, entropy=True)
    assert lse.tolist() == [-math.inf, -math.inf, math.inf, math.inf]
    assert lp.tolist() == [-math.inf] * 4 and h.tolist() == [0.0] * 4 and bool((best == -math.inf).all())
    assert which[0].tolist() == [0, 1, 2] and which[1].tolist() == [0, 1, 2]
    assert int(which[2, 0]) == 5 and which[3, :2].tolist() == [5, 9]
    d = kda.token_logprobs_grad(x, tokens, lse, torch.ones(4, device=DEV), entropy=h, d_entropy=torch.ones(4, device=DEV))
    assert not d.any()


def test_without_tokens_and_with_a_workspace():
    x = rows(5, 40000, BF16, seed=10)
    lp, lse, h, best, which = kda.token_logprobs(x, None, top=3)
    assert lp is None and h is None
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    again = check(x, some_tokens(5, 40000), 3, entropy=False, workspace=ws)
    assert torch.equal(lse, again[1]) and torch.equal(best, again[3]) and torch.equal(which, again[4])
    check(x, some_tokens(5, 40000), 3, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))  # too small: another


# ------------------------------------------------------------------------------------------------
# gradient
# ------------------------------------------------------------------------------------------------
def grad_inputs(R, V, dtype, seed, scale=3.0):
    x = rows(R, V, dtype, seed=seed, scale=scale)
    tokens = some_tokens(R, V, seed)
    _, lse, h, _, _ = kda.token_logprobs(x, tokens, entropy=True)
    return x, tokens, lse, h, *(torch.randn(R, generator=gen(seed + i)).to(DEV) for i in (1, 2, 3))


def check_grad(got, x, tokens, lse, h=None, d=None, dl=None, dh=None):
    def wide(t):
        return torch.zeros(x.shape[0], 1).double() if t is None else t.double().cpu()[:, None]

    v = x.double().cpu()
    d, dl, dh, hh = wide(d), wide(dl), wide(dh), wide(h)
    t = torch.full((x.shape[0],), -1) if tokens is None else tokens.long().cpu()
    pick = torch.arange(x.shape[1])[None] == t[:, None]
    d = torch.where(pick.any(1, keepdim=True), d, torch.zeros_like(d))
    lp = v - wide(lse)
    p = torch.exp(lp)
    lp = torch.where(p > 0, lp, torch.zeros_like(lp))
    want = p * (dl - d - dh * (lp + hh)) + d * pick
    size = d.abs() + dl.abs() + dh.abs() * (lp.abs() + hh.abs())
    tol = U * (3 * lp.abs() + 8) * p * size + 2 * U * (want.abs() + d.abs() * pick) + 1e-36 * (1 + size)
    tol = tol + STEP[x.dtype] * (want.abs() + tol)
    err = (got.double().cpu() - want).abs()
    assert got.dtype == x.dtype and got.shape == x.shape
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 7), (5, 1000), (2, 8193), (4, 32003), (70, 5000), (1030, 601), (0, 9)])
def test_gradient_matches_fp64(dtype, R, V):
    print(f"grad {dtype} R={R} V={V}", flush=True)
    x, tokens, lse, h, d, dl, dh = grad_inputs(R, V, dtype, V)
    check_grad(kda.token_logprobs_grad(x, tokens, lse, d), x, tokens, lse, None, d)
    check_grad(kda.token_logprobs_grad(x, tokens, lse, d, entropy=h, d_entropy=dh), x, tokens, lse, h, d, None, dh)
    check_grad(kda.token_logprobs_grad(x, tokens, lse, d, d_lse=dl, entropy=h, d_entropy=dh), x, tokens, lse, h, d, dl, dh)
    check_grad(kda.token_logprobs_grad(x, None, lse, d_lse=dl), x, None, lse, None, None, dl)
    check_grad(kda.token_logprobs_grad(x, None, lse, entropy=h, d_entropy=dh), x, None, lse, h, None, None, dh)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_in_place_and_strided(dtype):
    x, tokens, lse, h, d, dl, dh = grad_inputs(6, 5003, dtype, 3)
    want = kda.token_logprobs_grad(x, tokens, lse, d, entropy=h, d_entropy=dh)
    same = x.clone()
    assert kda.token_logprobs_grad(same, tokens, lse, d, entropy=h, d_entropy=dh, out=same) is same
    assert torch.equal(same, want)
    for at_x, at_y in ((1, 1), (0, 3), (3, 0)):
        a = torch.full((6, 5100), 7.0, dtype=dtype, device=DEV)
        b = torch.full((6, 5040), 7.0, dtype=dtype, device=DEV)
        a[:, at_x:at_x + 5003] = x
        kda.token_logprobs_grad(a[:, at_x:at_x + 5003], tokens, lse, d, entropy=h, d_entropy=dh,
                                out=b[:, at_y:at_y + 5003])
        check_grad(b[:, at_y:at_y + 5003], x, tokens, lse, h, d, None, dh)
        b[:, at_y:at_y + 5003] = 7.0
        assert bool((b == 7).all())


def test_gradient_of_masked_logits_is_zero():
    x, tokens, lse, h, d, dl, dh = grad_inputs(4, 5000, F32, 12)
    x[:, ::2] = -math.inf
    x[2, 1::4] = math.nan
    _, lse, h, _, _ = kda.token_logprobs(x, None, entropy=True)
    g = kda.token_logprobs_grad(x, None, lse, d_lse=dl, entropy=h, d_entropy=dh)
    assert bool(g.isfinite().all()) and not g[:, ::2].any() and not g[2, 1::4].any() and bool(g[0, 1::2].any())


def test_gradient_of_the_formula_and_of_differences():
    """The call on the results of token_logprobs against autograd through the fp64 formulas, and against central
    differences of the calls themselves."""
    R, V = 4, 300
    x, tokens, lse, h, d, dl, dh = grad_inputs(R, V, F32, 21, scale=1.0)
    tokens = torch.tensor([5, -1, 299, 0], dtype=torch.int32, device=DEV)
    g = kda.token_logprobs_grad(x, tokens, lse, d, d_lse=dl, entropy=h, d_entropy=dh)
    y = x.double().cpu().requires_grad_()
    lp = torch.log_softmax(y, 1)
    ok = (tokens >= 0).cpu()
    loss = (d.cpu().double() * lp.gather(1, tokens.long().cpu().clamp(min=0)[:, None])[:, 0] * ok).sum()
    loss = loss + (dl.cpu().double() * torch.logsumexp(y, 1)).sum() - (dh.cpu().double()[:, None] * lp.exp() * lp).sum()
    loss.backward()
    # the given lse and H are rounded and off by about 100 u themselves
    assert float((g.double().cpu() - y.grad).abs().max()) <= 500 * U * float((d.abs() + dl.abs() + 8 * dh.abs()).max())
    v = torch.randn(R, V, generator=gen(22)).to(DEV)
    step = 2.0 ** -7

    def value(z):
        a, b, c, _, _ = kda.token_logprobs(z, tokens, entropy=True)
        return float((a.double() * d + b.double() * dl + c.double() * dh).sum())

    slope = (value(x + step * v) - value(x - step * v)) / (2 * step)
    exact = float((g.double() * v.double()).sum())
    # each value is off by about 100 u of its terms (below 4 * 3 * 8), and a third derivative below 20 |v|^3
    assert abs(slope - exact) <= 100 * U * 96 / step + 20 * step * step * float(v.abs().max()) ** 3


@pytest.mark.parametrize("dtype,R", [(BF16, 4200), (F32, 2100)])
def test_logits_of_more_than_the_caches_hold(dtype, R):
    """Such calls pass the caches by: rows give what they give alone (where they are split: within the sums' bounds)."""
    V = 32768
    x = torch.zeros(R, V, dtype=dtype, device=DEV)
    x[-3:] = rows(3, V, dtype, seed=5)
    x[7] = x[-1]
    tokens = torch.arange(R, dtype=torch.int32, device=DEV) * 3
    d = torch.ones(R, device=DEV)
    for top, entropy in ((0, False), (0, True), (3, False), (3, True)):
        print(f"large {dtype} top={top} entropy={entropy}", flush=True)
        got = kda.token_logprobs(x, tokens, top=top, entropy=entropy)
        lp, lse, h, best, which, s, s2 = plain64(x[-3:], tokens[-3:], top)
        tol = U * (4 * s2 + (V / 1024 + 70) * (1 + s) + 8 * lse.abs())
        for a, b in zip(got[:3], (lp, lse, h)):
            if a is not None:
                assert bool(((a[-3:].cpu().double() - b).abs() <= tol + U * b.abs()).all())
        assert float(got[1][7]) == float(got[1][-1]) and abs(float(got[1][0]) - math.log(V)) <= 1e-5
        if top:
            assert torch.equal(got[4][-3:].cpu().long(), which) and got[4][0].tolist() == [0, 1, 2]
        lse, h = got[1], got[2]
        grad = kda.token_logprobs_grad(x, tokens, lse, d, entropy=h, d_entropy=d if entropy else None)
        alone = kda.token_logprobs_grad(x[-3:].clone(), tokens[-3:].clone(), lse[-3:].clone(), d[-3:].clone(),
                                        entropy=None if h is None else h[-3:].clone(), d_entropy=d[-3:].clone() if entropy else None)
        assert torch.equal(grad[-3:].contiguous().view(torch.uint8), alone.view(torch.uint8))


@pytest.mark.parametrize("R,V,top", [(5, 32000, 5), (5, 32000, 20), (3, 50000, 64), (70, 5000, 20), (1030, 6000, 5),
                                     (300, 20011, 20)])
@pytest.mark.parametrize("offset,spread", [(100.0, 0.1), (-100.0, 0.1), (1e4, 3.0), (1.0, 2.0 ** -9), (3e38, 1e31)])
def test_best_alternatives_of_rows_far_from_zero(R, V, top, offset, spread):
    """Logits that differ in their lower 16 bits alone, so that the bound's upper bits let much of a row pass."""
    print(f"R={R} V={V} top={top} {offset} +- {spread}", flush=True)
    x = (torch.randn(R, V, generator=gen(V + top)) * spread + offset).to(DEV)
    lp, lse, h, best, which = kda.token_logprobs(x, None, top=top)
    y, at = torch.sort(x.cpu(), dim=1, descending=True, stable=True)
    assert torch.equal(which.long().cpu(), at[:, :top])
    if offset < 1e30:
        check(x, some_tokens(R, V), top)


@pytest.mark.parametrize("R,V,top", [(5, 32000, 5), (1030, 6000, 20), (2048, 50257, 20)])
def test_rows_far_from_zero_are_not_read_once_for_each_place(R, V, top):
    """An offset costs a second look at a row, not one for each place: with those the scan takes 14 to 19 times as long
    as without an offset, with one about twice."""
    z = torch.randn(R, V, generator=gen(7)).to(DEV)

    def least_time(x):
        best = math.inf
        for _ in range(6):
            with kda.kernel_timing() as t:
                kda.token_logprobs(x, None, top=top)
            best = min(best, sum(ms for name, ms in t.records if name == "kda_logprob_scan"))
        return best

    plain, far = least_time(z * 3.0), least_time(z * 0.1 + 100.0)
    print(f"  scan {plain * 1e3:.1f} us, far from zero {far * 1e3:.1f} us", flush=True)
    assert far < 6 * plain
