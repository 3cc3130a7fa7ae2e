"""How exactly a chunk's attention with few rows carries its softmax weights in bf16: as two bf16 values each, which is
the weight but for 2^-16 of it (a bf16 rounding is off by 2^-8 at most, and so is that of what it left).

The scores here are exact: a query is 1 in one channel, so that its score with a key is that key's value there, and the
scale is 1.  A weight exp(s - m) then comes from an exponent of four roundings (u = 2^-24 of it each, |s - m| log2 e
<= 16) and the hardware's 2^x: off by the factor 1 +- w, w = (4 * 16 + 9) u.  Sums of n terms add (n + 64) u.  So
    |out - exact| <= sum p |v| (2 w + 2 (n + 64) u + 2^-16) + 2^-8 |out|    (the output's own rounding).
The values cancel in one output of each channel, so that the last term, which would hide a weight's rounding to one
bf16, is almost 0 there.  That mistake, made in the oracle, is beyond the bound."""
import math

import pytest
import torch

import gated_delta_rule_75_amd as kda
from test_gpu_serving import Cache, gen, i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U = 2.0 ** -24
BF16 = torch.bfloat16
DEV = "cuda"


def oracle(k, v, c, first, rounded=False):
    """Query i of head h at position first + i sees k[.., c[i, h]] as scores: out [m, H, d] and sum p |v|, fp64; with
    `rounded` the weights are one bf16 each in their product with the values."""
    m, H = c.shape
    seen = torch.arange(k.shape[0])[None] <= first + torch.arange(m)[:, None]
    s = k.double()[:, c].permute(1, 2, 0)  # [m, H, t]
    s = torch.where(seen[:, None], s, torch.full_like(s, -math.inf))
    w = torch.exp(s - s.amax(2, keepdim=True))
    total = w.sum(2, keepdim=True)
    p = (w.to(BF16).double() if rounded else w) / total
    return p @ v.double(), p @ v.double().abs()


def cancelling(length, d, c, first, seed):
    """Keys [length, d] (exact scores up to about 6) and values [length, d], bf16, with sum p v about 0 in channel j for
    the (query, head) pair j of c's, in turn."""
    g = gen(seed)
    m, H = c.shape
    k = torch.randn(length, d, generator=g) * 0.5
    heavy = torch.randperm(first, generator=g)[:11]  # (every query sees them, in whole tiles and others)
    k[heavy] += 4.0
    k = k.to(BF16)
    v = (torch.rand(length, d, generator=g) * 2 - 1).to(BF16)
    v[heavy[:3]] = 0.0
    for j in range(d):
        pair = j % (m * H)
        seen = first + pair // H + 1
        p = torch.softmax(k.double()[:seen, c[pair // H, pair % H]], 0)
        for a in heavy[:3]:
            v[a, j] = float(-(p * v.double()[:seen, j]).sum() / p[a])
    return k, v


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m,H,past", [(1, 4, 300), (3, 4, 60), (3, 8, 300), (8, 4, 1000), (2, 1, 2000)])
def test_few_rows_carry_their_weights_in_two_bf16(d, m, H, past):
    print(f"weights d={d} m={m} H={H} past={past}", flush=True)
    length = past + m
    c = torch.randperm(d, generator=gen(d))[:m * H].view(m, H)
    k, v = cancelling(length, d, c, past, seed=m + past)
    cache = Cache([length], 1, d, 16, BF16, seed=5)
    for t in range(length):
        at = (int(cache.table_cpu[0, t // 16]), 0, t % 16)
        cache.kp[at], cache.vp[at] = k[t].to(DEV), v[t].to(DEV)
    q = torch.zeros(m, H, d, dtype=BF16)
    q.scatter_(2, c[..., None], 1.0)
    out = kda.paged_prefill(q.to(DEV), cache.kp, cache.vp, cache.table, cache.len, i32([0, m]), scale=1.0)
    want, size = oracle(k, v, c, past)
    bound = size * (2 * (4 * 16 + 9) * U + 2 * (length + 64) * U + 2.0 ** -16)
    bound = bound + 2.0 ** -8 * (want.abs() + bound)
    worst = float(((out.cpu().double() - want).abs() / bound).max())
    once, _ = oracle(k, v, c, past, rounded=True)
    planted = float(((once - want).abs() / bound).max())
    print(f"  worst {worst:.3f} of the bound, weights of one bf16 {planted:.2f}", flush=True)
    assert planted > 1.2
    assert worst <= 1
