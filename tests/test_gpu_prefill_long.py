"""Attention of a chunk at serving sizes, a sample of its rows against 64-bit code on the GPU: a prompt next to single tokens
over long contexts, short windows in bf16 over long chunks, drafts of one key head over a long context.

Bounds as in test_gpu_prefill.py, with the row's own sum p |v| in place of the largest value: |out - exact| <= sum p |v|
(4 ds + 2 w + 2 (n + 64) u [+ 2^-8 where the weights may be rounded to bf16]) and the output's rounding.  A lane sums a
quarter of the weights of half of the keys that it holds, so that |lse - exact| <= 2 ds + w + (n / 8 + 140) u + 4 u |lse|:
for 65 536 keys 5e-4 beside 2 ds, where a part left out or taken twice (1/64 of the keys at least) is 1.5e-2 on average."""
import math

import pytest
import torch

import gated_delta_rule_75_amd as kda
from test_gpu_serving import i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def batch(new, past, hq, hkv, d, page, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    total = [a + b for a, b in zip(new, past)]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(new), max(need) + 2), -1, dtype=torch.int32, device=DEV)
    at = 0
    for n, m in enumerate(need):
        table[n, :m] = ids[at:at + m]
        at += m

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(dtype)

    kp, vp = normal(pages, hkv, page, d), normal(pages, hkv, page, d)
    q = normal(sum(new), hq, d) * 2
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    return q, kp, vp, table, total, cu


@pytest.mark.parametrize("name,dtype,new,past,hq,hkv,d,window,sinks", [
    ("prompt and single tokens", BF16, [1, 600, 1, 3, 1], [30000, 100, 9000, 20000, 1], 16, 4, 128, 0, 0),
    ("prompt and single tokens", F32, [1, 300, 1], [20000, 0, 5000], 8, 2, 128, 0, 0),
    ("prompt and single tokens", BF16, [1] * 40 + [900] + [2] * 40, [1500 + 37 * i for i in range(81)], 4, 1, 64, 0, 0),
    ("short window", BF16, [2048, 1500, 2000], [300, 0, 5000], 20, 4, 128, 19, 0),
    ("short window", BF16, [2048, 1500, 2000], [300, 0, 5000], 8, 4, 64, 128, 4),
    ("window", BF16, [3000, 20], [300, 40000], 8, 2, 256, 1024, 70),
    ("one key head", BF16, [5], [65531], 8, 1, 128, 0, 0),
    ("one key head", BF16, [3], [65533], 8, 1, 256, 0, 0),
    ("one key head", F32, [4], [50000], 8, 1, 64, 0, 0),
    ("two key heads", BF16, [2], [100001], 4, 2, 128, 0, 0),
])
def test_paged_prefill_at_serving_sizes(name, dtype, new, past, hq, hkv, d, window, sinks):
    print(f"{name} {dtype} new={sum(new)} past={max(past)} {hq}/{hkv} d={d} window={window}", flush=True)
    page = 64
    q, kp, vp, table, total, cu = batch(new, past, hq, hkv, d, page, dtype, 7)
    out, lse = kda.paged_prefill(q, kp, vp, table, i32(total), i32(cu), window=window, sinks=sinks, lse=True)
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    group = hq // hkv
    few = sum(new) * group <= 32 * len(new)
    worst = [0.0, 0.0]
    for n in range(len(new)) if len(new) < 9 else (0, 1, 39, 40, 41, 80):
        where = table[n, :-(-total[n] // page)].long()
        k = kp[where].transpose(1, 2).reshape(-1, hkv, d)[:total[n]].double()
        v = vp[where].transpose(1, 2).reshape(-1, hkv, d)[:total[n]].double()
        m = new[n]
        for i in sorted({0, 1, 31, 32, 127, 128, m // 3, m // 2, m - 2, m - 1} & set(range(m))):
            p = total[n] - m + i
            t = torch.arange(p + 1, device=DEV)
            seen = t if not window else t[(t > p - window) | (t < sinks)]
            for h in range(hkv):
                x = q[cu[n] + i, h * group:(h + 1) * group].double()
                kk, vv = k[seen, h], v[seen, h]
                s = x @ kk.T * d ** -0.5
                want_lse = torch.logsumexp(s, 1)
                w = torch.softmax(s, 1)
                want, size = w @ vv, w @ vv.abs()
                ds = (d + 3) * U * d ** -0.5 * (x.abs() @ kk.abs().T).amax(1)
                count = len(seen)
                tol = size * (4 * ds + 18 * U + 2 * (count + 64) * U + (2.0 ** -8 if dtype == BF16 and not few else
                                                                      2.0 ** -16 if dtype == BF16 else 0.0))[:, None]
                tol = tol + (2.0 ** -8 if dtype == BF16 else U) * (want.abs() + tol)
                tol_lse = 2 * ds + 9 * U + (count / 8 + 140) * U + 4 * U * want_lse.abs()
                mine = slice(h * group, (h + 1) * group)
                worst[0] = max(worst[0], float(((out[cu[n] + i, mine].double() - want).abs() / tol).max()))
                worst[1] = max(worst[1], float(((lse[cu[n] + i, mine].double() - want_lse).abs() / tol_lse).max()))
    print(f"  of the bounds: {worst[0]:.3f} {worst[1]:.3f}", flush=True)
    assert worst[0] <= 1 and worst[1] <= 1
