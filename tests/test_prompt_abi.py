"""Refusals of the prompt chunks' calls: host-side validation of the C ABI and of the binding, and the
frequencies of rotary positions (no GPU needed: every call here is refused before anything is launched)."""
import math
import os

import pytest
import torch

BASE = 1 << 40
P = [BASE + i * (1 << 34) for i in range(20)]  # aligned, non-overlapping fake buffers, never read


def _lib():
    from gated_delta_rule_75_amd import _lib

    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("HIP library not built")
    return _lib, _lib.load()


def _call(L, name, defaults, **kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    args = dict(defaults, **kw)
    return getattr(L, name)(*args.values())


ROTARY = dict(q=P[0], q_stride=1024, k=P[1], k_stride=256, positions=P[2], freqs=P[3], T=100, Hq=8, Hk=2, d=128, r=128,
              layout=0, amplitude=1.0, inverse=0, dtype=1, q_out=P[4], qo_stride=1024, k_out=P[5], ko_stride=256,
              stream=None)
PLACE = dict(q=P[0], q_stride=1024, k=P[1], k_stride=256, v=P[2], v_stride=256, cu=P[3], start=P[4], N=4, T=100,
             freqs=P[5], r=128, layout=0, amplitude=1.0, q_out=P[6], qo_stride=1024, kp=P[7], vp=P[8], kp_stride=4096,
             vp_stride=4096, n_pages=10, page=16, table=P[9], stride=8, width=8, Hq=8, Hkv=2, d=128, dtype=1,
             stream=None)
SCORE = dict(logits=P[0], row=1000, tokens=P[1], R=50, V=1000, top=4, dtype=1, logprobs=P[2], lse=P[3], entropy=P[4],
             best=P[5], which=P[6], ws=P[7], ws_bytes=1 << 20, stream=None)
GRAD = dict(logits=P[0], row=1000, tokens=P[1], lse=P[2], entropy=P[3], d_logprobs=P[4], d_lse=P[5], d_entropy=P[6], R=50,
            V=1000, dtype=1, out=P[7], out_row=1000, stream=None)
PREFILL = dict(q=P[0], q_stride=1024, kp=P[1], vp=P[2], kp_stride=8192, vp_stride=8192, n_pages=10, page=16, table=P[3],
               stride=8, width=8, lengths=P[4], cu=P[5], N=4, T=100, Hq=8, Hkv=4, d=128, dtype=1, scale=0.1, window=0,
               sinks=0, max_length=0, out=P[6], lse=P[7], ws=P[8], ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("name,defaults,change,status,says", [
    ("kda_rotary", ROTARY, dict(dtype=2), -1, b"dtype"),
    ("kda_rotary", ROTARY, dict(T=-1), -1, b"T must"),
    ("kda_rotary", ROTARY, dict(T=1 << 31), -1, b"T must"),
    ("kda_rotary", ROTARY, dict(d=100), -2, b"d=100"),
    ("kda_rotary", ROTARY, dict(d=520), -2, b"d=520"),
    ("kda_rotary", ROTARY, dict(d=0), -2, b"d=0"),
    ("kda_rotary", ROTARY, dict(r=130), -1, b"rotary_dim"),
    ("kda_rotary", ROTARY, dict(r=63), -1, b"rotary_dim"),
    ("kda_rotary", ROTARY, dict(r=0), -1, b"rotary_dim"),
    ("kda_rotary", ROTARY, dict(Hq=0), -1, b"H_q"),
    ("kda_rotary", ROTARY, dict(Hq=16385), -1, b"H_q"),
    ("kda_rotary", ROTARY, dict(Hk=1025), -1, b"H_k"),
    ("kda_rotary", ROTARY, dict(Hk=0), -1, b"go together"),
    ("kda_rotary", ROTARY, dict(k=None), -1, b"k is required"),
    ("kda_rotary", ROTARY, dict(k=None, Hk=0), -1, b"go together"),
    ("kda_rotary", ROTARY, dict(layout=2), -1, b"layout"),
    ("kda_rotary", ROTARY, dict(amplitude=float("nan")), -1, b"amplitude"),
    ("kda_rotary", ROTARY, dict(freqs=None), -1, b"freqs"),
    ("kda_rotary", ROTARY, dict(freqs=P[3] + 4), -3, b"8-byte"),
    ("kda_rotary", ROTARY, dict(positions=None), -1, b"positions"),
    ("kda_rotary", ROTARY, dict(positions=P[2] + 2), -3, b"4-byte"),
    ("kda_rotary", ROTARY, dict(q=None), -1, b"q is required"),
    ("kda_rotary", ROTARY, dict(q_out=None), -1, b"q_out is required"),
    ("kda_rotary", ROTARY, dict(q_stride=1016), -1, b"overlap"),
    ("kda_rotary", ROTARY, dict(q_stride=1 << 40), -1, b"strides"),
    ("kda_rotary", ROTARY, dict(ko_stride=260), -3, b"k_out"),
    ("kda_rotary", ROTARY, dict(q=P[0] + 8), -3, b"16-byte"),
    ("kda_rotary", ROTARY, dict(q_out=P[0] + 2048), -4, b"overlaps"),
    ("kda_rotary", ROTARY, dict(q_out=P[0], qo_stride=2048), -4, b"overlaps"),
    ("kda_rotary", ROTARY, dict(q_out=P[1]), -4, b"overlaps"),
    ("kda_rotary", ROTARY, dict(k_out=P[0]), -4, b"overlaps"),
    ("kda_rotary", ROTARY, dict(k_out=P[4]), -4, b"overlap"),
    ("kda_rotary", ROTARY, dict(q_out=P[2] - 1024), -4, b"positions or freqs"),
    ("kda_rotary", ROTARY, dict(freqs=P[5] + 64), -4, b"positions or freqs"),
    ("kda_rotary_append", PLACE, dict(d=96), -2, b"d=96"),
    ("kda_rotary_append", PLACE, dict(page=24), -2, b"page_size=24"),
    ("kda_rotary_append", PLACE, dict(dtype=7), -1, b"dtype"),
    ("kda_rotary_append", PLACE, dict(Hkv=0), -1, b"H_kv"),
    ("kda_rotary_append", PLACE, dict(Hq=0), -1, b"H_q"),
    ("kda_rotary_append", PLACE, dict(r=129), -1, b"rotary_dim"),
    ("kda_rotary_append", PLACE, dict(layout=-1), -1, b"layout"),
    ("kda_rotary_append", PLACE, dict(amplitude=float("inf")), -1, b"amplitude"),
    ("kda_rotary_append", PLACE, dict(cu=None), -1, b"T_total must be N"),
    ("kda_rotary_append", PLACE, dict(N=0), -1, b"at least one"),
    ("kda_rotary_append", PLACE, dict(T=-3), -1, b"T_total"),
    ("kda_rotary_append", PLACE, dict(start=None), -1, b"start"),
    ("kda_rotary_append", PLACE, dict(v=None), -1, b"v is required"),
    ("kda_rotary_append", PLACE, dict(v_stride=252), -1, b"tokens of v overlap"),
    ("kda_rotary_append", PLACE, dict(kp_stride=4088), -1, b"pages overlap"),
    ("kda_rotary_append", PLACE, dict(vp=P[7] + 16), -4, b"overlap"),
    ("kda_rotary_append", PLACE, dict(q=P[7]), -4, b"pages overlap"),
    ("kda_rotary_append", PLACE, dict(q_out=P[8]), -4, b"pages overlap"),
    ("kda_rotary_append", PLACE, dict(freqs=P[7] + 64), -4, b"pages overlap"),
    ("kda_rotary_append", PLACE, dict(q_out=P[1]), -4, b"q_out overlaps"),
    ("kda_rotary_append", PLACE, dict(q_out=P[0] + 1024), -4, b"q_out overlaps"),
    ("kda_rotary_append", PLACE, dict(q_out=P[9]), -4, b"q_out overlaps"),
    ("kda_rotary_append", PLACE, dict(stride=7), -1, b"table rows overlap"),
    ("kda_rotary_append", PLACE, dict(stride=1 << 40), -1, b"strides"),
    ("kda_rotary_append", PLACE, dict(n_pages=0), -1, b"n_pages"),
    ("kda_paged_prefill", PREFILL, dict(Hq=6), -1, b"multiple of H_kv"),
    ("kda_paged_prefill", PREFILL, dict(d=192), -2, b"d=192"),
    ("kda_paged_prefill", PREFILL, dict(dtype=2), -1, b"dtype"),
    ("kda_paged_prefill", PREFILL, dict(page=24), -2, b"page_size=24"),
    ("kda_paged_prefill", PREFILL, dict(scale=float("inf")), -1, b"scale"),
    ("kda_paged_prefill", PREFILL, dict(window=-1), -1, b"window"),
    ("kda_paged_prefill", PREFILL, dict(sinks=4), -1, b"sinks"),
    ("kda_paged_prefill", PREFILL, dict(max_length=-1), -1, b"max_length"),
    ("kda_paged_prefill", PREFILL, dict(width=1 << 27, stride=1 << 27), -1, b"2^31"),
    ("kda_paged_prefill", PREFILL, dict(T=-1), -1, b"T_total"),
    ("kda_paged_prefill", PREFILL, dict(T=1 << 31), -1, b"T_total"),
    ("kda_paged_prefill", PREFILL, dict(N=0), -1, b"at least one"),
    ("kda_paged_prefill", PREFILL, dict(lengths=None), -1, b"lengths"),
    ("kda_paged_prefill", PREFILL, dict(cu=None), -1, b"cu_seqlens"),
    ("kda_paged_prefill", PREFILL, dict(out=None), -1, b"out"),
    ("kda_paged_prefill", PREFILL, dict(q=None), -1, b"q is required"),
    ("kda_paged_prefill", PREFILL, dict(q_stride=1016), -1, b"overlap"),
    ("kda_paged_prefill", PREFILL, dict(q_stride=1 << 40), -1, b"strides"),
    ("kda_paged_prefill", PREFILL, dict(q=P[0] + 8), -3, b"16-byte"),
    ("kda_paged_prefill", PREFILL, dict(out=P[6] + 8), -3, b"16-byte"),
    ("kda_paged_prefill", PREFILL, dict(cu=P[5] + 2), -3, b"4-byte"),
    ("kda_paged_prefill", PREFILL, dict(kp_stride=8184), -1, b"pages overlap"),
    ("kda_paged_prefill", PREFILL, dict(stride=7), -1, b"table rows overlap"),
    ("kda_paged_prefill", PREFILL, dict(stride=1 << 62), -1, b"strides"),
    ("kda_paged_prefill", PREFILL, dict(out=P[0]), -4, b"overlaps an input"),
    ("kda_paged_prefill", PREFILL, dict(out=P[1]), -4, b"overlaps an input"),
    ("kda_paged_prefill", PREFILL, dict(lse=P[6] + 64), -4, b"overlap"),
    ("kda_paged_prefill", PREFILL, dict(lse=P[5]), -4, b"overlap"),
    ("kda_paged_prefill", PREFILL, dict(ws=P[8] + 16), -3, b"256-byte"),
    ("kda_paged_prefill", PREFILL, dict(T=4, width=1024, stride=1024, ws=None), -5, b"needed"),
    ("kda_paged_prefill", PREFILL, dict(T=4, width=1024, stride=1024, ws_bytes=64), -5, b"needed"),
    ("kda_token_logprobs", SCORE, dict(dtype=3), -1, b"dtype"),
    ("kda_token_logprobs", SCORE, dict(R=-1), -1, b"R must"),
    ("kda_token_logprobs", SCORE, dict(R=1 << 31), -1, b"R must"),
    ("kda_token_logprobs", SCORE, dict(V=0), -1, b"V=0"),
    ("kda_token_logprobs", SCORE, dict(V=1 << 24, row=1 << 24), -1, b"V=16777216"),
    ("kda_token_logprobs", SCORE, dict(row=999), -1, b"rows overlap"),
    ("kda_token_logprobs", SCORE, dict(row=1 << 40), -1, b"strides"),
    ("kda_token_logprobs", SCORE, dict(logits=None), -1, b"required"),
    ("kda_token_logprobs", SCORE, dict(logits=P[0] + 1), -3, b"aligned"),
    ("kda_token_logprobs", SCORE, dict(top=65), -1, b"top=65"),
    ("kda_token_logprobs", SCORE, dict(top=-1), -1, b"top=-1"),
    ("kda_token_logprobs", SCORE, dict(V=3), -1, b"top=4"),
    ("kda_token_logprobs", SCORE, dict(top=0), -1, b"go together"),
    ("kda_token_logprobs", SCORE, dict(which=None), -1, b"go together"),
    ("kda_token_logprobs", SCORE, dict(tokens=None), -1, b"go together"),
    ("kda_token_logprobs", SCORE, dict(logprobs=None), -1, b"go together"),
    ("kda_token_logprobs", SCORE, dict(lse=P[3] + 2), -3, b"4-byte"),
    ("kda_token_logprobs", SCORE, dict(lse=P[2] + 64), -4, b"overlap"),
    ("kda_token_logprobs", SCORE, dict(entropy=P[0]), -4, b"overlaps an input"),
    ("kda_token_logprobs", SCORE, dict(R=2, V=100000, row=100000, ws_bytes=8), -5, b"needed"),
    ("kda_token_logprobs", SCORE, dict(R=2, V=100000, row=100000, ws=None), -5, b"needed"),
    ("kda_token_logprobs", SCORE, dict(R=2, V=100000, row=100000, ws=P[7] + 8), -3, b"256-byte"),
    ("kda_token_logprobs_grad", GRAD, dict(dtype=3), -1, b"dtype"),
    ("kda_token_logprobs_grad", GRAD, dict(V=0), -1, b"V=0"),
    ("kda_token_logprobs_grad", GRAD, dict(out=None), -1, b"required"),
    ("kda_token_logprobs_grad", GRAD, dict(out_row=999), -1, b"rows overlap"),
    ("kda_token_logprobs_grad", GRAD, dict(lse=None), -1, b"lse"),
    ("kda_token_logprobs_grad", GRAD, dict(tokens=None), -1, b"needs tokens"),
    ("kda_token_logprobs_grad", GRAD, dict(entropy=None), -1, b"needs entropy"),
    ("kda_token_logprobs_grad", GRAD, dict(d_lse=P[5] + 1), -3, b"4-byte"),
    ("kda_token_logprobs_grad", GRAD, dict(out=P[0] + 2000), -4, b"not the same"),
    ("kda_token_logprobs_grad", GRAD, dict(out=P[0], out_row=1008), -4, b"not the same"),
    ("kda_token_logprobs_grad", GRAD, dict(out=P[3] - 64), -4, b"overlaps an input"),
])
def test_calls_are_refused_before_any_launch(name, defaults, change, status, says):
    _l, L = _lib()
    assert _call(L, name, defaults, **change) == status, L.kda_last_error()
    assert says in L.kda_last_error(), L.kda_last_error()


@pytest.mark.parametrize("name,defaults", [
    ("kda_rotary", ROTARY), ("kda_rotary", dict(ROTARY, q_out=P[0], k_out=P[1])),
    ("kda_rotary", dict(ROTARY, k=None, k_out=None, Hk=0)), ("kda_rotary", dict(ROTARY, T=0, q=None, q_out=None)),
    ("kda_rotary_append", PLACE), ("kda_rotary_append", dict(PLACE, q_out=P[0])),
    ("kda_rotary_append", dict(PLACE, cu=None, N=100, stride=8)),
    ("kda_paged_prefill", PREFILL), ("kda_paged_prefill", dict(PREFILL, vp=P[1], lse=None, window=5, sinks=2)),
    ("kda_paged_prefill", dict(PREFILL, T=0, q=None, out=None, N=0)),
    ("kda_token_logprobs", SCORE), ("kda_token_logprobs", dict(SCORE, tokens=None, logprobs=None, entropy=None)),
    ("kda_token_logprobs", dict(SCORE, top=0, best=None, which=None, lse=None)),
    ("kda_token_logprobs_grad", GRAD), ("kda_token_logprobs_grad", dict(GRAD, out=P[0])),
    ("kda_token_logprobs_grad", dict(GRAD, d_lse=None, d_entropy=None, entropy=None))])
def test_the_unchanged_calls_pass_validation(monkeypatch, name, defaults):
    """The refusals above are due to their one change: without it only the injected failure is left."""
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    assert _call(L, name, defaults) == _l.KDA_ERR_HIP and b"injected" in L.kda_last_error()


def test_queries_and_keys_may_be_slices_of_one_projection(monkeypatch):
    """Rows of equal stride that lie between one another do not overlap, in place or not."""
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    kw = dict(q=P[0], k=P[0] + 2 * 1024, q_stride=1536, k_stride=1536)
    assert _call(L, "kda_rotary", ROTARY, **kw) == _l.KDA_ERR_HIP, L.kda_last_error()
    inside = dict(kw, q_out=P[0], k_out=P[0] + 2 * 1024, qo_stride=1536, ko_stride=1536)
    assert _call(L, "kda_rotary", ROTARY, **inside) == _l.KDA_ERR_HIP, L.kda_last_error()
    assert _call(L, "kda_rotary", ROTARY, **dict(inside, k_out=P[0] + 2 * 1024 - 16)) == _l.KDA_ERR_ALIAS
    kw = dict(kw, v=P[0] + 2 * 1280, v_stride=1536, q_out=P[0], qo_stride=1536)
    assert _call(L, "kda_rotary_append", PLACE, **kw) == _l.KDA_ERR_HIP, L.kda_last_error()


@pytest.mark.parametrize("name,defaults,at_most,one_more", [
    ("kda_rotary", dict(ROTARY, k=None, k_out=None, Hk=0, Hq=1, d=512, r=512, q_stride=512, qo_stride=512, q=1 << 45,
                        q_out=1 << 46), dict(T=8 * ((1 << 24) - 1)), dict(T=8 * ((1 << 24) - 1) + 1)),
    ("kda_rotary_append", dict(PLACE, Hq=16384, q_stride=16384 * 64, qo_stride=16384 * 64, d=64, r=64, q=1 << 50,
                               q_out=1 << 52, k=1 << 53, v=1 << 54), dict(T=8 * ((1 << 24) - 1)), dict(T=8 * ((1 << 24) - 1) + 1)),
    ("kda_paged_prefill", dict(PREFILL, Hq=1, Hkv=1, d=64, q_stride=64, kp_stride=1024, vp_stride=1024, q=1 << 45,
                               out=1 << 46, N=1), dict(T=32 * ((1 << 24) - 2)), dict(T=32 * ((1 << 24) - 1))),
    ("kda_token_logprobs", dict(SCORE, V=4, row=4), dict(R=(1 << 24) - 1), dict(R=1 << 24)),
    ("kda_token_logprobs_grad", dict(GRAD, V=4, row=4, out_row=4), dict(R=4 * ((1 << 24) - 1)), dict(R=(1 << 26) - 3)),
])
def test_calls_whose_launch_has_2_to_32_threads_are_refused(monkeypatch, name, defaults, at_most, one_more):
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    assert _call(L, name, defaults, **at_most) == _l.KDA_ERR_HIP and b"injected" in L.kda_last_error()
    assert _call(L, name, defaults, **one_more) == _l.KDA_ERR_INVALID_ARG and b"2^32" in L.kda_last_error()


def test_binding_refuses_host_and_misshapen_tensors():
    import gated_delta_rule_75_amd as kda

    x, t = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    pages = torch.zeros(3, 4, 16, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.rotary(x, x, t, f)
    with pytest.raises(ValueError, match="unsupported dtype"):
        kda.rotary(x.half(), None, t, f)
    with pytest.raises(TypeError, match="torch.Tensor"):
        kda.rotary([1], None, t, f)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.rotary_append(x, x, x, pages, pages, t[:, None], t, f)


def test_workspace_of_paged_prefill():
    _l, L = _lib()
    bad = 2 ** 64 - 1
    good = (2, 10, 8, 2, 128, 1, 5000, 0, 0)
    assert L.kda_paged_prefill_workspace(*good) > 0
    assert L.kda_paged_prefill_workspace(2, 100000, 8, 2, 128, 1, 5000, 0, 0) == 0
    assert L.kda_paged_prefill_workspace(0, 0, 8, 2, 128, 1, 5000, 0, 0) == 0
    for i, x in ((0, -1), (1, -1), (1, 1 << 31), (2, 7), (3, 0), (4, 96), (5, 2), (6, -1), (6, 1 << 31), (7, -1), (8, -1),
                 (0, (1 << 31) - 1)):
        args = list(good)
        args[i] = x
        assert L.kda_paged_prefill_workspace(*args) == bad, args


def test_workspace_of_token_logprobs():
    _l, L = _lib()
    bad = 2 ** 64 - 1
    assert L.kda_token_logprobs_workspace(2, 100000, 5) > 0
    assert L.kda_token_logprobs_workspace(5000, 100000, 5) == 0 and L.kda_token_logprobs_workspace(0, 100000, 5) == 0
    for args in ((-1, 10, 1), (5, 0, 0), (5, 1 << 24, 1), (5, 10, 11), (5, 100, 65), (5, 100, -1), (1 << 31, 100, 1)):
        assert L.kda_token_logprobs_workspace(*args) == bad, args


def test_binding_refuses_misplaced_queries():
    import gated_delta_rule_75_amd as kda

    x, t, n = torch.zeros(2, 4, 64), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(3, 4, 16, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.paged_prefill(x, pages, pages, t, n, n)
    with pytest.raises(ValueError, match="unsupported dtype"):
        kda.paged_prefill(x.half(), pages, pages, t, n, n)
    with pytest.raises(ValueError, match="window"):
        kda.paged_prefill(x, pages, pages, t, n, n, window=2 ** 31)


def test_binding_refuses_misplaced_logits():
    import gated_delta_rule_75_amd as kda

    x, t, f = torch.zeros(2, 40), torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    for call in (lambda: kda.token_logprobs(x, t), lambda: kda.token_logprobs_grad(x, t, f, f)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="unsupported dtype"):
        kda.token_logprobs(x.half(), t)
    with pytest.raises(ValueError, match="top"):
        kda.token_logprobs(x, t, top=2 ** 32)


# ------------------------------------------------------------------------------------------------
# frequencies
# ------------------------------------------------------------------------------------------------
def test_rotary_frequencies():
    from gated_delta_rule_75_amd import rotary_frequencies as freq

    f = freq(128, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (64,)
    for i in (0, 1, 17, 63):
        assert abs(float(f[i]) - 10000.0 ** (-2 * i / 128)) <= 1e-15 * float(f[i]) * 8
    assert torch.equal(freq(128, scaling="linear", factor=4.0, device="cpu"), f / 4.0)
    ntk = freq(128, scaling="ntk", factor=8.0, device="cpu")
    assert float(ntk[0]) == 1.0 and abs(float(ntk[63] / f[63]) * 8.0 - 1) <= 1e-12
    turns = 8192 * f / (2 * math.pi)
    for kind in ("smooth", "ramp"):
        g = freq(128, scaling=kind, factor=16.0, original_length=8192, slow=1.0, fast=4.0, device="cpu")
        ratio = g / f
        assert bool((ratio[turns > 10] == 1.0).all()) and bool(((ratio[turns < 0.5] * 16 - 1).abs() < 1e-12).all())
        assert bool((ratio[1:] <= ratio[:-1] + 1e-12).all())
    smooth = freq(128, scaling="smooth", factor=16.0, original_length=8192, slow=1.0, fast=4.0, device="cpu")
    mid = ((turns > 1) & (turns < 4)).nonzero().flatten().tolist()
    assert mid
    for i in mid:
        keep = (float(turns[i]) - 1.0) / 3.0
        assert abs(float(smooth[i] / f[i]) - (keep + (1 - keep) / 16.0)) <= 1e-12


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0),
                                dict(rotary_dim=8, scaling="linear", factor=0.0), dict(rotary_dim=8, scaling="x"),
                                dict(rotary_dim=2, scaling="ntk"), dict(rotary_dim=8, scaling="smooth"),
                                dict(rotary_dim=8, scaling="ramp", original_length=100, slow=4.0, fast=4.0),
                                dict(rotary_dim=8, base=0.5, scaling="ramp", original_length=100)])
def test_rotary_frequencies_refusals(kw):
    from gated_delta_rule_75_amd import rotary_frequencies

    with pytest.raises(ValueError):
        rotary_frequencies(device="cpu", **kw)


@pytest.mark.parametrize("N,T,Hq,Hkv,d", [(1, 4, 8, 4, 128), (2, 10, 8, 2, 128), (1, 300, 8, 2, 256), (70, 3000, 4, 2, 64),
                                          (40, 9000, 4, 4, 128), (3, 8000, 16, 8, 64), (1, 1, 1, 1, 64), (64, 320, 32, 8, 128),
                                          (65, 325, 8, 1, 128), (2, 0, 8, 2, 128), (0, 0, 8, 2, 128)])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 3)])
def test_workspace_of_paged_prefill_without_a_bound(monkeypatch, N, T, Hq, Hkv, d, dtype, window, sinks):
    """max_length 0 is no bound there as in the call, so the size serves tables of any width: a call with the same
    arguments does not ask for more."""
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    need = L.kda_paged_prefill_workspace(N, T, Hq, Hkv, d, dtype, 0, window, sinks)
    assert need < 1 << 40
    for width in (0, 1, 2, 3, 7, 64, 65, 300, 8191, 1 << 20, (1 << 27) - 257):
        for most in {0, 1, 16 * width, 12345}:
            assert L.kda_paged_prefill_workspace(N, T, Hq, Hkv, d, dtype, max(most, 1), window, sinks) <= need
            status = _call(L, "kda_paged_prefill", PREFILL, q=1 << 45, out=1 << 46, lse=1 << 47, ws=1 << 48, kp=1 << 49,
                           vp=1 << 50, table=1 << 51, N=N, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, q_stride=Hq * d,
                           kp_stride=16 * Hkv * d, vp_stride=16 * Hkv * d, width=width, stride=max(width, 1), window=window,
                           sinks=sinks, max_length=most, ws_bytes=need)
            assert status == _l.KDA_ERR_HIP and b"injected" in L.kda_last_error(), (width, most, L.kda_last_error())


def test_segment_ends_of_the_largest_batch_are_kept_apart_from_the_pages(monkeypatch):
    """2^31 ends are 8 GiB that no output may overlap (the count of them does not fit 32 bits)."""
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    change = dict(N=(1 << 31) - 1, width=0, stride=0, table=None)
    assert _call(L, "kda_rotary_append", PLACE, **change) == _l.KDA_ERR_HIP, L.kda_last_error()
    for where in dict(kp=0, vp=0, q_out=0):
        assert _call(L, "kda_rotary_append", PLACE, **change, **{where: P[3] + (1 << 32)}) == _l.KDA_ERR_ALIAS, where
    from test_serving_abi import APPEND

    far = dict(APPEND, cu=P[10], **change)
    assert _call(L, "kda_cache_append", far) == _l.KDA_ERR_HIP, L.kda_last_error()
    assert _call(L, "kda_cache_append", far, kp=far["cu"] + (1 << 32)) == _l.KDA_ERR_ALIAS


@pytest.mark.parametrize("original_length", [1, 3, 6, 2 * math.pi, 6.3, 7, 40, 200, 201.1])
@pytest.mark.parametrize("kind", ["smooth", "ramp"])
def test_rotary_frequencies_of_short_originals(kind, original_length):
    """Where not even the fastest pair makes more than `slow` turns, all are slowed by the factor; pairs that make fewer
    are in any case."""
    from gated_delta_rule_75_amd import rotary_frequencies as freq

    f = freq(16, device="cpu")
    g = freq(16, scaling=kind, factor=8.0, original_length=original_length, device="cpu") / f
    turns = original_length * f / (2 * math.pi)
    assert bool(((g >= 1 / 8 - 1e-12) & (g <= 1)).all())
    assert bool(((g * 8 - 1).abs() < 1e-12)[turns < 1 - 1e-9].all())
    if float(turns[0]) <= 1:
        assert bool(((g * 8 - 1).abs() < 1e-12).all())
    if float(turns[0]) > 32:
        assert float(g[0]) == 1.0
