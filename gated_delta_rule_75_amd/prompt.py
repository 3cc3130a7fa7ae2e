"""Prompt chunks through the attention layers of a hybrid stack: rotary positions, attention over the
cache's pages, and log-probabilities of the tokens that follow.

New tokens are packed ``[T, H, d]`` with ``cu_seqlens`` int32 ``[N + 1]``; pages and tables are those of
``serving.py``.  Contracts: ``include/kda.h``.

As in the package's other calls, this module checks and marshals torch tensors; the work is done by
the library's HIP kernels on the current stream of the tensors' device.

Autograd records none of the calls: what they return requires no gradient, whatever their inputs do (an output that
is given is returned as it is).  In training they are the two sides of a ``torch.autograd.Function``: ``rotary`` with its own ``inverse=True`` as the backward,
``token_logprobs`` with ``token_logprobs_grad``; ``paged_prefill`` has no backward.  Tensors that a call is given to
write to (outputs, pages) count as modified in place, so that a backward pass that needs their old values fails.
"""
from __future__ import annotations

import math

import torch

from . import _lib, serving
from .serving import _EMPTY, _F32, _I32, _int32, _lead, _lib_, _row, _run, _run_scratch, _vector

_F64 = torch.float64
_WRITTEN = torch.autograd.graph.increment_version
_LAYOUTS = {"half": _lib.KDA_ROTARY_HALVES, "interleaved": _lib.KDA_ROTARY_INTERLEAVED}


def rotary_frequencies(rotary_dim, *, base=10000.0, scaling=None, factor=1.0, original_length=None, slow=1.0,
                       fast=32.0, device="cuda"):
    """Frequencies (radians per token) of rotary positions, float64 [rotary_dim / 2]: base^(-2 i / rotary_dim).

    scaling for contexts `factor` times longer than `original_length`, with t_i the turns of pair i over
    original_length tokens:
      "linear"  f / factor
      "ntk"     base * factor^(rotary_dim / (rotary_dim - 2)): the slowest pair turns 1 / factor as fast
      "smooth"  f / factor where t <= slow, f where t >= fast, linear in t between
      "ramp"    the same ends, linear in i between the pairs that make `fast` and `slow` turns (these rounded
                down and up, and kept in 0 .. rotary_dim - 1)
    Any other frequencies may be used as well.  The factor of the rotated channels that such scalings come with
    is the calls' `amplitude`, for instance 0.1 log(factor) + 1."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and positive, got {rotary_dim}")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling == "ntk":
        if rotary_dim < 4:
            raise ValueError("scaling 'ntk' needs a rotary_dim of 4 or more")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    i = torch.arange(rotary_dim // 2, dtype=_F64)
    f = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling in ("smooth", "ramp"):
        if original_length is None or not original_length > 0 or not fast > slow > 0:
            raise ValueError(f"scaling {scaling!r} needs original_length > 0 and fast > slow > 0")
        if scaling == "smooth":
            keep = (original_length * f / (2 * math.pi) - slow) / (fast - slow)
        else:
            if not base > 1:
                raise ValueError("scaling 'ramp' needs a base above 1")
            # the (fractional) pair that makes `turns` turns
            lo, hi = (rotary_dim * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))
                      for turns in (fast, slow))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rotary_dim - 1)
            # (hi <= 0: no pair makes more than `slow` turns)
            keep = 1.0 - (i - lo) / max(hi - lo, 1e-3) if hi > 0 else torch.zeros_like(i)
        keep = keep.clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device)


def _turn(freqs, layout, di, d):
    """Layout code and rotary_dim."""
    code = _LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    _vector(freqs, "freqs", _F64, None, di)
    if freqs.shape[0] < 1 or 2 * freqs.shape[0] > d:
        raise ValueError(f"freqs must have 1 .. {d // 2} values, got {freqs.shape[0]}")
    return code, 2 * freqs.shape[0]


def _turned(out, name, x, di):
    """The given output for x, or a new contiguous one, and its row stride."""
    if out is None:
        out = _EMPTY(x.shape, dtype=x.dtype, device=x.device)
        return out, out.stride(0)
    stride = _row(out, name, x.dtype, 3, di)
    if out.shape != x.shape:
        raise ValueError(f"{name} must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
    return out, stride


def rotary(q, k, positions, freqs, *, layout="half", amplitude=1.0, inverse=False, q_out=None, k_out=None):
    """Rotary positions of queries and keys.

    q [T,H_q,d], k [T,H_k,d] or None (float32 or bfloat16; rows of any stride), positions int32 [T], freqs
    float64 [rotary_dim / 2] (``rotary_frequencies``); channels from rotary_dim on are copied.  layout "half":
    pairs (i, i + rotary_dim / 2); "interleaved": pairs (2 i, 2 i + 1).  The rotated channels are multiplied by
    amplitude.  inverse=True rotates back by the same angles: given the gradients of the outputs, the call
    returns those of q and k (autograd does not do so by itself: the outputs require no gradient).  q_out, k_out:
    outputs, which may be q and k themselves.

    Returns (q_out, k_out), k_out None without k."""
    if serving._M is not None:
        done = serving._M.rotary(q, k, positions, freqs, layout, amplitude, inverse, q_out, k_out)
        if done is not False:
            return done
    code, di = _lead(q, "q")
    qs = _row(q, "q", q.dtype, 3, di)
    T, Hq, d = q.shape
    Hk = ks = kos = 0
    pk = pko = None
    if k is not None:
        ks = _row(k, "k", q.dtype, 3, di)
        if k.shape[0] != T or k.shape[2] != d:
            raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} do not go together")
        Hk = k.shape[1]
    elif k_out is not None:
        raise ValueError("k_out given without k")
    if (Hq | Hk | d) >> 31:
        _int32(H_q=Hq, H_k=Hk, d=d)
    _vector(positions, "positions", _I32, (T,), di)
    lay, r = _turn(freqs, layout, di, d)
    q_out, qos = _turned(q_out, "q_out", q, di)
    if k is not None:
        k_out, kos = _turned(k_out, "k_out", k, di)
        pk, pko = k.data_ptr(), k_out.data_ptr()
    _run(_lib_().kda_rotary, di, q.data_ptr(), qs, pk, ks, positions.data_ptr(), freqs.data_ptr(), T, Hq, Hk, d, r, lay,
         amplitude, int(bool(inverse)), code, q_out.data_ptr(), qos, pko, kos)
    _WRITTEN([q_out] if k is None else [q_out, k_out])
    return q_out, k_out


def rotary_append(q, k, v, k_pages, v_pages, page_table, start, freqs, *, cu_seqlens=None, layout="half",
                  amplitude=1.0, q_out=None):
    """``rotary`` and ``cache_append`` in one launch: the rotated keys and the values go into their pages.

    q [T,H_q,d], k, v [T,H_kv,d]; k_pages, v_pages, page_table, start and cu_seqlens as in cache_append: token i
    of sequence n is at position start[n] + i.  freqs, layout, amplitude as in rotary.
    Returns q_out [T,H_q,d] (which may be given as q itself), which requires no gradient.  Rows of q_out that belong
    to no sequence are not written."""
    if serving._M is not None:
        done = serving._M.rotary_append(q, k, v, k_pages, v_pages, page_table, start, freqs, cu_seqlens, layout,
                                        amplitude, q_out)
        if done is not False:
            return done
    code, di = _lead(q, "q")
    dt = q.dtype
    qs, ks, vs = _row(q, "q", dt, 3, di), _row(k, "k", dt, 3, di), _row(v, "v", dt, 3, di)
    kps, vps = _row(k_pages, "k_pages", dt, 4, di), _row(v_pages, "v_pages", dt, 4, di)
    T, Hq, d = q.shape
    pages = k_pages.shape
    n_pages, H, page_size, dp = pages
    if k.shape != v.shape or k.shape != (T, H, d) or v_pages.shape != pages or dp != d:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}, k_pages {tuple(pages)} and "
                         f"v_pages {tuple(v_pages.shape)} do not go together")
    ts = _row(page_table, "page_table", _I32, 2, di)
    N, P = page_table.shape
    if (N | P | Hq | H | d | n_pages | page_size) >> 31:
        _int32(N=N, P=P, H_q=Hq, H_kv=H, d=d, n_pages=n_pages, page_size=page_size)
    _vector(start, "start", _I32, (N,), di)
    cu = None
    if cu_seqlens is not None:
        _vector(cu_seqlens, "cu_seqlens", _I32, (N + 1,), di)
        cu = cu_seqlens.data_ptr()
    lay, r = _turn(freqs, layout, di, d)
    q_out, qos = _turned(q_out, "q_out", q, di)
    _run(_lib_().kda_rotary_append, di, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, cu, start.data_ptr(), N,
         T, freqs.data_ptr(), r, lay, amplitude, q_out.data_ptr(), qos, k_pages.data_ptr(), v_pages.data_ptr(), kps,
         vps, n_pages, page_size, page_table.data_ptr(), ts, P, Hq, H, d, code)
    _WRITTEN([q_out, k_pages, v_pages])
    return q_out


def paged_prefill(q, k_pages, v_pages, page_table, lengths, cu_seqlens, *, scale=None, window=0, sinks=0,
                  max_length=None, out=None, lse=None, workspace=None):
    """Softmax attention of the new tokens of every sequence over its pages (their own keys and values among them).

    q [T,H_q,d] (float32 or bfloat16; rows of any stride), packed segments with cu_seqlens int32 [N+1]; k_pages,
    v_pages [n_pages,H_kv,page_size,d], page_table int32 [N,P], lengths int32 [N], the new tokens included: the
    last one of sequence n is at position lengths[n] - 1.  A token sees those before it and itself; window > 0:
    of these only the last `window` and the first `sinks`.  scale: 1 / sqrt(d) by default.  max_length: an upper
    bound of lengths that sizes the launch (P * page_size by default); tokens behind it are not visible.
    Returns out [T,H_q,d] in q's dtype; with lse=True (or a tensor for it) (out, lse [T,H_q] float32).  A token
    that sees none gives 0 and -inf; rows that belong to no sequence are not written.  There is no backward: the
    results require no gradient."""
    if serving._M is not None:
        done = serving._M.paged_prefill(q, k_pages, v_pages, page_table, lengths, cu_seqlens, scale, window, sinks,
                                        max_length, out, lse, workspace)
        if done is not False:
            return done
    _int32(window=window, sinks=sinks)
    code, di = _lead(q, "q")
    dt = q.dtype
    qs = _row(q, "q", dt, 3, di)
    kps, vps = _row(k_pages, "k_pages", dt, 4, di), _row(v_pages, "v_pages", dt, 4, di)
    shape, pages = q.shape, k_pages.shape
    T, Hq, d = shape
    n_pages, H, page_size, dp = pages
    ts = _row(page_table, "page_table", _I32, 2, di)
    N, P = page_table.shape
    if v_pages.shape != pages or dp != d:
        raise ValueError(f"q {tuple(shape)}, k_pages {tuple(pages)} and v_pages {tuple(v_pages.shape)} do not go "
                         "together")
    if (N | P | Hq | H | d | n_pages | page_size) >> 31:
        _int32(N=N, P=P, H_q=Hq, H_kv=H, d=d, n_pages=n_pages, page_size=page_size)
    _vector(lengths, "lengths", _I32, (N,), di)
    _vector(cu_seqlens, "cu_seqlens", _I32, (N + 1,), di)
    dev = q.device
    if out is None:
        out = _EMPTY(shape, dtype=dt, device=dev)
    else:
        _vector(out, "out", dt, shape, di)
    if lse is None or lse is False:
        lse = pl = None
    else:
        if lse is True:
            lse = _EMPTY((T, Hq), dtype=_F32, device=dev)
        else:
            _vector(lse, "lse", _F32, (T, Hq), di)
        pl = lse.data_ptr()
    most = P * page_size
    if max_length is not None and max_length < most:
        if max_length < 0:
            raise ValueError("max_length must be >= 0")
        most = max_length
        if most == 0:
            P = 0  # the library's 0 is no bound; a table without columns shows nothing
    L = _lib_()
    _run_scratch(L.kda_paged_prefill, di, workspace,
                 (L.kda_paged_prefill_workspace, N, T, Hq, H, d, code, most, window, sinks), q.data_ptr(), qs,
                 k_pages.data_ptr(), v_pages.data_ptr(), kps, vps, n_pages, page_size, page_table.data_ptr(), ts, P,
                 lengths.data_ptr(), cu_seqlens.data_ptr(), N, T, Hq, H, d, code, d ** -0.5 if scale is None else scale,
                 window, sinks, most, out.data_ptr(), pl)
    if lse is None:
        _WRITTEN(out)
        return out
    _WRITTEN([out, lse])
    return out, lse


def _optional(t, name, dtype, shape, di):
    """Address of an optional contiguous tensor."""
    if t is None:
        return None
    _vector(t, name, dtype, shape, di)
    return t.data_ptr()


def token_logprobs(logits, tokens, *, top=0, entropy=False, workspace=None):
    """Log-probabilities of given tokens, the rows' log-sums, and on request their entropy and best alternatives.

    logits [R,V] (float32 or bfloat16; rows of any stride), tokens int32 [R], or None; a token outside [0, V) is
    ignored (0).  NaN logits count as -inf.
    Returns (logprobs [R], lse [R], entropy [R], top_logprobs [R,top], top_tokens int32 [R,top]), float32 but for
    the last; None for what was not asked for.  The alternatives are in descending order, ties to the lower
    token; top <= 64.  The results require no gradient: ``token_logprobs_grad`` forms that of the first three."""
    if serving._M is not None:
        done = serving._M.token_logprobs(logits, tokens, top, entropy, workspace)
        if done is not False:
            return done
    _int32(top=top)
    code, di = _lead(logits, "logits")
    stride = _row(logits, "logits", logits.dtype, 2, di)
    R, V = logits.shape
    if V >> 31:
        _int32(V=V)
    if top < 0 or top > V:
        raise ValueError(f"top must be in 0 .. V, got {top}")
    dev = logits.device
    pt = _optional(tokens, "tokens", _I32, (R,), di)
    lp = None if tokens is None else _EMPTY(R, dtype=_F32, device=dev)
    lse = _EMPTY(R, dtype=_F32, device=dev)
    ent = _EMPTY(R, dtype=_F32, device=dev) if entropy else None
    best = _EMPTY((R, top), dtype=_F32, device=dev) if top else None
    which = _EMPTY((R, top), dtype=_I32, device=dev) if top else None
    L = _lib_()
    _run_scratch(L.kda_token_logprobs, di, workspace, (L.kda_token_logprobs_workspace, R, V, top), logits.data_ptr(),
                 stride, pt, R, V, top, code, *(None if x is None else x.data_ptr() for x in (lp, lse, ent, best, which)))
    return lp, lse, ent, best, which


def token_logprobs_grad(logits, tokens, lse, d_logprobs=None, *, d_lse=None, entropy=None, d_entropy=None, out=None):
    """Gradient of ``token_logprobs`` with respect to the logits, in their dtype:
    p (d_lse - d_logprob - d_entropy (log p + entropy)) + d_logprob at the token.

    logits, tokens as given to token_logprobs, lse and entropy float32 [R] as it returned them; d_logprobs, d_lse,
    d_entropy float32 [R] or None (zero).  out: a tensor [R,V], which may be logits itself (they are lost then, also to
    what autograd has saved of them, which raises in its backward)."""
    if serving._M is not None:
        done = serving._M.token_logprobs_grad(logits, tokens, lse, d_logprobs, d_lse, entropy, d_entropy, out)
        if done is not False:
            return done
    code, di = _lead(logits, "logits")
    stride = _row(logits, "logits", logits.dtype, 2, di)
    R, V = logits.shape
    if V >> 31:
        _int32(V=V)
    _vector(lse, "lse", _F32, (R,), di)
    if d_logprobs is not None and tokens is None:
        raise ValueError("d_logprobs needs tokens")
    if d_entropy is not None and entropy is None:
        raise ValueError("d_entropy needs entropy")
    pt = _optional(tokens, "tokens", _I32, (R,), di)
    rows = [_optional(t, name, _F32, (R,), di) for t, name in (
        (entropy, "entropy"), (d_logprobs, "d_logprobs"), (d_lse, "d_lse"), (d_entropy, "d_entropy"))]
    if out is None:
        out = _EMPTY((R, V), dtype=logits.dtype, device=logits.device)
        os = V
    else:
        os = _row(out, "out", logits.dtype, 2, di)
        if out.shape != (R, V):
            raise ValueError(f"out must have shape {(R, V)}, got {tuple(out.shape)}")
    _run(_lib_().kda_token_logprobs_grad, di, logits.data_ptr(), stride, pt, lse.data_ptr(), *rows, R, V, code,
         out.data_ptr(), os)
    _WRITTEN(out)
    return out
