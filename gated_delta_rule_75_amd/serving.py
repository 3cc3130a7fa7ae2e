"""Serving next to the recurrence: attention over a paged key-value cache, the cache's pages, and beam
search with its reordering of the fixed-size states.

A hybrid stack runs softmax-attention layers between its recurrent ones.  Their keys and values live
in pages ``[n_pages, H_kv, page_size, d]``; ``page_table`` int32 ``[N, P]`` names the pages of each
sequence (-1: none), ``lengths`` int32 ``[N]`` its tokens, and ``refcount`` int32 ``[n_pages]`` how
many table entries name a page (0: free).  Contracts: ``include/kda.h``.

As in the package's other calls, this module checks and marshals torch tensors; the work is done by
the library's HIP kernels on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DT, _check, _lib, _ptr, _stream, _workspace

_GET_DEVICE = getattr(torch._C, "_cuda_getDevice", None)
_MINUS_ONE = 2 ** 64 - 1
_U8 = (torch.uint8, torch.bool)


def _run(fn, dev, *args):
    """Calls a library function on the current stream of `dev`, which is made the current device."""
    if (_GET_DEVICE() if _GET_DEVICE is not None else torch.cuda.current_device()) == dev.index:
        status = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(dev))
    if status:
        _lib.check(status)


def _gpu(t, name, dtype, dim, device=None):
    """A GPU tensor of `dtype` and `dim` axes, with any strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} axes, got {t.dim()}")
    if device is not None and t.get_device() != device.index:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(t, name, shape):
    """Elements between the rows of a tensor whose rows are contiguous."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    st, want = t.stride(), 1
    for i in range(len(shape) - 1, 0, -1):
        if st[i] != want and shape[i] > 1:
            raise ValueError(f"{name} must be contiguous in all axes but the first, got strides {st}")
        want *= shape[i]
    return st[0] if shape[0] > 1 else want


def _table(t, name, dev):
    _gpu(t, name, torch.int32, 2, dev)
    return _rows(t, name, t.shape)


def _pools(k_pages, v_pages, dt, dev):
    _gpu(k_pages, "k_pages", dt, 4, dev)
    _gpu(v_pages, "v_pages", dt, 4, dev)
    return _rows(k_pages, "k_pages", k_pages.shape), _rows(v_pages, "v_pages", k_pages.shape)


def _kind(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DT.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return code


def _scratch(nbytes, dev, workspace):
    if nbytes == _MINUS_ONE:
        raise _lib.KdaError(_lib.KDA_ERR_INVALID_ARG, "unsupported sizes")
    return _workspace(nbytes, dev, workspace)


def cache_append(k, v, k_pages, v_pages, page_table, start, *, cu_seqlens=None):
    """Writes the keys and values of new tokens into their pages.

    k, v [T,H_kv,d] (float32 or bfloat16; rows of any stride), k_pages, v_pages [n_pages,H_kv,page_size,d]
    (pages of any stride), page_table int32 [N,P], start int32 [N]: the position of each sequence's first
    new token.  cu_seqlens None: one token per sequence (T = N); else int32 [N+1], packed segments.
    Positions without a page are dropped."""
    dt = _kind(k, "k")
    dev = k.device
    _gpu(k, "k", k.dtype, 3)
    _gpu(v, "v", k.dtype, 3, dev)
    T, H, d = k.shape
    ks, vs = _rows(k, "k", k.shape), _rows(v, "v", k.shape)
    kps, vps = _pools(k_pages, v_pages, k.dtype, dev)
    n_pages, _, page_size, _ = k_pages.shape
    if k_pages.shape[1] != H or k_pages.shape[3] != d:
        raise ValueError(f"pages of {tuple(k_pages.shape)} do not hold tokens of {tuple(k.shape)}")
    ts = _table(page_table, "page_table", dev)
    N, P = page_table.shape
    _check(start, "start", torch.int32, (N,), dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    if start is None:
        raise TypeError("start must be a torch.Tensor")
    _run(_lib.load().kda_cache_append, dev, k.data_ptr(), v.data_ptr(), ks, vs, _ptr(cu_seqlens), start.data_ptr(), N,
         T, k_pages.data_ptr(), v_pages.data_ptr(), kps, vps, n_pages, page_size, page_table.data_ptr(), ts, P, H, d,
         dt)


def paged_decode(q, k_pages, v_pages, page_table, lengths, *, scale=None, window=0, sinks=0, max_length=None,
                 out=None, lse=None, workspace=None):
    """Softmax attention of one new token per sequence over its pages (its own key and value among them).

    q [N,H_q,d] (float32 or bfloat16; rows of any stride), k_pages, v_pages [n_pages,H_kv,page_size,d],
    page_table int32 [N,P], lengths int32 [N].  scale: 1 / sqrt(d) by default.  window > 0: only the last
    `window` tokens and the first `sinks` are visible.  max_length: an upper bound of lengths that sizes the
    launch (P * page_size by default).
    Returns out [N,H_q,d] float32; with lse=True (or a tensor for it) (out, lse [N,H_q] float32).  A sequence
    with no visible token gives 0 and -inf."""
    dt = _kind(q, "q")
    dev = q.device
    _gpu(q, "q", q.dtype, 3)
    N, Hq, d = q.shape
    qs = _rows(q, "q", q.shape)
    kps, vps = _pools(k_pages, v_pages, q.dtype, dev)
    n_pages, H, page_size, dp = k_pages.shape
    if dp != d:
        raise ValueError(f"pages of {tuple(k_pages.shape)} do not go with queries of {tuple(q.shape)}")
    ts = _table(page_table, "page_table", dev)
    P = page_table.shape[1]
    if page_table.shape[0] != N:
        raise ValueError(f"page_table must have {N} rows, got {page_table.shape[0]}")
    if lengths is None:
        raise TypeError("lengths must be a torch.Tensor")
    _check(lengths, "lengths", torch.int32, (N,), dev)
    if out is None:
        out = torch.empty((N, Hq, d), dtype=torch.float32, device=dev)
    else:
        _check(out, "out", torch.float32, (N, Hq, d), dev)
    want = lse is not None and lse is not False
    if not want:
        lse = None
    elif lse is True:
        lse = torch.empty((N, Hq), dtype=torch.float32, device=dev)
    else:
        _check(lse, "lse", torch.float32, (N, Hq), dev)
    room = P * page_size
    most = room if max_length is None or max_length > room else int(max_length)
    if most < 0:
        raise ValueError("max_length must be >= 0")
    if most == 0 and room:  # 0 would mean no bound
        most, max_length = 1, 1
    L = _lib.load()
    need = L.kda_paged_decode_workspace(N, Hq, H, d, dt, most, window, sinks)
    ws = _scratch(need, dev, workspace) if need != _MINUS_ONE else None  # the call says what is wrong
    _run(L.kda_paged_decode, dev, q.data_ptr(), qs, k_pages.data_ptr(), v_pages.data_ptr(), kps, vps, n_pages,
         page_size, page_table.data_ptr(), ts, P, lengths.data_ptr(), N, Hq, H, d, dt,
         d ** -0.5 if scale is None else scale, window, sinks, most, out.data_ptr(), _ptr(lse), _ptr(ws),
         need if ws is not None else 0)
    return (out, lse) if want else out


def cache_fork(page_table, lengths, refcount, parents, *, table_out=None, lengths_out=None):
    """A new set of sequences from an old one, sharing its pages: new sequence i is old sequence parents[i]
    (int32 [N_out]), or empty where that is outside [0, N).  The old set is released, so the call branches,
    reorders, keeps and drops sequences; refcount is updated in place.

    Returns (table_out [N_out,P], lengths_out [N_out])."""
    _gpu(page_table, "page_table", torch.int32, 2)
    dev = page_table.device
    ts = _table(page_table, "page_table", dev)
    N, P = page_table.shape
    _need(lengths=lengths, refcount=refcount, parents=parents)
    _check(lengths, "lengths", torch.int32, (N,), dev)
    _gpu(refcount, "refcount", torch.int32, 1, dev)
    _check(refcount, "refcount", torch.int32, None, dev)
    _gpu(parents, "parents", torch.int32, 1, dev)
    _check(parents, "parents", torch.int32, None, dev)
    N_out = parents.shape[0]
    if table_out is None:
        table_out = torch.empty((N_out, P), dtype=torch.int32, device=dev)
    os = _table(table_out, "table_out", dev)
    if table_out.shape != (N_out, P):
        raise ValueError(f"table_out must have shape {(N_out, P)}, got {tuple(table_out.shape)}")
    if lengths_out is None:
        lengths_out = torch.empty(N_out, dtype=torch.int32, device=dev)
    _check(lengths_out, "lengths_out", torch.int32, (N_out,), dev)
    _run(_lib.load().kda_cache_fork, dev, page_table.data_ptr(), ts, lengths.data_ptr(), N, P, refcount.data_ptr(),
         refcount.shape[0], parents.data_ptr(), N_out, table_out.data_ptr(), os, lengths_out.data_ptr())
    return table_out, lengths_out


def _need(**tensors):
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")


def cache_free(page_table, lengths, refcount, rows):
    """Drops sequences in place: the pages of every row in rows (int32 [R]) lose one reference, its entries
    become -1 and its length 0.  Rows outside the table are left out; one named twice is freed once."""
    _gpu(page_table, "page_table", torch.int32, 2)
    dev = page_table.device
    ts = _table(page_table, "page_table", dev)
    N, P = page_table.shape
    _need(lengths=lengths, refcount=refcount, rows=rows)
    _check(lengths, "lengths", torch.int32, (N,), dev)
    _gpu(refcount, "refcount", torch.int32, 1, dev)
    _check(refcount, "refcount", torch.int32, None, dev)
    _gpu(rows, "rows", torch.int32, 1, dev)
    _check(rows, "rows", torch.int32, None, dev)
    _run(_lib.load().kda_cache_free, dev, page_table.data_ptr(), ts, lengths.data_ptr(), N, P, refcount.data_ptr(),
         refcount.shape[0], rows.data_ptr(), rows.shape[0])


def cache_reserve(page_table, lengths, refcount, new_tokens, page_size, *, copies=None, granted=None,
                  workspace=None):
    """Makes room for new_tokens[n] (int32 [N]) more tokens of every sequence, in place: the pages of the new
    positions become the sequence's own, taken lowest first where there is none or a shared one.

    Returns (copies int32 [N,2], granted int32 [N]).  copies: the page pair (old, new) that pages_copy has to
    copy for a sequence whose shared page was partly filled, else (-1, -1).  granted: new_tokens[n], or 0 for
    a sequence that was left as it was because pages (or table columns) ran out; lengths grow by it."""
    _gpu(page_table, "page_table", torch.int32, 2)
    dev = page_table.device
    ts = _table(page_table, "page_table", dev)
    N, P = page_table.shape
    _need(lengths=lengths, refcount=refcount, new_tokens=new_tokens)
    _check(lengths, "lengths", torch.int32, (N,), dev)
    _gpu(refcount, "refcount", torch.int32, 1, dev)
    _check(refcount, "refcount", torch.int32, None, dev)
    _check(new_tokens, "new_tokens", torch.int32, (N,), dev)
    if copies is None:
        copies = torch.empty((N, 2), dtype=torch.int32, device=dev)
    _check(copies, "copies", torch.int32, (N, 2), dev)
    if granted is None:
        granted = torch.empty(N, dtype=torch.int32, device=dev)
    _check(granted, "granted", torch.int32, (N,), dev)
    L = _lib.load()
    need = L.kda_cache_workspace_size(N, refcount.shape[0])
    ws = _scratch(need, dev, workspace)
    _run(L.kda_cache_reserve, dev, page_table.data_ptr(), ts, lengths.data_ptr(), N, P, refcount.data_ptr(),
         refcount.shape[0], page_size, new_tokens.data_ptr(), copies.data_ptr(), granted.data_ptr(), _ptr(ws), need)
    return copies, granted


def cache_compact(page_table, refcount, *, table_out=None, refcount_out=None, moves=None, workspace=None):
    """Plans the move of the pages in use to the front of the pool, with the fewest copies.

    Returns (table_out, refcount_out, moves int32 [n_pages // 2, 2]); table_out and refcount_out may be given
    as page_table and refcount themselves.  The pages are moved by pages_copy(pools, moves)."""
    _gpu(page_table, "page_table", torch.int32, 2)
    dev = page_table.device
    ts = _table(page_table, "page_table", dev)
    N, P = page_table.shape
    _need(refcount=refcount)
    _gpu(refcount, "refcount", torch.int32, 1, dev)
    _check(refcount, "refcount", torch.int32, None, dev)
    n_pages = refcount.shape[0]
    if table_out is None:
        table_out = torch.empty((N, P), dtype=torch.int32, device=dev)
    os = _table(table_out, "table_out", dev)
    if table_out.shape != (N, P):
        raise ValueError(f"table_out must have shape {(N, P)}, got {tuple(table_out.shape)}")
    if refcount_out is None:
        refcount_out = torch.empty(n_pages, dtype=torch.int32, device=dev)
    _check(refcount_out, "refcount_out", torch.int32, (n_pages,), dev)
    if moves is None:
        moves = torch.empty((n_pages // 2, 2), dtype=torch.int32, device=dev)
    _check(moves, "moves", torch.int32, (n_pages // 2, 2), dev)
    L = _lib.load()
    need = L.kda_cache_workspace_size(N, n_pages)
    ws = _scratch(need, dev, workspace)
    _run(L.kda_cache_compact, dev, page_table.data_ptr(), ts, N, P, refcount.data_ptr(), n_pages, table_out.data_ptr(),
         os, refcount_out.data_ptr(), moves.data_ptr(), _ptr(ws), need)
    return table_out, refcount_out, moves


def _list_of(x, name):
    return [x] if isinstance(x, torch.Tensor) else list(x)


def pages_copy(pools, pairs):
    """Copies pages inside each pool: page pairs[i, 0] to page pairs[i, 1] (int32 [M,2]; pairs with an index
    outside the pool, such as -1, are left out).  No page may be the target of two pairs, or the source of one
    and the target of another.

    pools: a tensor [n_pages, ...] or a list of them (any dtypes and sizes, the same n_pages; pages
    contiguous, of any stride), for instance key and value pages, or recurrent states [n_pages,H,dk,dv]."""
    pools = _list_of(pools, "pools")
    _need(pairs=pairs)
    if not pools:
        return
    _need(**{f"pools[{i}]": t for i, t in enumerate(pools)})
    dev = pools[0].device
    _gpu(pairs, "pairs", torch.int32, 2, dev)
    _check(pairs, "pairs", torch.int32, (pairs.shape[0], 2), dev)
    n, n_pages = len(pools), pools[0].shape[0] if pools[0].dim() else 0
    base, stride, size = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)(), (ctypes.c_int64 * n)()
    for i, t in enumerate(pools):
        _gpu(t, f"pools[{i}]", t.dtype, t.dim(), dev)
        if t.dim() < 2 or t.shape[0] != n_pages:
            raise ValueError(f"pools[{i}] must be [{n_pages}, ...], got {tuple(t.shape)}")
        es = t.element_size()
        row = _rows(t, f"pools[{i}]", t.shape)
        base[i], stride[i] = t.data_ptr(), row * es
        size[i] = t[0].numel() * es if n_pages else 0
    _run(_lib.load().kda_pages_copy, dev, base, stride, size, n, n_pages, pairs.data_ptr(), pairs.shape[0])


def beam_select(logits, scores, *, n_out=None, finished=None, eos=-1, workspace=None):
    """One step of beam search: the n_out (default K) best continuations of each group over its K beams and
    the vocabulary, by scores + log_softmax(logits).

    logits [B,K,V] (float32 or bfloat16; rows of any stride, the same between all), scores float32 [B,K],
    finished uint8 or bool [B,K]: such a beam goes on with `eos` alone at its own score.
    Returns (scores [B,n_out] float32 descending, parents int32 [B,n_out], tokens int32 [B,n_out],
    finished [B,n_out] or None).  Ties go to the lower beam and token; NaN logits count as -inf."""
    dt = _kind(logits, "logits")
    dev = logits.device
    _gpu(logits, "logits", logits.dtype, 3)
    B, K, V = logits.shape
    st = logits.stride()
    row = st[1] if K > 1 else st[0] if B > 1 else V
    if (V > 1 and st[2] != 1) or (K > 1 and B > 1 and st[0] != K * st[1]):
        raise ValueError(f"logits must have contiguous rows of one stride, got strides {st}")
    _need(scores=scores)
    _check(scores, "scores", torch.float32, (B, K), dev)
    if n_out is None:
        n_out = K
    over = None
    if finished is not None:
        if not isinstance(finished, torch.Tensor) or finished.dtype not in _U8:
            raise ValueError("finished must be a uint8 or bool tensor")
        _check(finished, "finished", finished.dtype, (B, K), dev)
        over = torch.empty((B, n_out), dtype=finished.dtype, device=dev)
    L = _lib.load()
    need = L.kda_beam_select_workspace(B, K, V, n_out)
    if need == _MINUS_ONE:
        raise _lib.KdaError(_lib.KDA_ERR_INVALID_ARG, f"kda_beam_select: unsupported B={B} K={K} V={V} n_out={n_out}")
    ws = _scratch(need, dev, workspace)
    best = torch.empty((B, n_out), dtype=torch.float32, device=dev)
    parents = torch.empty((B, n_out), dtype=torch.int32, device=dev)
    tokens = torch.empty((B, n_out), dtype=torch.int32, device=dev)
    _run(L.kda_beam_select, dev, logits.data_ptr(), row, scores.data_ptr(), _ptr(finished), B, K, V, n_out, eos, dt,
         best.data_ptr(), parents.data_ptr(), tokens.data_ptr(), _ptr(over), _ptr(ws), need)
    return best, parents, tokens, over


def beam_reorder(states, parents):
    """Reorders fixed-size states to the beams they continue, in place: row b * K + k becomes what row
    b * K + parents[b, k] was (parents int32 [B,K]; outside [0, K): the row stays).

    states: a contiguous tensor [B*K, ...] or a list of them (the layers' recurrent states, for instance
    [B*K,H,dk,dv])."""
    states = _list_of(states, "states")
    _need(parents=parents)
    if not states:
        return
    _need(**{f"states[{i}]": t for i, t in enumerate(states)})
    dev = states[0].device
    _gpu(parents, "parents", torch.int32, 2, dev)
    _check(parents, "parents", torch.int32, None, dev)
    B, K = parents.shape
    n = len(states)
    base, size = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)()
    for i, t in enumerate(states):
        _check(t, f"states[{i}]", None, None, dev)
        if t.dim() < 1 or t.shape[0] != B * K:
            raise ValueError(f"states[{i}] must be [{B * K}, ...], got {tuple(t.shape)}")
        base[i], size[i] = t.data_ptr(), (t.numel() // (B * K)) * t.element_size() if B * K else 0
    _run(_lib.load().kda_beam_reorder, dev, base, size, n, parents.data_ptr(), B, K)
