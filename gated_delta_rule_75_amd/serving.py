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
import sys
import warnings

import torch

from . import _DT, _check, _lib

_T, _I32, _F32 = torch.Tensor, torch.int32, torch.float32
_EMPTY = torch.empty
_GET_DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_MINUS_ONE = 2 ** 64 - 1
_U8 = (torch.uint8, torch.bool)
_LIB = None
_M = None  # the marshalling module (binding/kda_marshal.cpp) once the library is loaded, if it is built


def _lib_():
    global _LIB, _M
    if _LIB is None:
        _LIB = _lib.load()
        try:
            from . import _kda_marshal
        except ImportError:
            return _LIB
        # it reads torch's and CPython's structures, so it serves the versions that it was built for only
        here = (torch.__version__, "%d.%d" % tuple(sys.version_info[:2]))
        built = (getattr(_kda_marshal, "torch_version", "?"), getattr(_kda_marshal, "python_version", "?"))
        if here != built:
            warnings.warn("_kda_marshal.so was built for torch %s, python %s, and this is torch %s, python %s: the "
                          "serving calls are marshalled in Python until it is built again" % (*built, *here),
                          RuntimeWarning)
            return _LIB
        _kda_marshal.setup(_RAW_STREAM or _stream_of, _lib.check,
                           {n: ctypes.cast(getattr(_LIB, n), ctypes.c_void_p).value for n in _lib.EXPORTS})
        _M = _kda_marshal
    return _LIB


# A small call costs what its host side takes, so the usual one (plain contiguous tensors on the current
# device) is marshalled in C (`_M`), which returns False for any other.  Those are checked here, each
# tensor in one expression first (`_plain`: a contiguous GPU tensor of the type and device) and described
# only when that fails (`_gpu`, `_rows`: the messages, and tensors with strides).
def _run(fn, di, *args):
    """Calls a library function on the current stream of device `di`, which is made the current one."""
    if _GET_DEVICE() == di:
        status = fn(*args, _stream_of(di))
    else:
        with torch.cuda.device(di):
            status = fn(*args, _stream_of(di))
    if status:
        _lib.check(status)


def _stream_of(di):
    return _RAW_STREAM(di) if _RAW_STREAM is not None else torch.cuda.current_stream(di).cuda_stream


def _plain(t, dtype, di):
    return type(t) is _T and t.dtype is dtype and t.get_device() == di and t.is_contiguous()


def _gpu(t, name, dtype, dim, di):
    """Raises unless t is a GPU tensor of `dtype` and `dim` axes on device `di`, with any strides."""
    if not isinstance(t, _T):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} axes, got {t.dim()}")
    if t.get_device() != di:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{di}")


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


def _row(t, name, dtype, dim, di):
    """Elements between the rows of a tensor of `dim` axes whose rows are contiguous."""
    if _plain(t, dtype, di) and t.dim() == dim:
        return t.stride(0)
    _gpu(t, name, dtype, dim, di)
    return _rows(t, name, t.shape)


def _vector(t, name, dtype, shape, di):
    """Raises unless t is a contiguous GPU tensor of that type and shape (None: any of one axis)."""
    if _plain(t, dtype, di) and (t.shape == shape if shape is not None else t.dim() == 1):
        return
    _gpu(t, name, dtype, 1 if shape is None else len(shape), di)
    _check(t, name, dtype, shape, None)


def _int32(**values):
    """Raises for a whole number that the library's 32-bit arguments do not hold (ctypes would cut it)."""
    for name, x in values.items():
        if not -2 ** 31 <= int(x) < 2 ** 31:
            raise ValueError(f"{name} must be a 32-bit whole number, got {x}")


def _lead(t, name):
    """Type code and device index of the tensor that the others go by."""
    if not isinstance(t, _T):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DT.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    di = t.get_device()
    if di < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return code, di


def _table(t, name):
    """Row stride and device index of a page table."""
    if not isinstance(t, _T):
        raise TypeError(f"{name} must be a torch.Tensor")
    di = t.get_device()
    if di < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return _row(t, name, _I32, 2, di), di


def _run_scratch(fn, di, workspace, size, *args):
    """_run with the workspace's address and bytes behind args: the caller's when it is large enough (the
    library says so), else a new one of size[0](*size[1:]) bytes."""
    if workspace is not None:
        if not _plain(workspace, torch.uint8, di):
            _gpu(workspace, "workspace", torch.uint8, None, di)
            _check(workspace, "workspace")
        if _GET_DEVICE() == di:
            status = fn(*args, workspace.data_ptr(), workspace.numel(), _stream_of(di))
            if status == 0:
                return
            if status != _lib.KDA_ERR_WORKSPACE:
                _lib.check(status)
    need = size[0](*size[1:])
    if need == _MINUS_ONE:
        need = 0  # the call says what is wrong
    ws = _EMPTY(need, dtype=torch.uint8, device=torch.device("cuda", di)) if need else None
    _run(fn, di, *args, ws.data_ptr() if need else None, need)


def cache_append(k, v, k_pages, v_pages, page_table, start, *, cu_seqlens=None):
    """Writes the keys and values of new tokens into their pages.

    k, v [T,H_kv,d] (float32 or bfloat16; rows of any stride), k_pages, v_pages [n_pages,H_kv,page_size,d]
    (pages of any stride), page_table int32 [N,P], start int32 [N]: the position of each sequence's first
    new token.  cu_seqlens None: one token per sequence (T = N); else int32 [N+1], packed segments.
    Positions without a page are dropped."""
    if _M is not None:
        done = _M.cache_append(k, v, k_pages, v_pages, page_table, start, cu_seqlens)
        if done is not False:
            return
    code, di = _lead(k, "k")
    dt = k.dtype
    ks, vs = _row(k, "k", dt, 3, di), _row(v, "v", dt, 3, di)
    kps, vps = _row(k_pages, "k_pages", dt, 4, di), _row(v_pages, "v_pages", dt, 4, di)
    shape, pages = k.shape, k_pages.shape
    T, H, d = shape
    n_pages, Hp, page_size, dp = pages
    if v.shape != shape or v_pages.shape != pages or Hp != H or dp != d:
        raise ValueError(f"k {tuple(shape)}, v {tuple(v.shape)}, k_pages {tuple(pages)} and v_pages "
                         f"{tuple(v_pages.shape)} do not go together")
    ts = _row(page_table, "page_table", _I32, 2, di)
    N, P = page_table.shape
    _vector(start, "start", _I32, (N,), di)
    cu = None
    if cu_seqlens is not None:
        _vector(cu_seqlens, "cu_seqlens", _I32, (N + 1,), di)
        cu = cu_seqlens.data_ptr()
    _run(_lib_().kda_cache_append, di, k.data_ptr(), v.data_ptr(), ks, vs, cu, start.data_ptr(), N, T,
         k_pages.data_ptr(), v_pages.data_ptr(), kps, vps, n_pages, page_size, page_table.data_ptr(), ts, P, H, d,
         code)


def paged_decode(q, k_pages, v_pages, page_table, lengths, *, scale=None, window=0, sinks=0, max_length=None,
                 out=None, lse=None, workspace=None):
    """Softmax attention of one new token per sequence over its pages (its own key and value among them).

    q [N,H_q,d] (float32 or bfloat16; rows of any stride), k_pages, v_pages [n_pages,H_kv,page_size,d],
    page_table int32 [N,P], lengths int32 [N].  scale: 1 / sqrt(d) by default.  window > 0: only the last
    `window` tokens and the first `sinks` are visible.  max_length: an upper bound of lengths that sizes the
    launch (P * page_size by default).
    Returns out [N,H_q,d] float32; with lse=True (or a tensor for it) (out, lse [N,H_q] float32).  A sequence
    with no visible token gives 0 and -inf."""
    if _M is not None:
        done = _M.paged_decode(q, k_pages, v_pages, page_table, lengths, scale, window, sinks, max_length, out, lse,
                               workspace)
        if done is not False:
            return done
    _int32(window=window, sinks=sinks)
    code, di = _lead(q, "q")
    dt = q.dtype
    qs = _row(q, "q", dt, 3, di)
    kps, vps = _row(k_pages, "k_pages", dt, 4, di), _row(v_pages, "v_pages", dt, 4, di)
    shape, pages = q.shape, k_pages.shape
    N, Hq, d = shape
    n_pages, H, page_size, dp = pages
    ts = _row(page_table, "page_table", _I32, 2, di)
    rows, P = page_table.shape
    if v_pages.shape != pages or dp != d or rows != N:
        raise ValueError(f"q {tuple(shape)}, k_pages {tuple(pages)}, v_pages {tuple(v_pages.shape)} and page_table "
                         f"{(rows, P)} do not go together")
    _vector(lengths, "lengths", _I32, (N,), di)
    dev = q.device
    if out is None:
        out = _EMPTY(shape, dtype=_F32, device=dev)
    else:
        _vector(out, "out", _F32, shape, di)
    if lse is None or lse is False:
        lse = pl = None
    else:
        if lse is True:
            lse = _EMPTY((N, Hq), dtype=_F32, device=dev)
        else:
            _vector(lse, "lse", _F32, (N, Hq), di)
        pl = lse.data_ptr()
    most = P * page_size
    if max_length is not None and max_length < most:
        if max_length < 0:
            raise ValueError("max_length must be >= 0")
        most = max_length if max_length else 1  # 0 would mean no bound
    L = _lib_()
    _run_scratch(L.kda_paged_decode, di, workspace,
                 (L.kda_paged_decode_workspace, N, Hq, H, d, code, most, window, sinks), q.data_ptr(), qs,
                 k_pages.data_ptr(), v_pages.data_ptr(), kps, vps, n_pages, page_size, page_table.data_ptr(), ts, P,
                 lengths.data_ptr(), N, Hq, H, d, code, d ** -0.5 if scale is None else scale, window, sinks, most,
                 out.data_ptr(), pl)
    return out if lse is None else (out, lse)


def cache_fork(page_table, lengths, refcount, parents, *, table_out=None, lengths_out=None):
    """A new set of sequences from an old one, sharing its pages: new sequence i is old sequence parents[i]
    (int32 [N_out]), or empty where that is outside [0, N).  The old set is released, so the call branches,
    reorders, keeps and drops sequences; refcount is updated in place.

    Returns (table_out [N_out,P], lengths_out [N_out])."""
    if _M is not None:
        done = _M.cache_fork(page_table, lengths, refcount, parents, table_out, lengths_out)
        if done is not False:
            return done
    ts, di = _table(page_table, "page_table")
    N, P = page_table.shape
    _vector(lengths, "lengths", _I32, (N,), di)
    _vector(refcount, "refcount", _I32, None, di)
    _vector(parents, "parents", _I32, None, di)
    N_out = parents.shape[0]
    dev = page_table.device
    if table_out is None:
        table_out = _EMPTY((N_out, P), dtype=_I32, device=dev)
        os = P
    else:
        os = _row(table_out, "table_out", _I32, 2, di)
        if table_out.shape != (N_out, P):
            raise ValueError(f"table_out must have shape {(N_out, P)}, got {tuple(table_out.shape)}")
    if lengths_out is None:
        lengths_out = _EMPTY(N_out, dtype=_I32, device=dev)
    else:
        _vector(lengths_out, "lengths_out", _I32, (N_out,), di)
    _run(_lib_().kda_cache_fork, di, page_table.data_ptr(), ts, lengths.data_ptr(), N, P, refcount.data_ptr(),
         refcount.shape[0], parents.data_ptr(), N_out, table_out.data_ptr(), os, lengths_out.data_ptr())
    return table_out, lengths_out


def cache_free(page_table, lengths, refcount, rows):
    """Drops sequences in place: the pages of every row in rows (int32 [R]) lose one reference, its entries
    become -1 and its length 0.  Rows outside the table are left out; one named twice is freed once."""
    if _M is not None:
        done = _M.cache_free(page_table, lengths, refcount, rows)
        if done is not False:
            return
    ts, di = _table(page_table, "page_table")
    N, P = page_table.shape
    _vector(lengths, "lengths", _I32, (N,), di)
    _vector(refcount, "refcount", _I32, None, di)
    _vector(rows, "rows", _I32, None, di)
    _run(_lib_().kda_cache_free, di, page_table.data_ptr(), ts, lengths.data_ptr(), N, P, refcount.data_ptr(),
         refcount.shape[0], rows.data_ptr(), rows.shape[0])


def cache_reserve(page_table, lengths, refcount, new_tokens, page_size, *, copies=None, granted=None,
                  workspace=None):
    """Makes room for new_tokens[n] (int32 [N]) more tokens of every sequence, in place: the pages of the new
    positions become the sequence's own, taken lowest first where there is none or a shared one.

    Returns (copies int32 [N,2], granted int32 [N]).  copies: the page pair (old, new) that pages_copy has to
    copy for a sequence whose shared page was partly filled, else (-1, -1).  granted: new_tokens[n], or 0 for
    a sequence that was left as it was because pages (or table columns) ran out; lengths grow by it."""
    if _M is not None:
        done = _M.cache_reserve(page_table, lengths, refcount, new_tokens, page_size, copies, granted, workspace)
        if done is not False:
            return done
    _int32(page_size=page_size)
    ts, di = _table(page_table, "page_table")
    N, P = page_table.shape
    _vector(lengths, "lengths", _I32, (N,), di)
    _vector(refcount, "refcount", _I32, None, di)
    _vector(new_tokens, "new_tokens", _I32, (N,), di)
    dev = page_table.device
    if copies is None:
        copies = _EMPTY((N, 2), dtype=_I32, device=dev)
    else:
        _vector(copies, "copies", _I32, (N, 2), di)
    if granted is None:
        granted = _EMPTY(N, dtype=_I32, device=dev)
    else:
        _vector(granted, "granted", _I32, (N,), di)
    L, n_pages = _lib_(), refcount.shape[0]
    _run_scratch(L.kda_cache_reserve, di, workspace, (L.kda_cache_workspace_size, N, n_pages), page_table.data_ptr(),
                 ts, lengths.data_ptr(), N, P, refcount.data_ptr(), n_pages, page_size, new_tokens.data_ptr(),
                 copies.data_ptr(), granted.data_ptr())
    return copies, granted


def cache_compact(page_table, refcount, *, table_out=None, refcount_out=None, moves=None, workspace=None):
    """Plans the move of the pages in use to the front of the pool, with the fewest copies.

    Returns (table_out, refcount_out, moves int32 [n_pages // 2, 2]); table_out and refcount_out may be given
    as page_table and refcount themselves.  The pages are moved by pages_copy(pools, moves)."""
    if _M is not None:
        done = _M.cache_compact(page_table, refcount, table_out, refcount_out, moves, workspace)
        if done is not False:
            return done
    ts, di = _table(page_table, "page_table")
    N, P = page_table.shape
    _vector(refcount, "refcount", _I32, None, di)
    n_pages = refcount.shape[0]
    dev = page_table.device
    if table_out is None:
        table_out = _EMPTY((N, P), dtype=_I32, device=dev)
        os = P
    else:
        os = _row(table_out, "table_out", _I32, 2, di)
        if table_out.shape != (N, P):
            raise ValueError(f"table_out must have shape {(N, P)}, got {tuple(table_out.shape)}")
    if refcount_out is None:
        refcount_out = _EMPTY(n_pages, dtype=_I32, device=dev)
    else:
        _vector(refcount_out, "refcount_out", _I32, (n_pages,), di)
    if moves is None:
        moves = _EMPTY((n_pages // 2, 2), dtype=_I32, device=dev)
    else:
        _vector(moves, "moves", _I32, (n_pages // 2, 2), di)
    L = _lib_()
    _run_scratch(L.kda_cache_compact, di, workspace, (L.kda_cache_workspace_size, N, n_pages), page_table.data_ptr(),
                 ts, N, P, refcount.data_ptr(), n_pages, table_out.data_ptr(), os, refcount_out.data_ptr(),
                 moves.data_ptr())
    return table_out, refcount_out, moves


def pages_copy(pools, pairs):
    """Copies pages inside each pool: page pairs[i, 0] to page pairs[i, 1] (int32 [M,2]; pairs with an index
    outside the pool, such as -1, are left out).  No page may be the target of two pairs, or the source of one
    and the target of another.

    pools: a tensor [n_pages, ...] or a list of them (any dtypes and sizes, the same n_pages; pages
    contiguous, of any stride), for instance key and value pages, or recurrent states [n_pages,H,dk,dv]."""
    if _M is not None:
        done = _M.pages_copy(pools, pairs)
        if done is not False:
            return
    if isinstance(pools, _T):
        pools = (pools,)
    n = len(pools)
    if n == 0:
        return
    if not isinstance(pools[0], _T):
        raise TypeError("pools[0] must be a torch.Tensor")
    di = pools[0].get_device()
    if di < 0:
        raise ValueError("pools[0] must be a GPU tensor")
    _vector(pairs, "pairs", _I32, (pairs.shape[0] if isinstance(pairs, _T) and pairs.dim() else 0, 2), di)
    base, stride, size, n_pages = [], [], [], pools[0].shape[0] if pools[0].dim() else 0
    for i, t in enumerate(pools):
        if not (type(t) is _T and t.get_device() == di and t.is_contiguous() and t.dim() > 1):
            _gpu(t, f"pools[{i}]", getattr(t, "dtype", None), None, di)
            if t.dim() < 2:
                raise ValueError(f"pools[{i}] must be [{n_pages}, ...], got {tuple(t.shape)}")
        if t.shape[0] != n_pages:
            raise ValueError(f"pools[{i}] must be [{n_pages}, ...], got {tuple(t.shape)}")
        es = t.element_size()
        row = t.numel() // n_pages * es if n_pages else 0
        base.append(t.data_ptr())
        size.append(row)
        stride.append(row if t.is_contiguous() else _rows(t, f"pools[{i}]", t.shape) * es)
    _run(_lib_().kda_pages_copy, di, (ctypes.c_void_p * n)(*base), (ctypes.c_int64 * n)(*stride),
         (ctypes.c_int64 * n)(*size), n, n_pages, pairs.data_ptr(), pairs.shape[0])


def beam_select(logits, scores, *, n_out=None, finished=None, eos=-1, workspace=None):
    """One step of beam search: the n_out (default K) best continuations of each group over its K beams and
    the vocabulary, by scores + log_softmax(logits).

    logits [B,K,V] (float32 or bfloat16; rows of any stride, the same between all), scores float32 [B,K],
    finished uint8 or bool [B,K]: such a beam goes on with `eos` alone at its own score.
    Returns (scores [B,n_out] float32 descending, parents int32 [B,n_out], tokens int32 [B,n_out],
    finished [B,n_out] or None).  Ties go to the lower beam and token; NaN logits count as -inf."""
    if _M is not None:
        done = _M.beam_select(logits, scores, n_out, finished, eos, workspace)
        if done is not False:
            return done
    code, di = _lead(logits, "logits")
    if logits.dim() != 3:
        raise ValueError(f"logits must have 3 axes, got {logits.dim()}")
    B, K, V = logits.shape
    if logits.is_contiguous():
        row = V
    else:
        st = logits.stride()
        row = st[1] if K > 1 else st[0] if B > 1 else V
        if (V > 1 and st[2] != 1) or (K > 1 and B > 1 and st[0] != K * st[1]):
            raise ValueError(f"logits must have contiguous rows of one stride, got strides {st}")
    _vector(scores, "scores", _F32, (B, K), di)
    if n_out is None:
        n_out = K
    _int32(n_out=n_out, eos=eos)
    if n_out < 0:
        raise ValueError("n_out must be positive")
    L = _lib_()
    dev = logits.device
    over = pf = po = None
    if finished is not None:
        if not isinstance(finished, _T) or finished.dtype not in _U8:
            raise ValueError("finished must be a uint8 or bool tensor")
        _vector(finished, "finished", finished.dtype, (B, K), di)
        over = _EMPTY((B, n_out), dtype=finished.dtype, device=dev)
        pf, po = finished.data_ptr(), over.data_ptr()
    best = _EMPTY((B, n_out), dtype=_F32, device=dev)
    parents, tokens = _EMPTY((2, B, n_out), dtype=_I32, device=dev).unbind()
    _run_scratch(L.kda_beam_select, di, workspace, (L.kda_beam_select_workspace, B, K, V, n_out), logits.data_ptr(),
                 row, scores.data_ptr(), pf, B, K, V, n_out, eos, code, best.data_ptr(), parents.data_ptr(),
                 tokens.data_ptr(), po)
    return best, parents, tokens, over


def beam_reorder(states, parents):
    """Reorders fixed-size states to the beams they continue, in place: row b * K + k becomes what row
    b * K + parents[b, k] was (parents int32 [B,K]; outside [0, K): the row stays).

    states: a contiguous tensor [B*K, ...] or a list of them (the layers' recurrent states, for instance
    [B*K,H,dk,dv])."""
    if _M is not None:
        done = _M.beam_reorder(states, parents)
        if done is not False:
            return
    if isinstance(states, _T):
        states = (states,)
    n = len(states)
    if n == 0:
        return
    if not isinstance(states[0], _T):
        raise TypeError("states[0] must be a torch.Tensor")
    di = states[0].get_device()
    if di < 0:
        raise ValueError("states[0] must be a GPU tensor")
    if not (_plain(parents, _I32, di) and parents.dim() == 2):
        _gpu(parents, "parents", _I32, 2, di)
        _check(parents, "parents", _I32)
    B, K = parents.shape
    rows = B * K
    base, size = [], []
    for i, t in enumerate(states):
        if not (type(t) is _T and t.get_device() == di and t.is_contiguous()):
            _gpu(t, f"states[{i}]", getattr(t, "dtype", None), None, di)
            _check(t, f"states[{i}]")
        if t.dim() < 1 or t.shape[0] != rows:
            raise ValueError(f"states[{i}] must be [{rows}, ...], got {tuple(t.shape)}")
        base.append(t.data_ptr())
        size.append(t.numel() // rows * t.element_size() if rows else 0)
    _run(_lib_().kda_beam_reorder, di, (ctypes.c_void_p * n)(*base), (ctypes.c_int64 * n)(*size), n,
         parents.data_ptr(), B, K)
