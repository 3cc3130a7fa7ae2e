"""Refusals of the paged-cache and beam-search calls: host-side validation of the C ABI and of the
binding (no GPU needed: every call here is refused before anything is launched)."""
import ctypes
import os

import numpy as np
import pytest
import torch

BASE = 1 << 40
P = [BASE + i * (1 << 34) for i in range(16)]  # aligned, non-overlapping fake buffers, never read


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


APPEND = dict(k=P[0], v=P[1], k_stride=512, v_stride=512, cu=None, start=P[2], N=4, T=4, kp=P[3], vp=P[4],
              kp_stride=8192, vp_stride=8192, n_pages=10, page=16, table=P[5], stride=8, width=8, H=4, d=128, dtype=1,
              stream=None)
DECODE = dict(q=P[0], q_stride=1024, kp=P[1], vp=P[2], kp_stride=8192, vp_stride=8192, n_pages=10, page=16, table=P[3],
              stride=8, width=8, lengths=P[4], N=4, Hq=8, Hkv=4, d=128, dtype=1, scale=0.1, window=0, sinks=0,
              max_length=0, out=P[5], lse=P[6], ws=P[7], ws_bytes=1 << 30, stream=None)
FORK = dict(table=P[0], stride=8, lengths=P[1], N=4, width=8, refs=P[2], n_pages=10, parents=P[3], N_out=6,
            out=P[4], out_stride=8, lengths_out=P[5], stream=None)
FREE = dict(table=P[0], stride=8, lengths=P[1], N=4, width=8, refs=P[2], n_pages=10, rows=P[3], n_rows=2, stream=None)
RESERVE = dict(table=P[0], stride=8, lengths=P[1], N=4, width=8, refs=P[2], n_pages=10, page=16, new=P[3],
               copies=P[4], granted=P[5], ws=P[6], ws_bytes=1 << 20, stream=None)
COMPACT = dict(table=P[0], stride=8, N=4, width=8, refs=P[1], n_pages=10, out=P[2], out_stride=8, refs_out=P[3],
               moves=P[4], ws=P[5], ws_bytes=1 << 20, stream=None)
SELECT = dict(logits=P[0], row=1000, scores=P[1], finished=None, B=2, K=4, V=1000, n_out=4, eos=-1, dtype=0,
              best=P[2], parents=P[3], tokens=P[4], over=None, ws=P[5], ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("name,defaults,change,status,says", [
    ("kda_cache_append", APPEND, dict(d=96), -2, b"d=96"),
    ("kda_cache_append", APPEND, dict(page=24), -2, b"page_size=24"),
    ("kda_cache_append", APPEND, dict(page=8), -2, b"page_size=8"),
    ("kda_cache_append", APPEND, dict(dtype=5), -1, b"dtype"),
    ("kda_cache_append", APPEND, dict(H=0), -1, b"H_kv"),
    ("kda_cache_append", APPEND, dict(T=5), -1, b"T_total must be N"),
    ("kda_cache_append", APPEND, dict(cu=P[6], N=0, T=5), -1, b"at least one"),
    ("kda_cache_append", APPEND, dict(k=None), -1, b"required"),
    ("kda_cache_append", APPEND, dict(k_stride=504), -1, b"tokens overlap"),
    ("kda_cache_append", APPEND, dict(k_stride=516), -3, b"16-byte"),
    ("kda_cache_append", APPEND, dict(v=P[1] + 8), -3, b"16-byte"),
    ("kda_cache_append", APPEND, dict(kp_stride=8184), -1, b"pages overlap"),
    ("kda_cache_append", APPEND, dict(kp_stride=8196), -3, b"16-byte"),
    ("kda_cache_append", APPEND, dict(kp_stride=1 << 41), -1, b"strides"),
    ("kda_cache_append", APPEND, dict(vp=P[3] + 8192), -4, b"overlap"),
    ("kda_cache_append", APPEND, dict(k=P[3]), -4, b"overlap an input"),
    ("kda_cache_append", APPEND, dict(table=P[3] + 64), -4, b"overlap an input"),
    ("kda_cache_append", APPEND, dict(n_pages=0), -1, b"n_pages"),
    ("kda_cache_append", APPEND, dict(n_pages=1 << 24), -1, b"n_pages"),
    ("kda_cache_append", APPEND, dict(stride=7), -1, b"table rows overlap"),
    ("kda_cache_append", APPEND, dict(N=-1), -1, b">= 0"),
    ("kda_paged_decode", DECODE, dict(Hq=6), -1, b"multiple of H_kv"),
    ("kda_paged_decode", DECODE, dict(d=192), -2, b"d=192"),
    ("kda_paged_decode", DECODE, dict(scale=float("nan")), -1, b"scale"),
    ("kda_paged_decode", DECODE, dict(window=-1), -1, b"window"),
    ("kda_paged_decode", DECODE, dict(sinks=4), -1, b"sinks"),
    ("kda_paged_decode", DECODE, dict(max_length=-1), -1, b"max_length"),
    ("kda_paged_decode", DECODE, dict(width=1 << 28, stride=1 << 28, N=1), -1, b"2^31"),
    ("kda_paged_decode", DECODE, dict(lengths=None), -1, b"lengths"),
    ("kda_paged_decode", DECODE, dict(q_stride=1016), -1, b"queries overlap"),
    ("kda_paged_decode", DECODE, dict(q=P[0] + 8), -3, b"16-byte"),
    ("kda_paged_decode", DECODE, dict(out=P[0]), -4, b"overlaps an input"),
    ("kda_paged_decode", DECODE, dict(lse=P[5] + 64), -4, b"overlap"),
    ("kda_paged_decode", DECODE, dict(ws=P[7] + 16), -3, b"256-byte"),
    ("kda_cache_fork", FORK, dict(out=P[0]), -4, b"overlaps"),
    ("kda_cache_fork", FORK, dict(out_stride=4), -1, b"rows overlap"),
    ("kda_cache_fork", FORK, dict(parents=None), -1, b"parents"),
    ("kda_cache_fork", FORK, dict(lengths_out=P[1]), -4, b"overlaps"),
    ("kda_cache_fork", FORK, dict(refs=P[2] + 2), -3, b"4-byte"),
    ("kda_cache_free", FREE, dict(rows=None), -1, b"rows"),
    ("kda_cache_free", FREE, dict(n_rows=-1), -1, b"rows"),
    ("kda_cache_free", FREE, dict(rows=P[1]), -4, b"overlaps"),
    ("kda_cache_reserve", RESERVE, dict(page=0), -1, b"page_size"),
    ("kda_cache_reserve", RESERVE, dict(ws_bytes=16), -5, b"needed"),
    ("kda_cache_reserve", RESERVE, dict(ws=None), -5, b"needed"),
    ("kda_cache_reserve", RESERVE, dict(granted=P[4] + 8), -4, b"overlap"),
    ("kda_cache_reserve", RESERVE, dict(new=P[0] + 16), -4, b"overlaps"),
    ("kda_cache_compact", COMPACT, dict(refs_out=P[1] + 4), -4, b"partially"),
    ("kda_cache_compact", COMPACT, dict(out=P[0], out_stride=9), -4, b"partially"),
    ("kda_cache_compact", COMPACT, dict(moves=P[0]), -4, b"overlaps"),
    ("kda_cache_compact", COMPACT, dict(moves=None), -1, b"moves"),
    ("kda_cache_compact", COMPACT, dict(ws_bytes=0), -5, b"needed"),
    ("kda_beam_select", SELECT, dict(K=65, n_out=4), -1, b"K=65"),
    ("kda_beam_select", SELECT, dict(n_out=65), -1, b"n_out=65"),
    ("kda_beam_select", SELECT, dict(V=0), -1, b"V=0"),
    ("kda_beam_select", SELECT, dict(K=1, V=3, row=3), -1, b"n_out"),
    ("kda_beam_select", SELECT, dict(row=999), -1, b"row_stride"),
    ("kda_beam_select", SELECT, dict(dtype=3), -1, b"dtype"),
    ("kda_beam_select", SELECT, dict(finished=P[6], over=P[7]), -1, b"eos"),
    ("kda_beam_select", SELECT, dict(finished=P[6], over=P[7], eos=1000), -1, b"eos"),
    ("kda_beam_select", SELECT, dict(finished=P[6], eos=2), -1, b"go together"),
    ("kda_beam_select", SELECT, dict(logits=P[0] + 2), -3, b"aligned"),
    ("kda_beam_select", SELECT, dict(tokens=P[3]), -4, b"overlap"),
    ("kda_beam_select", SELECT, dict(best=P[0]), -4, b"overlaps an input"),
    ("kda_beam_select", SELECT, dict(ws_bytes=8), -5, b"needed"),
])
def test_calls_are_refused_before_any_launch(name, defaults, change, status, says):
    _l, L = _lib()
    assert _call(L, name, defaults, **change) == status, L.kda_last_error()
    assert says in L.kda_last_error(), L.kda_last_error()


@pytest.mark.parametrize("name,defaults", [
    ("kda_cache_append", APPEND), ("kda_paged_decode", DECODE), ("kda_cache_fork", FORK), ("kda_cache_free", FREE),
    ("kda_cache_reserve", RESERVE), ("kda_cache_compact", COMPACT), ("kda_beam_select", SELECT)])
def test_the_unchanged_calls_pass_validation(monkeypatch, name, defaults):
    """The refusals above are due to their one change: without it only the injected failure is left."""
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    assert _call(L, name, defaults) == _l.KDA_ERR_HIP and b"injected" in L.kda_last_error()


FAR = [1 << 45, 1 << 46, 1 << 47]  # fake buffers far enough apart for the largest calls


@pytest.mark.parametrize("name,defaults,at_most,one_more", [
    ("kda_cache_append", dict(APPEND, cu=P[6], k=FAR[0], v=FAR[1], H=1, d=64, k_stride=64, v_stride=64, kp_stride=1024,
                              vp_stride=1024), dict(T=(1 << 28) - 16), dict(T=1 << 28)),
    ("kda_paged_decode", dict(DECODE, Hq=1, Hkv=1, d=64, q_stride=64, kp_stride=1024, vp_stride=1024),
     dict(N=(1 << 24) - 1), dict(N=1 << 24)),
    # 4096 tokens are two parts, and the launch that joins them has a workgroup for every query head
    ("kda_paged_decode", dict(DECODE, Hq=128, Hkv=8, d=64, q_stride=128 * 64, kp_stride=8 << 18, vp_stride=8 << 18,
                              n_pages=2, page=4096, width=1, ws=FAR[0], ws_bytes=1 << 40),
     dict(N=(1 << 17) - 1), dict(N=1 << 17)),
    ("kda_cache_fork", dict(FORK, width=1 << 26, stride=1 << 26, out_stride=1 << 26, N=0, table=None, out=FAR[0]),
     dict(N_out=63), dict(N_out=64)),
    ("kda_cache_free", FREE, dict(n_rows=(1 << 24) - 1), dict(n_rows=1 << 24)),
    ("kda_cache_reserve", dict(RESERVE, ws_bytes=1 << 33, table=FAR[0]), dict(N=4 * ((1 << 24) - 2)),
     dict(N=4 * ((1 << 24) - 2) + 1)),  # one workgroup for the ten pages, one for every four sequences
    ("kda_cache_compact", dict(COMPACT, ws_bytes=1 << 30), dict(N=(1 << 24) - 2), dict(N=(1 << 24) - 1)),
    ("kda_beam_select", dict(SELECT, K=1, V=4, row=4, n_out=1), dict(B=(1 << 24) - 1), dict(B=1 << 24)),
])
def test_calls_whose_launch_has_2_to_32_threads_are_refused(monkeypatch, name, defaults, at_most, one_more):
    """A grid holds fewer than 2^32 threads, 2^24 - 1 workgroups of 256."""
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    assert _call(L, name, defaults, **at_most) == _l.KDA_ERR_HIP and b"injected" in L.kda_last_error()
    assert _call(L, name, defaults, **one_more) == _l.KDA_ERR_INVALID_ARG and b"2^32" in L.kda_last_error()


@pytest.mark.parametrize("name,defaults", [("kda_cache_append", APPEND), ("kda_paged_decode", DECODE),
                                           ("kda_cache_fork", FORK), ("kda_cache_free", FREE),
                                           ("kda_cache_reserve", RESERVE), ("kda_cache_compact", COMPACT)])
@pytest.mark.parametrize("stride", [1 << 40, 1 << 61, 1 << 62, 2 ** 63 - 1])
def test_table_strides_beyond_2_to_40_are_refused(monkeypatch, name, defaults, stride):
    """In bytes such a stride can wrap to a small one, past the check for overlaps."""
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    assert _call(L, name, defaults, stride=stride) == _l.KDA_ERR_INVALID_ARG and b"stride" in L.kda_last_error()
    # a single row has no stride
    if name in ("kda_cache_append", "kda_paged_decode"):
        one = dict(N=1, T=1) if name == "kda_cache_append" else dict(N=1)
        assert _call(L, name, defaults, stride=stride, **one) == _l.KDA_ERR_HIP, L.kda_last_error()


def test_sizes_whose_products_leave_64_bits_are_refused(monkeypatch):
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    most = 2 ** 31 - 1
    assert _call(L, "kda_paged_decode", DECODE, N=most, Hq=16384, q_stride=16384 * 128, page=4096,
                 kp_stride=4 * 4096 * 128, vp_stride=4 * 4096 * 128, width=most, stride=most) == _l.KDA_ERR_INVALID_ARG
    assert L.kda_paged_decode_workspace(most, 16384, 1, 128, 1, most, 0, 0) == 2 ** 64 - 1
    assert L.kda_paged_decode_workspace(1 << 24, 1, 1, 128, 1, 64, 0, 0) == 2 ** 64 - 1


def test_calls_with_wide_tables_and_few_tokens_are_taken(monkeypatch):
    """16384 sequences of 128 heads with room for 2^20 tokens each, of which no more than 4096 are used."""
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    need = L.kda_paged_decode_workspace(16384, 128, 8, 128, 1, 4096, 0, 0)
    kw = dict(N=16384, Hq=128, Hkv=8, q_stride=128 * 128, kp_stride=8 * 128 * 128, vp_stride=8 * 128 * 128, page=128,
              width=8192, stride=8192, max_length=4096, q=FAR[0], out=FAR[1], ws=FAR[2], ws_bytes=need)
    assert _call(L, "kda_paged_decode", DECODE, **kw) == _l.KDA_ERR_HIP and b"injected" in L.kda_last_error()


def test_pages_of_keys_and_values_may_interleave(monkeypatch):
    """Keys and values in one pool [n_pages, 2, H, page_size, d]: the extents overlap, the pages do not."""
    _l, L = _lib()
    monkeypatch.setenv("KDA_TEST_FAIL_LAUNCH", "1")
    page = 4 * 16 * 128
    kw = dict(kp=P[3], vp=P[3] + page * 2, kp_stride=2 * page, vp_stride=2 * page)
    assert _call(L, "kda_cache_append", APPEND, **kw) == _l.KDA_ERR_HIP and b"injected" in L.kda_last_error()
    kw["vp"] = P[3] + page * 2 - 16
    assert _call(L, "kda_cache_append", APPEND, **kw) == _l.KDA_ERR_ALIAS
    kw["vp"] = P[3] + page * 2 + 16  # its last page ends inside the next key page
    assert _call(L, "kda_cache_append", APPEND, **kw) == _l.KDA_ERR_ALIAS


def _pools(*rows):
    base = (ctypes.c_void_p * len(rows))(*[r[0] for r in rows])
    stride = (ctypes.c_int64 * len(rows))(*[r[1] for r in rows])
    size = (ctypes.c_int64 * len(rows))(*[r[2] for r in rows])
    return base, stride, size


def test_buffer_lists_are_checked():
    _l, L = _lib()

    def copy(rows, n_pages=8, pairs=P[9], n_pairs=4):
        return L.kda_pages_copy(*_pools(*rows), len(rows), n_pages, pairs, n_pairs, None)

    good = (P[0], 4096, 4096)
    assert copy([(P[0], 4096, 4088)]) == _l.KDA_ERR_MISALIGNED
    assert copy([(P[0] + 4, 4096, 4096)]) == _l.KDA_ERR_MISALIGNED
    assert copy([(P[0], 4080, 4096)]) == _l.KDA_ERR_INVALID_ARG  # stride below the page
    assert copy([(P[0], 1 << 32, 1 << 32)]) == _l.KDA_ERR_INVALID_ARG
    assert copy([(None, 4096, 4096)]) == _l.KDA_ERR_INVALID_ARG and b"NULL" in L.kda_last_error()
    assert copy([good, (P[0] + 4096, 4096, 4096)]) == _l.KDA_ERR_ALIAS
    assert copy([good], pairs=P[0] + 64) == _l.KDA_ERR_ALIAS
    assert copy([good], pairs=None) == _l.KDA_ERR_INVALID_ARG
    assert copy([good], n_pairs=-1) == _l.KDA_ERR_INVALID_ARG
    assert L.kda_pages_copy(None, None, None, 1, 8, P[9], 4, None) == _l.KDA_ERR_INVALID_ARG

    def reorder(rows, parents=P[9], B=2, K=4):
        base, _, size = _pools(*rows)
        return L.kda_beam_reorder(base, size, len(rows), parents, B, K, None)

    assert reorder([good], K=65) == _l.KDA_ERR_INVALID_ARG and b"K <= 64" in L.kda_last_error()
    assert reorder([good], B=-1) == _l.KDA_ERR_INVALID_ARG
    assert reorder([good], parents=None) == _l.KDA_ERR_INVALID_ARG
    assert reorder([good], parents=P[0] + 256) == _l.KDA_ERR_ALIAS
    assert reorder([(P[0], 0, 40)]) == _l.KDA_ERR_MISALIGNED
    assert reorder([good, (P[0] + 4096 * 7, 0, 4096)]) == _l.KDA_ERR_ALIAS


def test_workspace_sizes():
    _l, L = _lib()
    bad = 2 ** 64 - 1
    assert L.kda_cache_workspace_size(-1, 8) == bad and L.kda_cache_workspace_size(4, 1 << 24) == bad
    assert L.kda_cache_workspace_size(4, 100000) % 256 == 0
    assert L.kda_beam_select_workspace(1, 0, 10, 1) == bad and L.kda_beam_select_workspace(1, 2, 10, 21) == bad
    assert L.kda_beam_select_workspace(0, 1, 1, 1) == 0
    assert L.kda_paged_decode_workspace(1, 6, 4, 128, 1, 100, 0, 0) == bad
    assert L.kda_paged_decode_workspace(1, 8, 4, 100, 1, 100, 0, 0) == bad
    assert L.kda_paged_decode_workspace(0, 8, 4, 128, 1, 100, 0, 0) == 0


def test_page_table_validator():
    _l, L = _lib()

    def valid(table, lengths, page=16, n_pages=5, most=0):
        t = np.ascontiguousarray(table, dtype=np.int32)
        n = np.ascontiguousarray(lengths, dtype=np.int32)
        return L.kda_validate_page_table(t.ctypes.data, t.shape[1], n.ctypes.data, t.shape[0], t.shape[1], page,
                                         n_pages, most)

    assert valid([[0, 4, -1], [3, -1, -1]], [32, 7]) == 0
    assert valid([[0, 4, -1], [3, -1, -1]], [49, 7]) == _l.KDA_ERR_INVALID_ARG and b"lengths[0]" in L.kda_last_error()
    assert valid([[0, 4, -1], [3, -1, -1]], [32, -1]) == _l.KDA_ERR_INVALID_ARG
    assert valid([[0, 5, -1], [3, -1, -1]], [32, 7]) == _l.KDA_ERR_INVALID_ARG and b"[0, 1]" in L.kda_last_error()
    assert valid([[0, 4, -1], [-2, -1, -1]], [32, 7]) == _l.KDA_ERR_INVALID_ARG
    assert valid([[0, 4, -1], [3, -1, -1]], [32, 7], most=31) == _l.KDA_ERR_INVALID_ARG


def test_binding_refuses_host_and_misshapen_tensors():
    import gated_delta_rule_75_amd as kda

    t = torch.zeros(2, 4, dtype=torch.int32)
    n = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 4, 64)
    pages = torch.zeros(3, 4, 16, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.cache_append(x, x, pages, pages, t, n)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.paged_decode(x, pages, pages, t, n)
    with pytest.raises(ValueError, match="unsupported dtype"):
        kda.paged_decode(x.half(), pages, pages, t, n)
    with pytest.raises(TypeError, match="torch.Tensor"):
        kda.paged_decode([1, 2], pages, pages, t, n)
    for call in (lambda: kda.cache_fork(t, n, n, n), lambda: kda.cache_free(t, n, n, n),
                 lambda: kda.cache_reserve(t, n, n, n, 16), lambda: kda.cache_compact(t, n),
                 lambda: kda.pages_copy([pages], t[:, :2]), lambda: kda.beam_select(x, n.float()),
                 lambda: kda.beam_reorder([x], t)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    from gated_delta_rule_75_amd.serving import _rows

    assert _rows(torch.zeros(4, 8, 64)[:, :4], "x", torch.Size((4, 4, 64))) == 512  # rows of a wider tensor
    assert _rows(torch.zeros(1, 4, 64), "x", torch.Size((1, 4, 64))) == 256
    with pytest.raises(ValueError, match="contiguous"):
        _rows(torch.zeros(4, 64, 4).transpose(1, 2), "x", torch.Size((4, 4, 64)))
    with pytest.raises(ValueError, match="shape"):
        _rows(x, "x", torch.Size((2, 4, 32)))


@pytest.mark.parametrize("what", ["torch", "python"])
def test_a_marshalling_module_built_for_another_torch_or_python_is_not_used(monkeypatch, what):
    """The module reads torch's and CPython's structures: one that was built for others is left aside with a
    warning, and the calls are marshalled in Python."""
    import sys

    _lib()
    from gated_delta_rule_75_amd import build, serving

    if not os.path.exists(build.MARSHAL):
        pytest.skip("marshalling module not built")
    monkeypatch.setattr(serving, "_LIB", None)
    monkeypatch.setattr(serving, "_M", None)
    serving._lib_()
    assert serving._M is not None
    monkeypatch.setattr(serving, "_LIB", None)
    monkeypatch.setattr(serving, "_M", None)
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "1.2.3")
    else:
        monkeypatch.setattr(sys, "version_info", (2, 7, 0))
    with pytest.warns(RuntimeWarning, match=what):
        assert serving._lib_() is not None
    assert serving._M is None


@pytest.mark.parametrize("missing", ["compiler", "headers"])
def test_the_build_goes_on_without_the_marshalling_module(monkeypatch, tmp_path, capsys, missing):
    """Without g++ or the headers the library is complete; a module of an earlier build is taken away."""
    import sysconfig

    from gated_delta_rule_75_amd import build

    old = tmp_path / "_kda_marshal.so"
    old.write_bytes(b"old")
    monkeypatch.setattr(build, "MARSHAL", str(old))
    if missing == "compiler":
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    else:
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build_marshal() is None
    assert not old.exists() and "not built" in capsys.readouterr().out
