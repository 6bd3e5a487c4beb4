"""Refusals of include/fs_attention.h: bad arguments are reported on the host,
before any device is looked at (no compute calls, so they run without a GPU)."""
import ctypes

import pytest

from streaming_sinkhorn_solver_amd import binding
from streaming_sinkhorn_solver_amd.binding import AttentionDesc, QkNormDesc, Rows


@pytest.fixture(scope="module")
def lib():
    return binding.load()


Q, K, V, O, LSE, WS = (x << 20 for x in (1, 2, 3, 4, 5, 6))
DO, DQ, DK, DV, DB = (x << 20 for x in (8, 9, 10, 11, 12))


def desc(**kw):
    a = AttentionDesc(1, 2, 5, 7, 4, 2, 64, 64, 0.125)
    for x, y in kw.items():
        if x == "edges":
            a.edges = (ctypes.c_int32 * max(len(y), 1))(*y)
            a.n_edges = len(y)
        else:
            setattr(a, x, y)
    return a


def rows(p, n, h, w):
    return Rows(p, n * h * w, h * w, w)


def forward(lib, a, q=None, k=None, v=None, o=None, lse=LSE, ws=WS, size=1 << 20):
    return lib.fs_attention_forward(ctypes.byref(a), q or rows(Q, 5, 4, 64), k or rows(K, 7, 2, 64),
                                    v or rows(V, 7, 2, 64), o or rows(O, 5, 4, 64), lse, ws, size,
                                    None)


def backward(lib, a, dq=None, dk=None, dv=None, db=None, lse=LSE, ws=WS, size=1 << 20):
    return lib.fs_attention_backward(ctypes.byref(a), rows(Q, 5, 4, 64), rows(K, 7, 2, 64),
                                     rows(V, 7, 2, 64), rows(O, 5, 4, 64), lse, rows(DO, 5, 4, 64),
                                     None, dq or rows(DQ, 5, 4, 64), dk or rows(DK, 7, 2, 64),
                                     dv or rows(DV, 7, 2, 64), db, ws, size, None)


BAD = [
    (dict(dtype=3), "fs_dtype"), (dict(batch=-1), "batch"), (dict(n=(1 << 28) + 1), "2^28"),
    (dict(heads=3), "multiple"), (dict(kv_heads=0), "multiple"), (dict(d=0), "d and dv"),
    (dict(dv=257), "d and dv"), (dict(dtype=0, d=129), "d and dv"), (dict(scale=0.0), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(offset=-(1 << 30)), "offset"),
    (dict(key_mask=64, key_mask_stride=3), "key_mask_stride"),
    (dict(bias=256, edges=[0]), "edges"), (dict(bias=256, edges=[3, 2]), "edges"),
    (dict(bias=256, edges=[1025]), "edges"), (dict(bias=256, edges=[1] * 256), "n_edges"),
    (dict(batch=1 << 20, n=1 << 20), "2^31"),
]


@pytest.mark.parametrize("kw,word", BAD, ids=lambda x: str(x))
def test_bad_descriptions(lib, kw, word):
    a = desc(**kw)
    for call in (forward, backward):
        assert call(lib, a) == binding.FS_ERR_INVALID_ARG
        assert word in binding.fs_last_error()
    assert lib.fs_attention_workspace_bytes(ctypes.byref(a), 0) == 0
    assert lib.fs_attention_workspace_bytes(ctypes.byref(a), 1) == 0


def test_bad_tensors(lib):
    a = desc()
    inv = binding.FS_ERR_INVALID_ARG
    assert forward(lib, a, q=Rows(None, 0, 0, 0)) == inv
    assert forward(lib, a, k=rows(K + 1, 7, 2, 64)) == inv and "aligned" in binding.fs_last_error()
    assert forward(lib, a, v=Rows(V, -1, 128, 64)) == inv and "stride" in binding.fs_last_error()
    # an output whose rows overlap one another, an output on an input
    assert forward(lib, a, o=Rows(O, 1280, 256, 63)) == inv and "overlap" in binding.fs_last_error()
    assert forward(lib, a, o=Rows(O, 0, 256, 64)) == inv
    assert forward(lib, a, o=rows(V, 5, 4, 64)) == inv and "overlaps" in binding.fs_last_error()
    assert forward(lib, a, lse=Q) == inv
    assert forward(lib, a, o=rows(WS, 5, 4, 64)) == inv
    assert forward(lib, desc(bias=O, edges=[1, 2])) == inv
    # inputs may overlap themselves (broadcast); then the workspace is looked at
    assert forward(lib, a, k=Rows(K, 0, 0, 0), ws=WS + 8) == binding.FS_ERR_WORKSPACE
    assert forward(lib, a, ws=None) == binding.FS_ERR_WORKSPACE
    assert forward(lib, a, size=255) == binding.FS_ERR_WORKSPACE
    assert lib.fs_attention_forward(None, *[rows(Q, 5, 4, 64)] * 4, None, WS, 256, None) == inv


def test_bad_gradients(lib):
    a = desc()
    inv = binding.FS_ERR_INVALID_ARG
    assert backward(lib, a, lse=None) == inv
    assert backward(lib, a, db=DB) == inv and "bias" in binding.fs_last_error()
    assert backward(lib, a, dk=Rows(DK, 0, 128, 64)) == inv and "overlap" in binding.fs_last_error()
    assert backward(lib, a, dq=rows(DO, 5, 4, 64)) == inv
    assert backward(lib, a, dv=rows(DK, 7, 2, 64)) == inv and "same memory" in binding.fs_last_error()
    assert backward(lib, desc(bias=256, edges=[1, 2]), db=DQ) == inv
    need = lib.fs_attention_workspace_bytes(ctypes.byref(a), 1)
    assert backward(lib, a, size=need - 1) == binding.FS_ERR_WORKSPACE


def test_workspace_sizes(lib):
    size = lambda b, **kw: lib.fs_attention_workspace_bytes(ctypes.byref(desc(**kw)), b)
    assert size(0) == 256 and size(0, n=0) == 256 and size(1, m=0) >= 256
    # a token against a long cache is split over workgroups, never n x m
    assert 256 < size(0, n=1, m=1 << 20) < 64 * 2 * 4 * (64 + 2) * 4 + 1024
    # the backward pass keeps two numbers per query row, none per pair
    assert size(1, n=4096, m=4096, batch=8, heads=16, kv_heads=16) < 2 * 8 * 16 * 4096 * 4 + 4096


def test_bucket_edges(lib):
    assert binding.fs_bucket_edges(16, 128) == [1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 23, 32, 46, 64, 91]
    out = (ctypes.c_int32 * 64)()
    for side, far in ((1, 100), (65, 100), (16, 8), (16, 1025)):
        assert lib.fs_bucket_edges(side, far, out) == binding.FS_ERR_INVALID_ARG
    assert lib.fs_bucket_edges(16, 128, None) == binding.FS_ERR_INVALID_ARG
    # every edge is the smallest x with x^r >= first^(r - k) far^k
    for side, far in ((2, 64), (4, 64), (7, 20), (32, 128), (64, 1024), (64, 33)):
        first, rest = side // 2, side - side // 2
        for u, e in enumerate(binding.fs_bucket_edges(side, far), 1):
            if u <= first:
                assert e == u
            else:
                bound = first ** (rest - (u - first)) * far ** (u - first)
                assert e ** rest >= bound > (e - 1) ** rest


def norm_desc(**kw):
    a = QkNormDesc(1, 2, 5, 4, 2, 64, 64, 0, 1e-6, 256, 512, 10)
    for x, y in kw.items():
        setattr(a, x, y)
    return a


def norm(lib, a, q=None, k=None, qo=None, ko=None):
    return lib.fs_qk_norm_rotate(ctypes.byref(a), q or rows(Q, 5, 4, 64), k or rows(K, 5, 2, 64),
                                 None, None, qo or rows(O, 5, 4, 64), ko or rows(V, 5, 2, 64), None)


NORM_BAD = [dict(dtype=-1), dict(n=-1), dict(d=63), dict(d=258), dict(rot=66), dict(rot=3),
            dict(eps=-1.0), dict(eps=float("inf")), dict(cos_table=None), dict(n_pos=0),
            dict(positions=256, positions_stride=4), dict(heads_q=-1),
            dict(batch=1 << 16, n=1 << 15)]


@pytest.mark.parametrize("kw", NORM_BAD, ids=lambda x: str(x))
def test_bad_norms(lib, kw):
    a = norm_desc(**kw)
    assert norm(lib, a) == binding.FS_ERR_INVALID_ARG
    assert lib.fs_qk_norm_workspace_bytes(ctypes.byref(a)) == 0


def test_bad_norm_tensors(lib):
    inv = binding.FS_ERR_INVALID_ARG
    a = norm_desc()
    assert norm(lib, a, qo=rows(Q, 5, 4, 64)) == inv
    assert norm(lib, a, qo=Rows(O, 1280, 256, 32)) == inv
    assert norm(lib, a, ko=rows(O, 5, 2, 64)) == inv
    assert norm(lib, a, k=Rows(None, 0, 0, 0)) == inv
    r = rows(Q, 5, 4, 64), rows(K, 5, 2, 64)
    g = rows(DO, 5, 4, 64), rows(DB, 5, 2, 64)
    d = rows(DQ, 5, 4, 64), rows(DK, 5, 2, 64)
    need = lib.fs_qk_norm_workspace_bytes(ctypes.byref(a))
    back = lambda *d, gw=None, size=need: lib.fs_qk_norm_rotate_backward(
        ctypes.byref(a), *r, None, None, *g, *d, gw, None, WS, size, None)
    assert back(*d, size=need - 1) == binding.FS_ERR_WORKSPACE
    assert back(d[0], rows(DQ, 5, 2, 64)) == inv
    assert back(*d, gw=DQ) == inv and back(g[0], d[1]) == inv


@pytest.mark.parametrize("kw", [dict(batch=1 << 18, heads=32, kv_heads=32, n=1),    # few rows
                                dict(batch=1 << 18, heads=64, kv_heads=2, n=100),   # many rows
                                dict(batch=1 << 23, heads=2, kv_heads=2, n=1, m=100)])
def test_more_threads_than_a_launch_has(lib, kw):
    a = desc(**kw)
    for call in (forward, backward):
        assert call(lib, a) == binding.FS_ERR_INVALID_ARG
        assert "2^32 threads" in binding.fs_last_error()
    assert lib.fs_attention_workspace_bytes(ctypes.byref(a), 0) == 0
    # half of it is fine
    a.batch //= 4
    assert lib.fs_attention_workspace_bytes(ctypes.byref(a), 0) > 0


def test_numbers_beyond_32_bits():
    """The binding refuses what would reach the library as another number."""
    import torch

    one = torch.zeros(1, 1, 1, 32)
    long = one.expand(1, (1 << 32) + 7, 1, 32)
    size = binding.fs_attention_workspace_bytes
    assert size(one, one, one) == 256
    for args, kw in (((long, one, one), {}), ((one, long, long), {}),
                     ((one, one, one), {"edges": [1, (1 << 32) + 2]})):
        with pytest.raises(ValueError, match="32 bits"):
            size(*args, **kw)
    with pytest.raises(ValueError, match="32 bits"):
        binding.fs_bucket_edges((1 << 32) + 16, 128)
    with pytest.raises(ValueError, match="32 bits"):
        binding.fs_bucket_edges(16, (1 << 32) + 128)
    with pytest.raises(binding.FsError):
        binding.fs_bucket_edges(1 << 30, 128)


def test_scales_that_leave_the_range(lib):
    """A finite scale that times log2 e is not finite would make every score NaN."""
    for scale, ok in ((1e-38, True), (2e38, True), (3e38, False), (float("inf"), False)):
        a = desc(scale=scale)
        assert (lib.fs_attention_workspace_bytes(ctypes.byref(a), 0) > 0) == ok
        if not ok:
            assert forward(lib, a) == binding.FS_ERR_INVALID_ARG and "scale" in binding.fs_last_error()
