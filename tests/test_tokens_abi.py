"""Token table, cross entropy and routing: what the C ABI and the binding
refuse, on the host (no GPU; nothing here launches a kernel)."""

import ctypes

import pytest
import torch

import lsh_bucketed_sparse_b200 as lsh
from lsh_bucketed_sparse_b200 import build as B

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
OFF8 = ctypes.c_void_p((1 << 20) + 8)
OFF2 = ctypes.c_void_p((1 << 20) + 2)
OFF16 = ctypes.c_void_p((1 << 20) + 16)
STREAM = ctypes.c_void_p(0)
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    B.build()
    return lsh.lib()


def table(**kw):
    a = dict(rows=100, vocab=1000, d_model=64)
    a.update(kw)
    return lsh.make_table_shape(**a)


def route(**kw):
    a = dict(tokens=100, top_k=2, n_experts=8, d_model=64)
    a.update(kw)
    return lsh.make_route_shape(**a)


def ref(s):
    return None if s is None else ctypes.byref(s)


def embed(L, s, tokens=FAKE, tab=FAKE, out=FAKE):
    return L.lsh_attn_embed(ref(s), tokens, tab, out, STREAM)


def embed_bwd(L, s, tokens=FAKE, dout=FAKE, init=None, dtable=FAKE, ws=FAKE, n=BIG):
    return L.lsh_attn_embed_backward(ref(s), tokens, dout, init, dtable, ws, n, STREAM)


def xent(L, s, x=FAKE, tab=FAKE, targets=FAKE, loss=FAKE, lse=FAKE, ws=FAKE, n=BIG):
    return L.lsh_attn_xent(ref(s), x, tab, targets, loss, lse, ws, n, STREAM)


def xent_bwd(L, s, x=FAKE, tab=FAKE, targets=FAKE, lse=FAKE, dloss=FAKE, dx=FAKE, dtable=FAKE,
             ws=FAKE, n=BIG):
    return L.lsh_attn_xent_backward(ref(s), x, tab, targets, lse, dloss, dx, dtable, ws, n, STREAM)


def sort(L, s, experts=FAKE, perm=FAKE, undo=FAKE, offsets=FAKE, ws=FAKE, n=BIG):
    return L.lsh_attn_route_sort(ref(s), experts, perm, undo, offsets, ws, n, STREAM)


def gather(L, s, x=FAKE, undo=FAKE, offsets=FAKE, xs=FAKE):
    return L.lsh_attn_route_gather(ref(s), x, undo, offsets, xs, STREAM)


def gather_bwd(L, s, dxs=FAKE, undo=FAKE, offsets=FAKE, dx=FAKE):
    return L.lsh_attn_route_gather_backward(ref(s), dxs, undo, offsets, dx, STREAM)


def combine(L, s, y=FAKE, weights=FAKE, undo=FAKE, offsets=FAKE, out=FAKE):
    return L.lsh_attn_route_combine(ref(s), y, weights, undo, offsets, out, STREAM)


def combine_bwd(L, s, dout=FAKE, y=FAKE, weights=FAKE, undo=FAKE, offsets=FAKE, dy=FAKE, dw=FAKE):
    return L.lsh_attn_route_combine_backward(ref(s), dout, y, weights, undo, offsets, dy, dw,
                                             STREAM)


TABLE_CALLS = [embed, embed_bwd, xent, xent_bwd]
ROUTE_CALLS = [sort, gather, gather_bwd, combine, combine_bwd]


@pytest.mark.parametrize("call", TABLE_CALLS)
@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=(1 << 30) + 1), dict(vocab=0), dict(vocab=(1 << 20) + 1),
    dict(d_model=0), dict(d_model=12), dict(d_model=16392), dict(d_model=-8), dict(dtype=2),
    dict(index_type=2), dict(scale=float("inf")), dict(scale=float("nan"))])
def test_bad_table_shape_is_refused(L, call, kw):
    assert call(L, table(**kw)) == 1
    assert L.lsh_attn_last_error()


@pytest.mark.parametrize("call", ROUTE_CALLS)
@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(tokens=(1 << 29) + 1), dict(top_k=0), dict(top_k=65),
    dict(n_experts=0), dict(n_experts=1024), dict(d_model=4), dict(dtype=5), dict(index_type=-1)])
def test_bad_route_shape_is_refused(L, call, kw):
    assert call(L, route(**kw)) == 1
    assert L.lsh_attn_last_error()


def test_unknown_flags_and_missing_shapes(L):
    for s, calls in ((table(), TABLE_CALLS), (route(), ROUTE_CALLS)):
        s.flags = 2
        for call in calls:
            assert call(L, s) == 1
            assert call(L, None) == 1


@pytest.mark.parametrize("call,names", [
    (embed, ["tab", "out"]), (embed_bwd, ["dout", "dtable"]), (xent, ["x", "tab"]),
    (xent_bwd, ["x", "tab", "dx", "dtable"])])
def test_rows_of_the_table_are_needed_and_aligned(L, call, names):
    for name in names:
        for bad in (None, OFF8):
            assert call(L, table(), **{name: bad}) == 1, (name, bad)
    assert embed_bwd(L, table(), init=OFF8) == 1


@pytest.mark.parametrize("call,names", [
    (gather, ["x", "xs"]), (gather_bwd, ["dxs", "dx"]), (combine, ["y", "out"]),
    (combine_bwd, ["dout", "y", "dy"])])
def test_routed_rows_are_needed_and_aligned(L, call, names):
    for name in names:
        for bad in (None, OFF8):
            assert call(L, route(), **{name: bad}) == 1, (name, bad)


@pytest.mark.parametrize("call,shape,names", [
    (embed, table, ["tokens"]), (embed_bwd, table, ["tokens"]),
    (xent, table, ["targets", "loss", "lse"]), (xent_bwd, table, ["targets", "lse", "dloss"]),
    (sort, route, ["experts", "perm", "undo", "offsets"]), (gather, route, ["undo", "offsets"]),
    (gather_bwd, route, ["undo", "offsets"]), (combine, route, ["weights", "undo", "offsets"]),
    (combine_bwd, route, ["weights", "undo", "offsets", "dw"])])
def test_vectors_are_needed_and_aligned_to_their_values(L, call, shape, names):
    for name in names:
        for bad in (None, OFF2):
            assert call(L, shape(), **{name: bad}) == 1, (name, bad)


@pytest.mark.parametrize("call,shape,query", [
    (embed_bwd, table, "lsh_attn_embed_backward_workspace_size"),
    (xent, table, "lsh_attn_xent_workspace_size"),
    (xent_bwd, table, "lsh_attn_xent_backward_workspace_size"),
    (sort, route, "lsh_attn_route_sort_workspace_size")])
@pytest.mark.parametrize("dtype", [lsh.BF16, lsh.F32])
def test_workspaces_are_sized_and_checked(L, call, shape, query, dtype):
    # (up to 16384 entries are sorted by expert without a workspace)
    s, n = shape(dtype=dtype, **({"tokens": 40000} if shape is route else {})), ctypes.c_size_t()
    assert getattr(L, query)(ref(s), ctypes.byref(n)) == 0
    assert n.value > 0
    assert call(L, s, n=n.value - 1) == 3
    assert b"workspace" in L.lsh_attn_last_error()
    assert call(L, s, ws=None) == 1
    assert call(L, s, ws=OFF16) == 1          # not 256-byte aligned
    assert getattr(L, query)(ref(s), None) == 1
    assert getattr(L, query)(None, ctypes.byref(n)) == 1
    assert getattr(lsh, query)(s) == n.value


def test_workspace_grows_with_the_sizes_that_it_serves(L):
    # monotone over rows, so that one workspace for the longest batch serves all
    for query, shape, key in (("lsh_attn_embed_backward_workspace_size", table, "rows"),
                              ("lsh_attn_route_sort_workspace_size", route, "tokens")):
        sizes = [getattr(lsh, query)(shape(**{key: n})) for n in (0, 1, 100, 5000, 100000)]
        assert sizes == sorted(sizes)


def test_no_rows_need_no_buffers(L):
    for call, s in ((gather, route(tokens=0)),):
        assert call(L, s, x=None, undo=None, xs=None) == 0
    assert embed(L, table(rows=0), tokens=None, out=None) == 0
    assert xent(L, table(rows=0), x=None, targets=None, loss=None, lse=None, ws=None, n=0) == 0
    assert gather_bwd(L, route(tokens=0), dxs=None, undo=None, dx=None) == 0
    assert combine(L, route(tokens=0), y=None, weights=None, undo=None, out=None) == 0
    assert combine_bwd(L, route(tokens=0), dout=None, y=None, weights=None, undo=None, dy=None,
                       dw=None) == 0
    # the gradient of an empty batch added in place is what was there
    assert embed_bwd(L, table(rows=0), tokens=None, dout=None, init=FAKE, dtable=FAKE, ws=None,
                     n=0) == 0


def test_binding_refuses_host_tensors_and_wrong_ranks():
    t, w = torch.zeros(4, dtype=torch.int64), torch.zeros(8, 16)
    calls = [lambda: lsh.lsh_attn_embed(t, w),
             lambda: lsh.lsh_attn_embed_backward(t, torch.zeros(4, 16), 8),
             lambda: lsh.lsh_attn_xent(torch.zeros(4, 16), w, t),
             lambda: lsh.lsh_attn_xent_backward(torch.zeros(4, 16), w, t, torch.zeros(4),
                                                torch.zeros(4)),
             lambda: lsh.lsh_attn_route_sort(t[:, None], 4),
             lambda: lsh.lsh_attn_route_gather(w, t[:, None].int(), t.int()),
             lambda: lsh.lsh_attn_route_combine(w, w, t[:, None].int(), t.int())]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("wide", [(1 << 32) + 8, -(1 << 32) + 8, 1 << 31])
@pytest.mark.parametrize("make,names", [
    (lsh.make_table_shape, ("rows", "vocab", "d_model")),
    (lsh.make_route_shape, ("tokens", "top_k", "n_experts", "d_model"))])
def test_sizes_beyond_32_bits_do_not_wrap(make, names, wide):
    # the sizes of the C structure are 32 bits wide, but for the first
    for name in names[1:]:
        sizes = dict.fromkeys(names, 8)
        assert getattr(make(**sizes), name) == 8
        sizes[name] = wide
        with pytest.raises(ValueError, match=f"{name}={wide}"):
            make(**sizes)


def test_an_output_may_not_lie_over_an_input():
    # (the kernels read their inputs while others of their threads write)
    buf = torch.zeros(64)
    a, b, c = buf[:16], buf[16:32], buf[8:24]
    lsh._apart(a, "out", x=b, init=None, undo=buf[32:])
    lsh._apart(buf[:0], "out", x=buf)
    lsh._apart(a, "out", x=buf[3:3])
    for out, other in ((a, a), (a, c), (c, b), (buf, c), (c, buf)):
        with pytest.raises(ValueError, match="out lies over dxs"):
            lsh._apart(out, "out", x=b[:0], dxs=other)


def test_binding_index_types():
    with pytest.raises(TypeError, match="int32 or int64"):
        lsh._index_code(torch.zeros(2, dtype=torch.int16), "tokens")
    assert lsh._index_code(torch.zeros(2, dtype=torch.int32), "t") == lsh.I32
    assert lsh._index_code(torch.zeros(2, dtype=torch.int64), "t") == lsh.I64
