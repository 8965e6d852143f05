"""Token table, cross entropy and routing on the GPU against float64 torch
(tokens_ref.py has the formulas and the bounds)."""

import ctypes
import math

import pytest
import torch

import lsh_bucketed_sparse_b200 as lsh
import tokens_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dtype)


def make_tokens(g, n, vocab, index, skew=0.0, holes=0.0):
    """Ids in [0, vocab); a share `skew` is one id, a share `holes` outside."""
    t = torch.randint(0, vocab, (n,), device=DEV, generator=g)
    u = torch.rand(n, device=DEV, generator=g)
    t = torch.where(u < skew, torch.full_like(t, vocab // 2), t)
    out = torch.where(torch.rand(n, device=DEV, generator=g) < 0.5, torch.full_like(t, -1),
                      torch.full_like(t, vocab))
    return torch.where(u > 1 - holes, out, t).to(index)


# ---- token table ---------------------------------------------------------------
EMBED = [  # rows, vocab, d, dtype, index, scale
    (0, 16, 8, BF16, torch.int64, 1.0),
    (1, 1, 8, F32, torch.int32, 2.0),
    (8, 1000, 512, BF16, torch.int64, math.sqrt(512)),
    (257, 50, 24, BF16, torch.int32, 0.5),
    (1000, 33, 1032, F32, torch.int64, 1.0),
    (3, 20, 16384, BF16, torch.int64, 1.0),
]


@pytest.mark.parametrize("n,vocab,d,dtype,index,scale", EMBED)
def test_embed(n, vocab, d, dtype, index, scale):
    g = gen(n + vocab)
    tok = make_tokens(g, n, vocab, index, holes=0.2)
    table = randn(g, vocab, d, dtype=dtype)
    R.check("out", lsh.lsh_attn_embed(tok, table, scale=scale), R.embed(tok, table, scale))


EMBED_BWD = [  # rows, vocab, d, dtype, index, skew, holes
    (0, 16, 8, BF16, torch.int64, 0, 0),
    (1, 1, 8, F32, torch.int32, 0, 0),
    (1, 300, 16, BF16, torch.int64, 0, 1.0),       # nothing but padding
    (64, 4, 40, BF16, torch.int32, 1.0, 0),        # one run as long as a chunk
    (65, 4, 40, F32, torch.int64, 1.0, 0),         # one longer
    (1000, 7, 72, BF16, torch.int64, 0, 0.1),
    (2047, 1023, 136, F32, torch.int32, 0.3, 0.1),
    (2048, 1024, 8, BF16, torch.int64, 0.5, 0),    # the first size of two digits
    (6000, 50021, 24, F32, torch.int64, 0.2, 0.2),
    (5000, 1 << 20, 8, BF16, torch.int32, 0.1, 0.1),
    (20000, 300, 264, BF16, torch.int64, 0.9, 0),
    (300, 10, 16384, F32, torch.int64, 0.5, 0),
    (257, 3, 1032, BF16, torch.int64, 0.9, 0),
    (16384, 40000, 8, BF16, torch.int64, 0.1, 0.1),  # the most of a cluster
    (16385, 1 << 20, 8, BF16, torch.int32, 0.1, 0.1),  # one more than it takes
    (65537, 200, 16, BF16, torch.int32, 0.2, 0.1),
    (70001, 40000, 8, F32, torch.int32, 0.1, 0.1),
    (140001, 5000, 8, F32, torch.int64, 0.3, 0.1),   # counts scanned by a kernel of their own
]


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("n,vocab,d,dtype,index,skew,holes", EMBED_BWD)
def test_embed_backward(n, vocab, d, dtype, index, skew, holes, into):
    g = gen(n * 3 + vocab)
    tok = make_tokens(g, n, vocab, index, skew, holes)
    dout = randn(g, n, d, dtype=dtype)
    init = randn(g, vocab, d, dtype=dtype) if into else None
    want = R.embed_backward(tok, dout, vocab, 0.75, init)
    got = lsh.lsh_attn_embed_backward(tok, dout, vocab, scale=0.75, init=init)
    R.check("dtable", got, want)
    # the same bits again, and added in place
    again = lsh.lsh_attn_embed_backward(tok, dout, vocab, scale=0.75, init=init,
                                        out=init if into else None)
    assert torch.equal(got, again)


def test_embed_takes_any_leading_shape_and_a_slice_of_tokens():
    g = gen(5)
    ids = torch.randint(0, 40, (2 * 3 * 5 + 1,), device=DEV, generator=g)
    tok, table = ids[1:].view(2, 3, 5), randn(g, 40, 16)     # 8 bytes off a 16-byte address
    out = lsh.lsh_attn_embed(tok, table)
    assert out.shape == (2, 3, 5, 16)
    assert torch.equal(out, table[tok])
    dt = lsh.lsh_attn_embed_backward(tok, out, 40)
    R.check("dtable", dt, R.embed_backward(tok, out, 40, 1.0))


def test_tokens_far_outside_the_table_are_padding():
    # int64 ids whose low 32 bits are a valid id
    tok = torch.tensor([3, 3 + (1 << 32), -(1 << 40) + 3, (1 << 62), 7], device=DEV)
    table = randn(gen(1), 8, 8)
    want = table[torch.tensor([3, 0, 0, 0, 7], device=DEV)]
    want[1:4] = 0
    assert torch.equal(lsh.lsh_attn_embed(tok, table), want)
    dt = lsh.lsh_attn_embed_backward(tok, torch.ones(5, 8, device=DEV), 8)
    assert dt.sum() == 16 and dt[3, 0] == 1 and dt[7, 0] == 1
    loss, lse = lsh.lsh_attn_xent(want, table, tok)
    assert torch.equal(loss == 0, torch.tensor([0, 1, 1, 1, 0], device=DEV).bool())
    assert bool(torch.isfinite(lse).all())


# ---- cross entropy ---------------------------------------------------------------
XENT = [  # rows, vocab, d, dtype, index, scale, holes
    (1, 1, 8, BF16, torch.int64, 1.0, 0),
    (1, 2, 8, F32, torch.int32, 1.0, 0),
    (5, 1000, 64, BF16, torch.int32, 1.0, 0),
    (128, 256, 64, BF16, torch.int64, 1.0, 0),
    (129, 257, 72, BF16, torch.int64, 0.125, 0.3),
    (256, 255, 128, F32, torch.int32, 1.0, 0),
    (255, 513, 520, BF16, torch.int32, 1.0, 0.1),
    (300, 777, 136, F32, torch.int64, -0.5, 0.5),
    (513, 2049, 264, BF16, torch.int64, 1.0, 1.0),  # nothing but padding
    (700, 5000, 64, BF16, torch.int64, 1.0, 0.05),
    (1025, 3001, 40, F32, torch.int64, 1.0, 0.1),
    (33, 20011, 24, BF16, torch.int64, 1.0, 0),
    (40, 300, 64, BF16, torch.int64, 0.0, 0.1),     # every word as likely
    (3, 70, 16384, BF16, torch.int64, 1.0, 0),
    (3, 70, 16384, F32, torch.int32, 1.0, 0),
    (9, 1 << 20, 16, BF16, torch.int64, 1.0, 0),
    (2, 100003, 72, F32, torch.int64, 1.0, 0),
    (4, 3001, 136, F32, torch.int64, 1.0, 0.3),
    (5, 31, 8, F32, torch.int32, 2.0, 0),
    (8, 2001, 1032, F32, torch.int64, 1.0, 0.3),
    (9, 777, 520, F32, torch.int32, 1.0, 0.2),
    (16, 5003, 264, F32, torch.int64, -1.0, 0.1),
    (17, 300, 128, F32, torch.int64, 1.0, 1.0),
    (32, 1111, 1600, F32, torch.int64, 1.0, 0.2),
    (33, 1111, 264, F32, torch.int64, 1.0, 0.2),
]


def make_xent(n, vocab, d, dtype, index, holes, seed=0):
    """Rows that lean to their targets by 0 to 10, as a trained model's."""
    g = gen(n * 7 + vocab + seed)
    t = make_tokens(g, n, vocab, index, 0.1, holes)
    table = randn(g, vocab, d, scale=d ** -0.5)
    lift = 10 * torch.rand(n, 1, device=DEV, generator=g)
    x = randn(g, n, d) + lift * table[t.long().clamp(0, vocab - 1)]
    return x.to(dtype), table.to(dtype), t, randn(g, n)


@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("n,vocab,d,dtype,index,scale,holes", XENT)
def test_xent(n, vocab, d, dtype, index, scale, holes, portable):
    x, table, t, dloss = make_xent(n, vocab, d, dtype, index, holes)
    loss, lse = lsh.lsh_attn_xent(x, table, t, scale=scale, portable=portable)
    want_loss, want_lse = R.xent(x, table, t, scale)
    R.check("lse", lse, want_lse)
    R.check("loss", loss, want_loss)
    dx, dw = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss, scale=scale, portable=portable)
    lsh.lsh_attn_device_check()
    want_dx, want_dw = R.xent_backward(x, table, t, dloss, scale,
                                       BF16 if dtype == BF16 and not portable else None)
    R.check("dx", dx, want_dx)
    R.check("dtable", dw, want_dw)
    # the same inputs give the same bits
    again = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss, scale=scale, portable=portable)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [1.0, -0.5])
@pytest.mark.parametrize("n,vocab", [(1, 700), (30, 257), (33, 1000), (128, 300), (129, 300), (700, 65)])
def test_xent_of_sure_rows_keeps_its_digits(n, vocab, scale, dtype, portable):
    # The target's logit is 8 to 40 above the others: the loss is exp(-8) to
    # exp(-40), and its relative error is the logits' absolute one.
    d = 16
    g = gen(n + vocab)
    t = torch.randint(0, vocab, (n,), device=DEV, generator=g)
    table = randn(g, vocab, d, dtype=dtype)
    lift = 8 + 32 * torch.rand(n, 1, device=DEV, generator=g)
    own = table[t].float()
    x = (own * lift / (own.square().sum(1, keepdim=True) * scale)).to(dtype)
    loss, lse = lsh.lsh_attn_xent(x, table, t, scale=scale, portable=portable)
    xd, wd = x.double(), table.double()
    z = xd @ wd.T * scale
    zt = z.gather(1, t[:, None])
    rest = (z - zt).scatter(1, t[:, None], float("-inf"))
    want = torch.logsumexp(torch.cat([rest, torch.zeros_like(zt)], 1), 1)
    small = torch.logsumexp(rest, 1)
    want = torch.where(small < -20, small.exp() * (1 - small.exp() / 2), want)
    # a logit of 16 products: at most 16 + 6 roundings (planes, additions, the
    # scale), each cut off (2^-23) of what is summed; two logits; the exponentials,
    # sums and the logarithm: 64 more half steps
    size = (xd.abs() @ wd.abs().T).amax(1) * abs(scale)
    bound = want * (2 * 22 * 2.0 ** -23 * size + 64 * 2.0 ** -24) + 2.0 ** -140
    R.check("loss", loss, (want, bound))
    R.check("lse", lse, (want + zt[:, 0], 44 * 2.0 ** -23 * size + 2.0 ** -22 * zt[:, 0].abs() + 2.0 ** -22))


@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,vocab", [(2, 40), (40, 300), (200, 777)])
def test_xent_without_scale(n, vocab, dtype, portable):
    # all logits are 0: log V, in a handful of float32 steps of at most 4 half ones
    x, table, t, dloss = make_xent(n, vocab, 32, dtype, torch.int32, 0.2)
    live = (t >= 0) & (t < vocab)
    loss, lse = lsh.lsh_attn_xent(x, table, t, scale=0.0, portable=portable)
    want = torch.full((n,), float(vocab), device=DEV, dtype=torch.float64).log()
    R.check("lse", lse, (want, want * 2.0 ** -20))
    R.check("loss", loss, (want * live, want * 2.0 ** -20))
    dx, dw = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss, scale=0.0, portable=portable)
    assert not bool(dx.any()) and not bool(dw.any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("valid", [0, 1, 31, 32, 63, 64, 65, 97, 128, 255, 256, 257, 449, 600])
def test_xent_backward_of_as_many_rows(valid, dtype):
    # the rows with a target are gathered; what lies behind them is not read
    x, table, t, dloss = make_xent(600, 333, 72, dtype, torch.int64, 0)
    keep = torch.randperm(600, device=DEV, generator=gen(valid))[:valid]
    targets = torch.full_like(t, -1)
    targets[keep] = t[keep]
    loss, lse = lsh.lsh_attn_xent(x, table, targets)
    need = lsh.lsh_attn_xent_backward_workspace_size(
        lsh.make_table_shape(600, 333, 72, dtype))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)    # NaN everywhere
    dx, dw = lsh.lsh_attn_xent_backward(x, table, targets, lse, dloss, workspace=ws)
    want_dx, want_dw = R.xent_backward(x, table, targets, dloss, 1.0,
                                       BF16 if dtype == BF16 else None)
    R.check("dx", dx, want_dx)
    R.check("dtable", dw, want_dw)


@pytest.mark.parametrize("n,vocab,d", [(1, 700, 264), (5, 3001, 520), (64, 333, 72), (100, 2000, 136),
                                       (128, 513, 1024)])
def test_xent_backward_of_few_bf16_rows_rounds_once(n, vocab, d):
    # g is held in 16 bits or more up to 128 rows: the results' own rounding is
    # what shows.  Half a step of bfloat16 (2^-8) of each value, and 2^-14 of the
    # sum of the products' sizes: 2^-17 for g in two planes, 2^-15 for the
    # logits (below 2^6 in size, cut 22 times at 2^-23), the rest for the sums.
    x, table, t, dloss = make_xent(n, vocab, d, BF16, torch.int64, 0.1)
    lse = lsh.lsh_attn_xent(x, table, t)[1]
    dx, dw = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss)
    xd, wd = x.double(), table.double()
    live = (t >= 0) & (t < vocab)
    grad = torch.softmax(xd @ wd.T, 1)
    grad[live.nonzero()[:, 0], t[live].long()] -= 1
    # (p - 1 of a sure target is cut off at p's size)
    size = torch.softmax(xd @ wd.T, 1)
    size[live.nonzero()[:, 0], t[live].long()] += 1
    up = torch.where(live, dloss, torch.zeros_like(dloss)).double()[:, None]
    grad, size = grad * up, size * up.abs()
    for name, got, want, sums in (("dx", dx, grad @ wd, size @ wd.abs()),
                                  ("dtable", dw, grad.T @ xd, size.T @ xd.abs())):
        R.check(name, got, (want, want.abs() * 2.0 ** -8 + sums * 2.0 ** -14 + 1e-30))


@pytest.mark.parametrize("n,vocab,d,holes", [(129, 700, 264, 0), (212, 3162, 104, 0.5),
                                             (251, 4342, 72, 0.5), (258, 863, 136, 0),
                                             (1658, 380, 232, 0.5), (3737, 885, 840, 0.1)])
def test_xent_backward_of_many_bf16_rows_rounds_once(n, vocab, d, holes):
    # g in two bfloat16 planes: half a step of the first leaves 2^-8 of g, half a
    # step of the second 2^-16.  The rest is the float32 path's bound: g from
    # float32 logits, sums of K terms at 2 K steps (twice: two planes), and the
    # result's own rounding.
    x, table, t, dloss = make_xent(n, vocab, d, BF16, torch.int64, holes)
    lse = lsh.lsh_attn_xent(x, table, t)[1]
    dx, dw = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss)
    xd, wd = x.double(), table.double()
    live = (t >= 0) & (t < vocab)
    size = torch.softmax(xd @ wd.T, 1)
    at = live.nonzero()[:, 0]
    size[at, t[live].long()] -= 1
    size = size.abs() * torch.where(live, dloss.abs(), torch.zeros_like(dloss)).double()[:, None]
    want_dx, want_dw = R.xent_backward(x, table, t, dloss, 1.0)
    for name, got, (want, bound), sums, k in (
            ("dx", dx, want_dx, size @ wd.abs(), vocab),
            ("dtable", dw, want_dw, size.T @ xd.abs(), n)):
        more = (2.0 ** -16 + (2 * k + 8) * R.U) * (1 + R.half_step(BF16)) * sums
        R.check(name, got, (want, bound + more))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,valid", [(7, 0), (7, 5), (100, 0), (100, 1), (100, 33), (100, 64), (100, 65),
                                     (128, 127)])
def test_xent_backward_of_few_rows_with_a_target(n, valid, dtype):
    x, table, t, dloss = make_xent(n, 530, 72, dtype, torch.int32, 0)
    keep = torch.randperm(n, device=DEV, generator=gen(valid))[:valid]
    targets = torch.full_like(t, 530)
    targets[keep] = t[keep]
    lse = lsh.lsh_attn_xent(x, table, targets)[1]
    need = lsh.lsh_attn_xent_backward_workspace_size(lsh.make_table_shape(n, 530, 72, dtype))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)    # NaN everywhere
    dx, dw = lsh.lsh_attn_xent_backward(x, table, targets, lse, dloss, workspace=ws)
    want_dx, want_dw = R.xent_backward(x, table, targets, dloss, 1.0,
                                       BF16 if dtype == BF16 else None)
    R.check("dx", dx, want_dx)
    R.check("dtable", dw, want_dw)


@pytest.mark.parametrize("n,vocab,d,dtype", [(20011, 14001, 24, BF16), (9001, 10007, 40, F32)])
def test_xent_backward_in_pieces(n, vocab, d, dtype):
    # more gradient values than one piece of the vocabulary holds
    x, table, t, dloss = make_xent(n, vocab, d, dtype, torch.int64, 0.02)
    lse = lsh.lsh_attn_xent(x, table, t)[1]
    dx, dw = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss)
    want_dx, want_dw = R.xent_backward(x, table, t, dloss, 1.0, BF16 if dtype == BF16 else None)
    R.check("dx", dx, want_dx)
    R.check("dtable", dw, want_dw)
    again = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


PIECES = [  # rows, vocab, d, dtype, bytes of g, pieces, portable
    # tiles of 256 words, rows x 512 bytes each in every plane of g: 2 (bf16), 3 (float32)
    (300, 2100, 72, BF16, 2 * 2 * 300 * 512, 5, False),     # 2 + 2 + 2 + 2 + 1 tiles
    (300, 2049, 264, BF16, 2 * 2 * 300 * 512, 5, False),    # one word in the last piece
    (129, 1100, 136, BF16, 0, 5, False),                    # a tile each
    (100, 2100, 72, BF16, 2 * 2 * 100 * 512, 5, False),     # few rows
    (9001, 1100, 1032, BF16, 0, 5, False),                  # dx in whole sums over a piece
    (300, 2100, 72, F32, 2 * 3 * 300 * 512, 5, False),
    (33, 2049, 520, F32, 2 * 3 * 33 * 512, 5, False),
    (4001, 1100, 1032, F32, 0, 5, False),
    (50, 300, 72, BF16, 50 * 4 * 64, 5, True),              # 64 columns each, the last of 44
    (70, 257, 40, F32, 0, 5, True),
]


@pytest.mark.parametrize("n,vocab,d,dtype,limit,pieces,portable", PIECES)
def test_xent_backward_in_several_pieces(n, vocab, d, dtype, limit, pieces, portable):
    # the last piece is shorter, and has fewer blocks than the first has parts of K
    x, table, t, dloss = make_xent(n, vocab, d, dtype, torch.int64, 0.1)
    t[:3] = torch.tensor([0, vocab - 1, vocab - 2], device=DEV)
    lse = lsh.lsh_attn_xent(x, table, t, scale=0.5, portable=portable)[1]
    whole = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss, scale=0.5, portable=portable)
    lib = lsh.lib()
    before = lib.lsh_attn_test_xent_piece_bytes(limit)
    try:
        launches = lib.lsh_attn_kernel_launches()
        dx, dw = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss, scale=0.5, portable=portable)
        launches = lib.lsh_attn_kernel_launches() - launches
        again = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss, scale=0.5, portable=portable)
    finally:
        assert lib.lsh_attn_test_xent_piece_bytes(before) == limit
    lsh.lsh_attn_device_check()
    # once: order, rows, table planes (float32), dx's rows; or the cleaned rows.
    # A piece: g, dx, dW, and dW's sum where its K is in parts.
    once = 1 if portable else 3 + (dtype == F32)
    assert launches - once in (3 * pieces, 4 * pieces)
    want_dx, want_dw = R.xent_backward(x, table, t, dloss, 0.5, BF16 if dtype == BF16 else None)
    for got in ((dx, dw), whole):
        R.check("dx", got[0], want_dx)
        R.check("dtable", got[1], want_dw)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_xent_of_no_rows(dtype):
    x, table = torch.empty(0, 16, device=DEV, dtype=dtype), randn(gen(0), 9, 16, dtype=dtype)
    t, f = torch.empty(0, device=DEV, dtype=torch.int64), torch.empty(0, device=DEV)
    loss, lse = lsh.lsh_attn_xent(x, table, t)
    assert loss.shape == lse.shape == (0,)
    dx, dw = lsh.lsh_attn_xent_backward(x, table, t, f, f)
    assert dx.shape == (0, 16) and not bool(dw.any())


@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_padding_rows_may_hold_anything(dtype, portable):
    x, table, t, dloss = make_xent(300, 400, 64, dtype, torch.int64, 0.3)
    pad = (t < 0) | (t >= 400)
    assert bool(pad.any())
    bad, up = x.clone(), dloss.clone()
    bad[pad] = float("nan")
    up[pad] = float("inf")
    loss, lse = lsh.lsh_attn_xent(bad, table, t, portable=portable)
    (want, bound), (want_lse, lse_bound) = R.xent(x, table, t, 1.0)
    assert not bool(loss[pad].any())
    R.check("loss", loss[~pad], (want[~pad], bound[~pad]))
    R.check("lse", lse[~pad], (want_lse[~pad], lse_bound[~pad]))
    dx, dw = lsh.lsh_attn_xent_backward(bad, table, t, lse, up, portable=portable)
    assert not bool(dx[pad].any())
    want_dx, want_dw = R.xent_backward(x, table, t, dloss, 1.0,
                                       BF16 if dtype == BF16 and not portable else None)
    R.check("dx", dx[~pad], (want_dx[0][~pad], want_dx[1][~pad]))
    R.check("dtable", dw, want_dw)


@pytest.mark.parametrize("n", [3, 20])
def test_few_rows_of_padding_may_hold_anything(n):
    x, table, t, dloss = make_xent(n, 500, 72, F32, torch.int64, 0)
    t[1::2] = -1
    pad = t < 0
    bad, up = x.clone(), dloss.clone()
    bad[pad], up[pad] = float("nan"), float("inf")
    loss, lse = lsh.lsh_attn_xent(bad, table, t)
    dx, dw = lsh.lsh_attn_xent_backward(bad, table, t, lse, up)
    assert not bool(loss[pad].any()) and not bool(dx[pad].any())
    want_dx, want_dw = R.xent_backward(x, table, t, dloss, 1.0)
    R.check("dx", dx[~pad], (want_dx[0][~pad], want_dx[1][~pad]))
    R.check("dtable", dw, want_dw)


@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [3, 7, 16, 20, 33, 200])
def test_padding_rows_next_to_infinite_words_have_no_gradient(n, dtype, portable):
    x, table, t, dloss = make_xent(n, 300, 72, dtype, torch.int32, 0)
    table[11, 3], table[250, 70] = -float("inf"), float("inf")
    t[1::2] = 300
    lse = lsh.lsh_attn_xent(x, table, t, portable=portable)[1]
    dx, _ = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss, portable=portable)
    assert not bool(dx[1::2].any())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_logits_do_not_overflow(dtype):
    # logits of some +-12000: exp of any of them alone is 0 or infinite
    g = gen(11)
    x, table = randn(g, 130, 64, dtype=dtype, scale=8), randn(g, 300, 64, dtype=dtype, scale=8)
    t = torch.randint(0, 300, (130,), device=DEV, generator=g)
    loss, lse = lsh.lsh_attn_xent(x, table, t, scale=4.0)
    want_loss, want_lse = R.xent(x, table, t, 4.0)
    assert float(want_lse[0].max()) > 5000
    R.check("lse", lse, want_lse)
    R.check("loss", loss, want_loss)
    dx, dw = lsh.lsh_attn_xent_backward(x, table, t, lse, torch.ones(130, device=DEV), scale=4.0)
    assert bool(torch.isfinite(dx.float()).all()) and bool(torch.isfinite(dw.float()).all())


def test_words_at_minus_infinity_take_no_part():
    # a word that is ruled out by a logit of -inf: probability and gradient 0
    g = gen(12)
    x = randn(g, 40, 16).abs()
    table = randn(g, 50, 16)
    table[10:20, 3] = -float("inf")
    t = torch.randint(20, 50, (40,), device=DEV, generator=g)
    loss, lse = lsh.lsh_attn_xent(x, table, t, portable=True)
    keep = torch.cat([torch.arange(10), torch.arange(20, 50)]).to(DEV)
    (want, bound), (want_lse, lse_bound) = R.xent(x, table[keep], t - 10, 1.0)
    R.check("lse", lse, (want_lse, lse_bound))
    R.check("loss", loss, (want, bound))


@pytest.mark.parametrize("n,dtype", [(1, F32), (4, F32), (7, F32), (16, F32), (32, F32),
                                     (1, BF16), (20, BF16), (128, BF16), (129, BF16), (300, BF16)])
def test_words_at_minus_infinity_take_no_part_on_every_path(n, dtype):
    g = gen(14 + n)
    x, table = randn(g, n, 72, dtype=dtype).abs(), randn(g, 700, 72, dtype=dtype, scale=0.1)
    table[10:90, 3] = -float("inf")     # 64 words side by side among them
    table[650, 71] = -float("inf")
    keep = torch.cat([torch.arange(10), torch.arange(90, 650), torch.arange(651, 700)]).to(DEV)
    at = torch.randint(0, keep.numel(), (n,), device=DEV, generator=g)
    loss, lse = lsh.lsh_attn_xent(x, table, keep[at])
    want_loss, want_lse = R.xent(x, table[keep], at, 1.0)
    R.check("lse", lse, want_lse)
    R.check("loss", loss, want_loss)
    dloss = randn(g, n)
    dx, dw = lsh.lsh_attn_xent_backward(x, table, keep[at], lse, dloss)
    _, want_dw = R.xent_backward(x, table[keep], at, dloss, 1.0, BF16 if dtype == BF16 else None)
    R.check("dtable", dw[keep], want_dw)
    assert not bool(dw[10:90].any()) and not bool(dw[650].any())
    # (0 times -inf: these columns alone have no value)
    assert bool(torch.isnan(dx[:, 3]).all()) and bool(torch.isfinite(dx[:, 4:71].float()).all())


def test_infinite_float32_words_on_the_tensor_cores_are_nan():
    x, table, t, _ = make_xent(33, 300, 72, F32, torch.int64, 0)
    table[11, 3] = -float("inf")
    loss, lse = lsh.lsh_attn_xent(x, table, t)
    assert bool(torch.isnan(lse).all()) and bool(torch.isnan(loss).all())


@pytest.mark.parametrize("n,dtype", [(20, F32), (40, F32), (20, BF16), (300, BF16)])
@pytest.mark.parametrize("portable", [False, True])
def test_gradient_of_sure_rows_is_off_by_the_rounding_of_lse(n, dtype, portable):
    # dx for a table of unit vectors is g itself.  z stands near 20 and the
    # losses lie between exp(-4) and exp(-30); lse rounds by 2^-24 of itself,
    # log2's units of both by as much again, 16 products by 22 steps of 2^-23
    # as above; g's own 2^-16 on top.
    d = 16
    g = gen(n)
    t = torch.randint(0, d, (n,), device=DEV, generator=g)
    table = torch.eye(d, device=DEV, dtype=dtype)
    x = torch.zeros(n, d, device=DEV)
    x[torch.arange(n, device=DEV), t] = 4 + 26 * torch.rand(n, device=DEV, generator=g)
    x = x.to(dtype)
    lse = lsh.lsh_attn_xent(x, table, t, portable=portable)[1]
    dx, _ = lsh.lsh_attn_xent_backward(x, table, t, lse, torch.ones(n, device=DEV),
                                       portable=portable)
    z = x.double()
    p = torch.softmax(z, 1)
    others = torch.where(torch.nn.functional.one_hot(t, d).bool(), torch.zeros_like(p), p)
    want = others - torch.nn.functional.one_hot(t, d) * others.sum(1, keepdim=True)
    err = p * (26 * 2.0 ** -23 * z.amax(1, keepdim=True) + 2.0 ** -21)
    size = want.abs() + err
    R.check("dx", dx, (want, err + size * (R.half_step(dtype) + 2.0 ** -15)))


@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("scale", [1.0, -0.37])
@pytest.mark.parametrize("n", [2, 30, 60, 400])
def test_gradient_of_sure_rows_is_off_by_half_a_step_of_lse(n, scale, portable):
    # as above, with logits of one exact product each.  lse = z scale + loss in
    # one rounding, half a step of it; the loss itself 64 half steps of its own;
    # z scale - lse in one rounding and log2's unit in another, 2^-24 each of the
    # difference; the exponential 2 steps of 2^-22.
    d = 16
    g = gen(n + 1)
    t = torch.randint(0, d, (n,), device=DEV, generator=g)
    table = torch.eye(d, device=DEV)
    x = torch.zeros(n, d, device=DEV)
    x[torch.arange(n, device=DEV), t] = (4 + 36 * torch.rand(n, device=DEV, generator=g)) / scale
    lse = lsh.lsh_attn_xent(x, table, t, scale=scale, portable=portable)[1]
    up = randn(g, n)
    dx, _ = lsh.lsh_attn_xent_backward(x, table, t, lse, up, scale=scale, portable=portable)
    z = x.double() * float(torch.tensor(scale))
    p, full = torch.softmax(z, 1), torch.logsumexp(z, 1, keepdim=True)
    hot = torch.nn.functional.one_hot(t, d).bool()
    others = torch.where(hot, torch.zeros_like(p), p)
    loss = others.sum(1, keepdim=True) / p.gather(1, t[:, None])
    R.check("lse", lse, (full[:, 0], (2.0 ** -24 * full + 2.0 ** -18 * loss)[:, 0]))
    want = torch.where(hot, -others.sum(1, keepdim=True), others)
    err = p * (2.0 ** -24 * full + 2.0 ** -18 * loss + 2.0 ** -23 * (z - full).abs() + 2.0 ** -21)
    up = (up.double() * float(torch.tensor(scale)))[:, None]
    size = up.abs() * (want.abs() + err)
    # (planes of g, the roundings of up and of the products with it)
    R.check("dx", dx, (up * want, up.abs() * err + size * 2.0 ** -20 + 1e-35))


@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_words_masked_by_the_lowest_value_take_no_part(dtype, portable):
    # x's last column is 1, a masked word's entry there the type's lowest value
    g = gen(13)
    x, table = randn(g, 140, 64, dtype=dtype), randn(g, 400, 64, dtype=dtype, scale=0.1)
    x[:, -1] = 1
    masked = torch.rand(400, device=DEV, generator=g) < 0.3
    table[masked, -1] = torch.finfo(dtype).min
    keep = torch.nonzero(~masked)[:, 0]
    at = torch.randint(0, keep.numel(), (140,), device=DEV, generator=g)
    dloss = randn(g, 140)
    loss, lse = lsh.lsh_attn_xent(x, table, keep[at], portable=portable)
    want_loss, want_lse = R.xent(x, table[keep], at, 1.0)
    R.check("lse", lse, want_lse)
    R.check("loss", loss, want_loss)
    dx, dw = lsh.lsh_attn_xent_backward(x, table, keep[at], lse, dloss, portable=portable)
    want_dx, want_dw = R.xent_backward(x, table[keep], at, dloss, 1.0,
                                       BF16 if dtype == BF16 and not portable else None)
    R.check("dx", dx, want_dx)
    R.check("dtable", dw[keep], want_dw)
    assert not bool(dw[masked].any())


def test_a_nan_in_a_row_stays_in_that_row():
    x, table, t, dloss = make_xent(200, 300, 64, BF16, torch.int64, 0)
    x[7, 3] = float("nan")
    loss, lse = lsh.lsh_attn_xent(x, table, t)
    assert bool(torch.isnan(lse[7])) and bool(torch.isnan(loss[7]))
    others = torch.arange(200, device=DEV) != 7
    assert bool(torch.isfinite(lse[others]).all())
    dx, _ = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss)
    assert bool(torch.isnan(dx[7].float()).any())
    assert bool(torch.isfinite(dx[others].float()).all())


@pytest.mark.parametrize("portable", [False, True])
def test_xent_gradient_against_differences(portable):
    # float64 central differences of the definition along random directions
    x, table, t, dloss = make_xent(150, 270, 48, F32, torch.int64, 0.2, seed=3)
    lse = lsh.lsh_attn_xent(x, table, t, scale=0.7, portable=portable)[1]
    dx, dw = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss, scale=0.7, portable=portable)
    g = gen(99)
    ux, uw = randn(g, *x.shape).double(), randn(g, *table.shape).double()

    def f(h):
        loss = R.xent(x.double() + h * ux, table.double() + h * uw, t, 0.7)[0][0]
        return float((loss * dloss.double()).sum())

    # third-order error of the differences: with h = 1e-4 relative 1e-8 of sums
    # of the order of their terms; the gradient's own bound on top
    slope = (f(1e-4) - f(-1e-4)) / 2e-4
    mine = float((dx.double() * ux).sum() + (dw.double() * uw).sum())
    want_dx, want_dw = R.xent_backward(x, table, t, dloss, 0.7)
    size = float((want_dx[0] * ux).abs().sum() + (want_dw[0] * uw).abs().sum())
    bound = float((want_dx[1] * ux.abs()).sum() + (want_dw[1] * uw.abs()).sum()) + 1e-6 * size
    assert abs(slope - mine) <= bound


def test_xent_of_any_leading_shape_and_a_slice_of_targets():
    g = gen(21)
    ids = torch.randint(0, 300, (2 * 7 * 5 + 1,), device=DEV, generator=g)
    targets, x = ids[1:].view(2, 7, 5), randn(g, 2, 7, 5, 64, dtype=BF16)
    table = randn(g, 300, 64, dtype=BF16)
    loss, lse = lsh.lsh_attn_xent(x, table, targets)
    assert loss.shape == lse.shape == targets.shape
    flat = lsh.lsh_attn_xent(x.view(-1, 64), table, targets.reshape(-1).clone())
    assert torch.equal(loss.view(-1), flat[0]) and torch.equal(lse.view(-1), flat[1])
    up = torch.ones_like(loss)
    dx, dw = lsh.lsh_attn_xent_backward(x, table, targets, lse, up)
    want = lsh.lsh_attn_xent_backward(x.view(-1, 64), table, targets.reshape(-1).clone(),
                                      flat[1], up.view(-1))
    assert torch.equal(dx.view(-1, 64), want[0]) and torch.equal(dw, want[1])


def test_loss_and_lse_are_tensors_of_their_own():
    # the loss may be weighted in place with weights that have a gradient, and
    # keeping one of the two does not keep the other's memory
    x, table, t, _ = make_xent(20, 50, 16, F32, torch.int64, 0)
    loss, lse = lsh.lsh_attn_xent(x, table, t)
    assert loss.untyped_storage().nbytes() == lse.untyped_storage().nbytes() == 20 * 4
    value, kept = loss.clone(), lse.clone()
    w = torch.rand(20, device=DEV, requires_grad=True)
    loss.mul_(w)
    loss.sum().backward()
    assert torch.equal(w.grad, value) and torch.equal(lse, kept)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_xent_wait_that_runs_out_reports_timeout_and_next_call_is_clean(dtype):
    # the first wait gives up at once, before any product is issued: both CTAs
    # of every pair leave their loops, and the context stays usable
    x, table, t, dloss = make_xent(700, 900, 64, dtype, torch.int64, 0)
    lib = lsh.lib()
    lsh.lsh_attn_device_check()
    prev = lib.lsh_attn_test_xent_first_wait(0)
    try:
        lsh.lsh_attn_xent(x, table, t)
        with pytest.raises(lsh.LshError) as err:
            lsh.lsh_attn_device_check()
        assert err.value.status == 5  # LSH_ERR_DEVICE_TIMEOUT
    finally:
        assert lib.lsh_attn_test_xent_first_wait(prev) == 0
    loss, lse = lsh.lsh_attn_xent(x, table, t)
    dx, dw = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss)
    lsh.lsh_attn_device_check()
    want_loss, want_lse = R.xent(x, table, t, 1.0)
    R.check("lse", lse, want_lse)
    R.check("loss", loss, want_loss)
    want_dx, want_dw = R.xent_backward(x, table, t, dloss, 1.0, BF16 if dtype == BF16 else None)
    R.check("dx", dx, want_dx)
    R.check("dtable", dw, want_dw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,vocab,d", [(700, 900, 1024), (700, 90000, 264), (60, 900, 1024)])
def test_xent_wait_that_runs_out_while_loads_wait_for_a_slot(n, vocab, d, dtype):
    # more blocks of D than the ring of operands holds, or several tiles to a
    # pair: the loaders stand before a full ring when the wait gives up.  What
    # they have issued lands well within the limit of that second wait (bit 3).
    x, table, t, dloss = make_xent(n, vocab, d, dtype, torch.int64, 0)
    want = lsh.lsh_attn_xent(x, table, t)
    want_grads = lsh.lsh_attn_xent_backward(x, table, t, want[1], dloss)
    lib = lsh.lib()
    lsh.lsh_attn_device_check()
    for call in (lambda: lsh.lsh_attn_xent(x, table, t),
                 lambda: lsh.lsh_attn_xent_backward(x, table, t, want[1], dloss)):
        prev = lib.lsh_attn_test_xent_first_wait(0)
        try:
            call()
            with pytest.raises(lsh.LshError, match="code 0x") as err:
                lsh.lsh_attn_device_check()
        finally:
            assert lib.lsh_attn_test_xent_first_wait(prev) == 0
        assert err.value.status == 5  # LSH_ERR_DEVICE_TIMEOUT
        code = int(str(err.value).split("code ")[1].rstrip(")"), 16)
        assert code & 2 and not code & 8, hex(code)
    loss, lse = lsh.lsh_attn_xent(x, table, t)
    grads = lsh.lsh_attn_xent_backward(x, table, t, lse, dloss)
    lsh.lsh_attn_device_check()
    for got, ref in zip((loss, lse, *grads), (*want, *want_grads)):
        assert torch.equal(got, ref)


# ---- routing ---------------------------------------------------------------------
ROUTE = [  # tokens, k, experts, d, dtype, index, dropped
    (0, 2, 4, 16, BF16, torch.int64, 0),
    (1, 1, 1, 8, F32, torch.int32, 0),
    (64, 2, 8, 512, BF16, torch.int64, 0),
    (100, 1, 5, 40, F32, torch.int64, 1.0),           # every entry dropped
    (1000, 4, 1023, 72, BF16, torch.int32, 0.1),
    (341, 6, 160, 264, F32, torch.int32, 0.3),
    (1025, 2, 64, 1032, BF16, torch.int64, 0.02),
    (3000, 64, 70, 8, BF16, torch.int64, 0.05),
    (2049, 8, 256, 128, F32, torch.int64, 0),
    (5, 3, 2, 16384, BF16, torch.int32, 0.2),
    (1000, 1, 16, 256, BF16, torch.int64, 0.1),
    (301, 1, 4, 1032, F32, torch.int64, 0.1),
    (1001, 2, 16, 72, BF16, torch.int32, 0.1),
    (77, 20, 33, 520, BF16, torch.int64, 0.1),        # entries in three batches, long rows
    (512, 4, 16, 24, BF16, torch.int64, 0.1),         # the most of one CTA
    (683, 3, 9, 24, F32, torch.int64, 0.1),           # one entry more
    (5461, 3, 40, 8, BF16, torch.int64, 0.1),         # eight CTAs, one short
    (8192, 2, 7, 8, BF16, torch.int64, 0.1),          # the most of a cluster
    (3277, 5, 40, 8, BF16, torch.int64, 0.1),         # one more than it takes
    (17001, 8, 300, 8, BF16, torch.int64, 0.1),
    (70001, 2, 33, 8, F32, torch.int32, 0.1),
]


@pytest.mark.parametrize("T,k,E,d,dtype,index,dropped", ROUTE)
def test_route(T, k, E, d, dtype, index, dropped):
    g = gen(T + k * 31 + E)
    ids = make_tokens(g, T * k, E, index, 0.2, dropped).view(T, k)
    w = torch.rand(T, k, device=DEV, generator=g)
    perm, undo, offsets = lsh.lsh_attn_route_sort(ids, E)
    for name, got, want in zip(("perm", "undo", "offsets"), (perm, undo, offsets),
                               R.route_plan(ids.cpu(), E)):
        assert torch.equal(got.cpu(), want), name
    kept = int(offsets[-1])
    x, y = randn(g, T, d, dtype=dtype), randn(g, T * k, d, dtype=dtype)
    # rows and weights of dropped entries are never read
    y[kept:] = float("nan")
    w = torch.where(undo < kept, w, torch.full_like(w, float("nan")))
    assert torch.equal(lsh.lsh_attn_route_gather(x, undo, offsets), R.route_gather(x, undo, kept))
    R.check("out", lsh.lsh_attn_route_combine(y, w, undo, offsets),
            R.route_combine(y, w, undo, kept))
    R.check("dx", lsh.lsh_attn_route_gather_backward(y, undo, offsets),
            R.route_combine(y, None, undo, kept))
    dout = randn(g, T, d, dtype=dtype)
    dy, dw = lsh.lsh_attn_route_combine_backward(dout, y, w, undo, offsets)
    want_dy, want_dw = R.route_combine_backward(dout, y, w, undo, kept)
    R.check("dy", dy, want_dy)
    R.check("dweights", dw, want_dw)


def test_an_expert_named_twice_by_one_token():
    ids = torch.tensor([[2, 2], [0, 2], [1, 1]], device=DEV)
    perm, undo, offsets = lsh.lsh_attn_route_sort(ids, 3)
    assert perm.tolist() == [2, 4, 5, 0, 1, 3]
    assert offsets.tolist() == [0, 1, 3, 6]
    x = randn(gen(2), 3, 8)
    xs = lsh.lsh_attn_route_gather(x, undo, offsets)
    assert torch.equal(xs, x[perm.long() // 2])
    assert torch.equal(lsh.lsh_attn_route_gather_backward(xs, undo, offsets), 2 * x)


# ---- streams, graphs, several calls ------------------------------------------------
def _step(tok, table, targets, ids, w):
    """Tokens in, routed copies, loss against the same table, every gradient."""
    h = lsh.lsh_attn_embed(tok, table, scale=2.0)
    _, undo, off = lsh.lsh_attn_route_sort(ids, 8)
    xs = lsh.lsh_attn_route_gather(h, undo, off)
    x = lsh.lsh_attn_route_combine(xs, w, undo, off)
    loss, lse = lsh.lsh_attn_xent(x, table, targets)
    dloss = (targets >= 0).float() / targets.numel()
    dx, dw_table = lsh.lsh_attn_xent_backward(x, table, targets, lse, dloss)
    dxs, dweights = lsh.lsh_attn_route_combine_backward(dx, xs, w, undo, off)
    dh = lsh.lsh_attn_route_gather_backward(dxs, undo, off)
    dtable = lsh.lsh_attn_embed_backward(tok, dh, table.shape[0], scale=2.0, init=dw_table,
                                         out=dw_table)
    return loss, dweights, dtable


def _step_inputs(seed, dtype, n=333, vocab=600, d=64):
    g = gen(seed)
    tok = make_tokens(g, n, vocab, torch.int64, 0.3, 0.05)
    table = randn(g, vocab, d, dtype=dtype, scale=d ** -0.5)
    ids = make_tokens(g, n * 2, 8, torch.int64, 0, 0.1).view(n, 2)
    return tok, table, make_tokens(g, n, vocab, torch.int64, 0.1, 0.1), ids, \
        torch.rand(n, 2, device=DEV, generator=g)


def test_a_step_against_float64_autograd():
    tok, table, targets, ids, w = _step_inputs(0, F32)
    loss, dweights, dtable = _step(tok, table, targets, ids, w)
    lsh.lsh_attn_device_check()
    V, D = table.shape
    t64, w64 = table.double().requires_grad_(), w.double().requires_grad_()
    pad = torch.cat([t64, torch.zeros(1, D, device=DEV, dtype=torch.float64)])
    h = 2.0 * pad[torch.where((tok >= 0) & (tok < V), tok, V)]
    kept = (ids >= 0) & (ids < 8)
    x = (torch.where(kept, w64, torch.zeros_like(w64))[..., None] * h[:, None]).sum(1)
    z = x @ t64.T
    valid = (targets >= 0) & (targets < V)
    zt = z.gather(1, torch.where(valid, targets, 0)[:, None])[:, 0]
    want = torch.where(valid, torch.logsumexp(z, 1) - zt, 0.0)
    up = ((targets >= 0).double() / targets.numel())
    (want * up).sum().backward()
    # float32 throughout: sums of up to n = 333 or V = 600 terms at every step
    # of a chain of seven, each of relative error 2 * 600 * 2^-24 of magnitudes
    # that stand within 2^3 of the largest result
    tol = 7 * 8 * 2 * 600 * 2.0 ** -24
    for name, got, ref in (("loss", loss, want.detach()), ("dweights", dweights, w64.grad),
                           ("dtable", dtable, t64.grad)):
        err = float((got.detach().double() - ref).abs().max() / ref.abs().max())
        assert err <= tol, f"{name}: {err:.3e} > {tol:.3e}"


def test_a_language_model_step_through_the_attention():
    """Token table, LSH attention in one chunk (so every position sees every
    other: the definition is a dense softmax), routed copies, loss against the
    same table, and the whole gradient, against float64 autograd."""
    g = gen(31)
    B, H, L, dk, V = 2, 2, 64, 16, 300
    D = H * dk
    tok = make_tokens(g, B * L, V, torch.int64, 0.1).view(B, L)
    targets = torch.cat([tok[:, 1:], torch.full_like(tok[:, :1], -1)], dim=1)
    table = randn(g, V, D, scale=D ** -0.5)
    ids = make_tokens(g, B * L * 2, 5, torch.int64, 0, 0.1).view(B * L, 2)
    w = torch.rand(B * L, 2, device=DEV, generator=g)

    def heads(t):
        return t.view(B, L, H, dk).transpose(1, 2).contiguous()

    def rows(t):
        return t.transpose(1, 2).reshape(B * L, D)

    h = lsh.lsh_attn_embed(tok, table, scale=4.0)
    qk = heads(h)
    buckets, inv_norm = lsh.lsh_attn_hash(qk, None, 1)
    perm, _, _ = lsh.lsh_attn_sort(buckets, 1)
    out, lse_a = lsh.lsh_attn_forward(qk, qk, None, 1, 1, L, True)
    a = rows(out).contiguous()
    _, undo, off = lsh.lsh_attn_route_sort(ids, 5)
    ys = lsh.lsh_attn_route_gather(a, undo, off)
    x = lsh.lsh_attn_route_combine(ys, w, undo, off) + h.view(B * L, D)
    loss, lse = lsh.lsh_attn_xent(x, table, targets.view(-1))
    up = (targets.view(-1) >= 0).float() / (targets >= 0).sum()
    dx, dtable = lsh.lsh_attn_xent_backward(x, table, targets.view(-1), lse, up)
    dys, dw = lsh.lsh_attn_route_combine_backward(dx, ys, w, undo, off)
    da = lsh.lsh_attn_route_gather_backward(dys, undo, off)
    dqk, dv = lsh.lsh_attn_backward(qk, qk, inv_norm, perm, out, lse_a, heads(da), L, True,
                                    n_buckets=1)
    dh = dx + rows(dqk + dv)
    lsh.lsh_attn_embed_backward(tok, dh.view(B, L, D), V, scale=4.0, init=dtable, out=dtable)
    lsh.lsh_attn_device_check()

    t64, w64 = table.double().requires_grad_(), w.double().requires_grad_()
    h64 = 4.0 * t64[tok]
    q = h64.view(B, L, H, dk).transpose(1, 2)
    s = (q @ (q / q.norm(dim=-1, keepdim=True)).transpose(2, 3)) / math.sqrt(dk)
    eye = torch.eye(L, device=DEV, dtype=torch.bool)
    s = s.masked_fill(eye, -1e5).masked_fill(torch.ones_like(eye).triu(1), -math.inf)
    a64 = (s.softmax(-1) @ q).transpose(1, 2).reshape(B * L, D)
    kept = ((ids >= 0) & (ids < 5)).double()
    x64 = (w64 * kept).sum(1, keepdim=True) * a64 + h64.view(B * L, D)
    z = x64 @ t64.T
    t = targets.view(-1)
    want = torch.where(t >= 0, torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0],
                       0.0)
    (want * up.double()).sum().backward()
    # float32 throughout: eight steps of sums of up to V terms, each off by
    # 2 * 300 * 2^-24 of magnitudes within 2^4 of the largest result
    tol = 8 * 16 * 2 * 300 * 2.0 ** -24
    for name, got, ref in (("loss", loss, want.detach()), ("dweights", dw, w64.grad),
                           ("dtable", dtable, t64.grad)):
        err = float((got.double() - ref).abs().max() / ref.abs().max())
        assert err <= tol, f"{name}: {err:.3e} > {tol:.3e}"


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_step_captured_and_replayed_on_new_inputs(dtype):
    a, b = _step_inputs(1, dtype), _step_inputs(2, dtype)
    want_a, want_b = _step(*a), _step(*b)
    held = [t.clone() for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(*held)
    for inputs, want in ((a, want_a), (b, want_b), (a, want_a)):
        for h, t in zip(held, inputs):
            h.copy_(t)
        graph.replay()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    lsh.lsh_attn_device_check()


def test_calls_on_another_stream():
    inputs = _step_inputs(4, BF16)
    want = _step(*inputs)
    tok, table, targets, ids, w = inputs
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _step(*inputs)
    # and with the stream handed over
    out = lsh.lsh_attn_embed(tok, table, scale=2.0, stream=s)
    perm = lsh.lsh_attn_route_sort(ids, 8, stream=s)[0]
    loss, lse = lsh.lsh_attn_xent(out, table, targets, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert torch.equal(out, lsh.lsh_attn_embed(tok, table, scale=2.0))
    assert torch.equal(perm, lsh.lsh_attn_route_sort(ids, 8)[0])
    assert torch.equal(loss, lsh.lsh_attn_xent(out, table, targets)[0])


def test_memory_let_go_is_kept_for_the_stream_handed_over():
    # the caller's tensors die while the stream has not begun to read them; what
    # is allocated next on the caller's own stream may not take their memory
    g = gen(41)
    T, V, D, k = 1001, 500, 64, 2
    table, x0 = randn(g, V, D), randn(g, T, D)
    tok, ids = make_tokens(g, T, V, torch.int64), make_tokens(g, T * k, 9, torch.int32).view(T, k)
    lse, up = torch.rand(T, device=DEV, generator=g) + 5, randn(g, T)
    _, undo, off = lsh.lsh_attn_route_sort(ids, 9)
    y, w = randn(g, T * k, D), torch.rand(T, k, device=DEV, generator=g)
    calls = {
        "embed": (lsh.lsh_attn_embed, (tok, table), {}),
        "embed_backward": (lsh.lsh_attn_embed_backward, (tok, x0, V), dict(init=table)),
        "xent": (lsh.lsh_attn_xent, (x0, table, tok), {}),
        "xent_backward": (lsh.lsh_attn_xent_backward, (x0, table, tok, lse, up), {}),
        "sort": (lsh.lsh_attn_route_sort, (ids, 9), {}),
        "gather": (lsh.lsh_attn_route_gather, (x0, undo, off), {}),
        "gather_backward": (lsh.lsh_attn_route_gather_backward, (y, undo, off), {}),
        "combine": (lsh.lsh_attn_route_combine, (y, w, undo, off), {}),
        "combine_backward": (lsh.lsh_attn_route_combine_backward, (x0, y, w, undo, off), {}),
    }

    def tensors(out):
        return out if isinstance(out, tuple) else (out,)

    s = torch.cuda.Stream()
    for name, (call, args, kw) in calls.items():
        want = tensors(call(*args, **kw))
        own = [a.clone() if isinstance(a, torch.Tensor) else a for a in args]
        own_kw = {n: a.clone() for n, a in kw.items()}
        sizes = [a.numel() * a.element_size() for a in (*own, *own_kw.values())
                 if isinstance(a, torch.Tensor)]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)        # some 10 ms
        got = tensors(call(*own, **own_kw, stream=s))
        del own, own_kw
        taken = [torch.full((n,), 0x7f, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(got, want):
            assert torch.equal(a, b), name
        del taken


def test_two_streams_at_once():
    a, b = _step_inputs(5, BF16, n=3001), _step_inputs(6, BF16, n=2500)
    want_a, want_b = _step(*a), _step(*b)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(sa):
            got_a = _step(*a)
        with torch.cuda.stream(sb):
            got_b = _step(*b)
    torch.cuda.synchronize()
    for x, y in zip(got_a + got_b, want_a + want_b):
        assert torch.equal(x, y)


def test_nothing_is_written_past_the_ends():
    # outputs inside larger buffers whose borders keep their value
    g = gen(8)
    n, V, d = 130, 259, 72
    tok = make_tokens(g, n, V, torch.int64, 0.6, 0.1)
    x, table = randn(g, n, d, dtype=BF16), randn(g, V, d, dtype=BF16)

    def framed(rows, cols, dtype):
        buf = torch.full((rows * cols + 2048,), 7, dtype=dtype, device=DEV)
        return buf, buf[1024:1024 + rows * cols].view(rows, cols)

    def whole(buf, size):
        return bool((buf[:1024] == 7).all()) and bool((buf[1024 + size:] == 7).all())

    buf, out = framed(n, d, BF16)
    lsh.lsh_attn_embed(tok, table, out=out)
    assert whole(buf, n * d)
    buf, out = framed(V, d, BF16)
    lsh.lsh_attn_embed_backward(tok, x, V, out=out)
    assert whole(buf, V * d)
    # cross entropy and its gradients through the C ABI, workspaces framed too
    L, st = lsh.lib(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for portable in (False, True):
        s = lsh.make_table_shape(n, V, d, BF16, lsh.I64, 1.0, portable)
        ref = ctypes.byref(s)
        bl, loss = framed(1, n, F32)
        be, lse = framed(1, n, F32)
        need = lsh.lsh_attn_xent_workspace_size(s)
        bw, ws = framed(1, need, torch.uint8)
        assert L.lsh_attn_xent(ref, lsh._ptr(x), lsh._ptr(table), lsh._ptr(tok), lsh._ptr(loss),
                               lsh._ptr(lse), lsh._ptr(ws), need, st) == 0
        assert whole(bl, n) and whole(be, n) and whole(bw, need)
        up = torch.ones(n, device=DEV)
        bx, dx = framed(n, d, BF16)
        bt, dt = framed(V, d, BF16)
        need = lsh.lsh_attn_xent_backward_workspace_size(s)
        bw, ws = framed(1, need, torch.uint8)
        assert L.lsh_attn_xent_backward(ref, lsh._ptr(x), lsh._ptr(table), lsh._ptr(tok),
                                        lsh._ptr(lse), lsh._ptr(up), lsh._ptr(dx), lsh._ptr(dt),
                                        lsh._ptr(ws), need, st) == 0
        assert whole(bx, n * d) and whole(bt, V * d) and whole(bw, need)


def test_outputs_over_inputs_are_refused():
    tok = torch.tensor([3, 0, 2, 1], device=DEV)
    buf = torch.zeros(12, 16, device=DEV)
    table, ids = buf[:4], tok.view(4, 1)
    _, undo, off = lsh.lsh_attn_route_sort(ids, 4)
    w = torch.ones(4, 1, device=DEV)
    for call in (lambda: lsh.lsh_attn_embed(tok, table, out=table),
                 lambda: lsh.lsh_attn_embed(tok, table, out=buf[1:5]),
                 lambda: lsh.lsh_attn_embed_backward(tok, table, 4, out=table),
                 lambda: lsh.lsh_attn_embed_backward(tok, buf[8:], 4, init=table, out=buf[1:5]),
                 lambda: lsh.lsh_attn_route_gather(table, undo, off, out=table),
                 lambda: lsh.lsh_attn_route_gather_backward(table, undo, off, out=table),
                 lambda: lsh.lsh_attn_route_combine(table, w, undo, off, out=table)):
        with pytest.raises(ValueError, match="out lies over"):
            call()
    # a gradient added in place is what init is for
    lsh.lsh_attn_embed_backward(tok, buf[8:] + 1, 4, init=table, out=table)
    assert bool((buf[:4] == 1).all()) and not bool(buf[4:].any())


def test_binding_checks_its_tensors():
    tok = torch.zeros(4, dtype=torch.int64, device=DEV)
    table = torch.zeros(8, 16, device=DEV)
    x = torch.zeros(4, 16, device=DEV)
    f = torch.zeros(4, device=DEV)
    with pytest.raises(TypeError, match="int32 or int64"):
        lsh.lsh_attn_embed(tok.short(), table)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        lsh.lsh_attn_embed(tok, table.half())
    with pytest.raises(ValueError, match="vocab"):
        lsh.lsh_attn_embed(tok, table[0])
    with pytest.raises(ValueError, match="contiguous"):
        lsh.lsh_attn_embed(tok, table.T)
    with pytest.raises(ValueError, match="out must have shape"):
        lsh.lsh_attn_embed(tok, table, out=x[:2])
    with pytest.raises(ValueError, match="dout must be"):
        lsh.lsh_attn_embed_backward(tok, x[:3], 8)
    with pytest.raises(ValueError, match="init must have shape"):
        lsh.lsh_attn_embed_backward(tok, x, 8, init=x)
    with pytest.raises(TypeError, match="table must be"):
        lsh.lsh_attn_xent(x, table.bfloat16(), tok)
    with pytest.raises(ValueError, match="targets must have shape"):
        lsh.lsh_attn_xent(x, table, tok[:3])
    with pytest.raises(TypeError, match="lse must be"):
        lsh.lsh_attn_xent_backward(x, table, tok, f.double(), f)
    with pytest.raises(TypeError, match="workspace must be"):
        lsh.lsh_attn_xent(x, table, tok, workspace=f)
    with pytest.raises(lsh.LshError, match="LSH_ERR_WORKSPACE"):
        lsh.lsh_attn_xent(x, table, tok, workspace=torch.empty(1, dtype=torch.uint8, device=DEV))
    with pytest.raises(lsh.LshError, match="multiple of 8"):
        lsh.lsh_attn_embed(tok, torch.zeros(8, 12, device=DEV))
    with pytest.raises(ValueError, match="undo must be"):
        lsh.lsh_attn_route_gather(x, tok.int(), tok.int())
    with pytest.raises(ValueError, match=r"y must be \[8, d_model\]"):
        lsh.lsh_attn_route_combine(x, torch.zeros(4, 2, device=DEV),
                                   torch.zeros(4, 2, dtype=torch.int32, device=DEV), tok.int())
    with pytest.raises(ValueError, match="stream is on|CUDA"):
        lsh.lsh_attn_embed(tok.cpu(), table)
