"""The token-table, cross-entropy and routing operators in float64 torch, and
bounds on what float32 sums and the roundings of the result types may add.

Each function returns (value, bound): the kernels' result may differ from
``value`` by ``bound``, element by element.  U is the unit roundoff of the
float32 sums; matrix instructions may truncate instead of rounding, so a sum
of K terms counts 2 K U of the sum of magnitudes.
"""

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(value, err, dtype):
    """Bound after one rounding to dtype of something within err of value."""
    return err + (value.abs() + err) * half_step(dtype) + torch.finfo(torch.float32).tiny


def embed(tokens, table, scale):
    there = (tokens >= 0) & (tokens < table.shape[0])
    rows = table.double()[torch.where(there, tokens, torch.zeros_like(tokens)).long()] * scale
    rows = torch.where(there[..., None], rows, torch.zeros_like(rows))
    return rows, rounded(rows, rows.abs() * 2 * U, table.dtype)


def embed_backward(tokens, dout, vocab, scale, init=None):
    tok, g = tokens.reshape(-1).long(), dout.double().reshape(-1, dout.shape[-1])
    rows = torch.nonzero((tok >= 0) & (tok < vocab))[:, 0]
    total = torch.zeros(vocab, g.shape[1], dtype=torch.float64, device=g.device)
    size, count = torch.zeros_like(total), torch.zeros(vocab, dtype=torch.float64, device=g.device)
    total.index_add_(0, tok[rows], g[rows])
    size.index_add_(0, tok[rows], g[rows].abs())
    count.index_add_(0, tok[rows], torch.ones_like(rows, dtype=torch.float64))
    value, err = total * scale, (count[:, None] + 3) * U * size * abs(scale)
    if init is not None:
        value = value + init.double()
        err = err + 2 * U * (value.abs() + init.double().abs())
    return value, rounded(value, err, dout.dtype)


def logits(x, table, scale):
    z = scale * (x.double() @ table.double().T)
    size = abs(scale) * (x.double().abs() @ table.double().abs().T)
    return z, (2 * x.shape[-1] + 2) * U * size


def xent(x, table, targets, scale):
    """((loss, bound), (lse, bound)) for x [n, D], targets [n]."""
    z, ez = logits(x, table, scale)
    V = table.shape[0]
    lse = torch.logsumexp(z, dim=1)
    # exp of a difference: its rounding, exp's own error (4 U) and the sum of
    # V positive terms, at most V / 16 + 64 of them after one another
    rel = 2 * U * (z.amax(1).abs() + (z.amax(1) - z.amin(1))) + (V / 16 + 64 + 8) * U
    e_lse = ez.amax(1) + rel + 4 * U * (lse.abs() + 1)
    t = targets.long()
    valid = (t >= 0) & (t < V)
    at = torch.where(valid, t, torch.zeros_like(t))[:, None]
    zt, ezt = z.gather(1, at)[:, 0], ez.gather(1, at)[:, 0]
    zero = torch.zeros_like(lse)
    loss = torch.where(valid, lse - zt, zero)
    e_loss = torch.where(valid, e_lse + ezt + 2 * U * loss.abs(), zero)
    return (loss, e_loss), (lse, e_lse)


def xent_backward(x, table, targets, dloss, scale, g_dtype=None):
    """((dx, bound), (dtable, bound)); g is rounded to g_dtype before the two
    products when one is given."""
    z, ez = logits(x, table, scale)
    n, V = z.shape
    _, (lse, e_lse) = xent(x, table, targets, scale)
    t = targets.long()
    valid = (t >= 0) & (t < V)
    up = torch.where(valid, dloss.double() * scale, torch.zeros_like(lse))[:, None]
    p = torch.exp(z - lse[:, None])
    hot = torch.zeros_like(p)
    hot[torch.nonzero(valid)[:, 0], t[valid]] = 1.0
    g = up * (p - hot)
    ep = p * (ez + e_lse[:, None] + 2 * U * (z.abs() + lse.abs()[:, None]) + 8 * U)
    eg = up.abs() * ep + 4 * U * g.abs()
    if g_dtype is not None:
        eg = eg + (g.abs() + eg) * half_step(g_dtype)
    xd = torch.where(valid[:, None], x.double(), torch.zeros_like(x, dtype=torch.float64))
    w = table.double()
    dx, dw = g @ w, g.T @ xd
    sx, sw = (g.abs() + eg) @ w.abs(), (g.abs() + eg).T @ xd.abs()
    ex = eg @ w.abs() + (2 * V + 8) * U * sx
    ew = eg.T @ xd.abs() + (2 * n + 8) * U * sw
    return (dx, rounded(dx, ex, x.dtype)), (dw, rounded(dw, ew, x.dtype))


def route_plan(experts, n_experts):
    """perm, undo, offsets by Python's stable sort."""
    flat = [int(e) if 0 <= int(e) < n_experts else n_experts
            for e in experts.reshape(-1).tolist()]
    perm = sorted(range(len(flat)), key=lambda i: flat[i])
    undo = [0] * len(flat)
    for slot, entry in enumerate(perm):
        undo[entry] = slot
    offsets = [sum(1 for e in flat if e < v) for v in range(n_experts + 1)]
    return (torch.tensor(perm, dtype=torch.int32),
            torch.tensor(undo, dtype=torch.int32).reshape(experts.shape),
            torch.tensor(offsets, dtype=torch.int32))


def route_gather(x, undo, kept):
    xs = torch.zeros(undo.numel(), x.shape[1], dtype=x.dtype, device=x.device)
    for j in range(undo.shape[1]):
        s = undo[:, j].long()
        on = s < kept
        xs[s[on]] = x[on]
    return xs


def route_combine(y, weights, undo, kept):
    """weights None: every weight 1."""
    on = undo < kept
    w = torch.ones_like(undo, dtype=torch.float64) if weights is None else weights.double()
    w = torch.where(on, w, torch.zeros_like(w))
    rows = y.double()[torch.where(on, undo, torch.zeros_like(undo)).long()]
    rows = torch.where(on[..., None], rows, torch.zeros_like(rows))
    out = (w[..., None] * rows).sum(1)
    err = (undo.shape[1] + 1) * U * (w.abs()[..., None] * rows.abs()).sum(1)
    return out, rounded(out, err, y.dtype)


def route_combine_backward(dout, y, weights, undo, kept):
    on = undo < kept
    dy = torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    dw = torch.zeros(undo.shape, dtype=torch.float64, device=y.device)
    ew = torch.zeros_like(dw)
    g = dout.double()
    for j in range(undo.shape[1]):
        o = on[:, j]
        s = undo[o, j].long()
        dy[s] = weights[o, j].double()[:, None] * g[o]
        dw[o, j] = (g[o] * y.double()[s]).sum(1)
        ew[o, j] = (y.shape[1] + 1) * U * (g[o].abs() * y.double()[s].abs()).sum(1)
    return (dy, rounded(dy, 2 * U * dy.abs(), y.dtype)), (dw, ew + torch.finfo(torch.float32).tiny)


def check(name, got, want):
    value, bound = want
    assert got.shape == value.shape, f"{name}: shape {tuple(got.shape)}, not {tuple(value.shape)}"
    if got.numel() == 0:
        return
    diff = (got.double() - value).abs()
    bad = ~(diff <= bound)
    if bool(bad.any()):
        at = tuple(int(i) for i in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {got.numel()} beyond their bound, first "
                             f"at {at}: {float(got[at])!r}, not {float(value[at])!r} "
                             f"+- {float(bound[at]):.3e}")
