"""Cases of the operators at a language model's two ends and around its routed layers.

Three families, each as a user's training or serving program calls it next to
the LSH attention:

* the token table's lookup (``embed``) and its gradient by sorted tokens
  (``embed_grad``);
* tokens sorted by expert (``route``), brought back with their weights
  (``unroute``), and a whole training step of the two with every gradient
  (``route_step``);
* the softmax cross entropy over the vocabulary without stored logits
  (``loss``) and with its gradients (``loss_step``).

``run`` computes a case with the framework's calls when ``own`` is true, and
with elementary torch operations in 32 bits otherwise.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one new token for each of eight running sequences: launch latency
        dict(name="embed-step", op="embed", rows=8, vocab=32768, d=512, dtype="bf16", scale=22.627416997969522,
             idx="i64", holes=0.0),
        # the long-text sequence of the repository's benchmark, 65536 tokens, in one lookup
        dict(name="embed-long", op="embed", rows=65536, vocab=32768, d=1024, dtype="bf16", scale=1.0,
             idx="i64", holes=0.0),
        # its gradient: Zipf-distributed tokens, some of them very frequent
        dict(name="embed-grad-long", op="embed_grad", rows=65536, vocab=32768, d=1024, dtype="bf16", scale=1.0,
             idx="i64", holes=0.0, into=False),
        # float32, an odd token count with padding, added into a gradient that is there (a tied table)
        dict(name="embed-grad-into", op="embed_grad", rows=12287, vocab=50021, d=520, dtype="f32", scale=0.5,
             idx="i32", holes=0.1, into=True),
        # serving: a step of 64 sequences, two experts each
        dict(name="route-step-small", op="route", tokens=64, top_k=2, experts=8, d=512, dtype="bf16", idx="i64",
             dropped=0.0),
        # the experts' rows of a long batch brought back
        dict(name="unroute-long", op="unroute", tokens=65536, top_k=2, experts=64, d=1024, dtype="bf16", idx="i64",
             dropped=0.0),
        # a training step, all moves and their gradients
        dict(name="route-train", op="route_step", tokens=32768, top_k=4, experts=128, d=1024, dtype="bf16", idx="i64",
             dropped=0.02),
        # float32, odd sizes, many experts, a tenth of the entries over capacity
        dict(name="route-train-odd", op="route_step", tokens=4093, top_k=6, experts=160, d=264, dtype="f32", idx="i32",
             dropped=0.1),
        # bytes as tokens: the smallest vocabulary and a short batch
        dict(name="loss-bytes", op="loss", rows=250, vocab=256, d=512, dtype="bf16", scale=1.0, idx="i64", holes=0.0),
        # float32 training step with odd sizes and ignored targets
        dict(name="loss-train-f32", op="loss_step", rows=2047, vocab=8009, d=520, dtype="f32", scale=1.0, idx="i32",
             holes=0.1),
        # the loss of an evaluation batch over a large vocabulary
        dict(name="loss-eval", op="loss", rows=4093, vocab=131071, d=512, dtype="bf16", scale=1.0, idx="i64",
             holes=0.05),
        # a training step over 32768 tokens and 32768 words
        dict(name="loss-train", op="loss_step", rows=32768, vocab=32768, d=1024, dtype="bf16", scale=1.0, idx="i64",
             holes=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "route", "unroute", "route_step", "loss", "loss_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    case = dict(op=op, dtype=dtype, idx=rng.choice(["i64", "i32"]))
    d = 8 * _log(rng, 8, 128)
    if op in ("embed", "embed_grad"):
        case.update(rows=_log(rng, 1, 65536), vocab=_log(rng, 256, 131072), d=d, scale=rng.choice([1.0, math.sqrt(d)]),
                    holes=rng.choice([0.0, 0.1, 0.5]))
        if op == "embed_grad":
            case.update(into=rng.choice([False, True]))
    elif op in ("route", "unroute", "route_step"):
        k = rng.choice([1, 2, 4, 6, 8])
        case.update(tokens=_log(rng, 1, 131072 // k), top_k=k, experts=max(k, _log(rng, 8, 256)), d=d,
                    dropped=rng.choice([0.0, 0.02, 0.3]))
    else:
        vocab = _log(rng, 256, 131072)
        # float32 logits of the plain form within 2 GB, its work below the largest listed case's
        most = min(16384, 2 ** 29 // vocab)
        case.update(rows=_log(rng, 1, most), vocab=vocab, d=d, scale=rng.choice([1.0, 1.0, d ** -0.5]),
                    holes=rng.choice([0.0, 0.05, 0.5]))
    return case


# ---- inputs -------------------------------------------------------------------
def _gen(seed):
    return torch.Generator("cuda").manual_seed(1000003 * 7 + int(seed))


def _tokens(case, g):
    """Zipf(1.1)-distributed ids in a shuffled vocabulary; a share `holes` is -1."""
    n, vocab = case["rows"], case["vocab"]
    # (the distribution's sums are made on the host, where their order is fixed)
    share = torch.arange(1, vocab + 1, dtype=torch.float64).pow(-1.1).cumsum(0)
    below = (share / share[-1]).cuda()
    ids = torch.searchsorted(below, torch.rand(n, device="cuda", generator=g, dtype=torch.float64))
    ids = torch.randperm(vocab, device="cuda", generator=g)[ids.clamp(max=vocab - 1)]
    if case["holes"]:
        gone = torch.rand(n, device="cuda", generator=g) < case["holes"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.to(torch.int64 if case["idx"] == "i64" else torch.int32)


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32)


def prepare(case, seed):
    g, dt, d = _gen(seed), DTYPES[case["dtype"]], case["d"]
    s = dict(case=case)
    if case["op"] in ("embed", "embed_grad"):
        s["tokens"] = _tokens(case, g)
        if case["op"] == "embed":
            s["table"] = (_randn(g, case["vocab"], d) * d ** -0.5).to(dt)
        else:
            s["dout"] = (_randn(g, case["rows"], d) * 1e-2).to(dt)
            if case["into"]:
                s["dtable0"] = (_randn(g, case["vocab"], d) * 1e-2).to(dt)
    elif case["op"] in ("loss", "loss_step"):
        n = case["rows"]
        s["targets"] = _tokens(case, g)
        table = _randn(g, case["vocab"], d) * d ** -0.5
        # the target's logit stands 0 to 14 above the others', as in a model that has learned
        lift = 14.0 * torch.rand(n, 1, device="cuda", generator=g)
        x = (_randn(g, n, d) + lift * table[s["targets"].clamp(min=0).long()]) / case["scale"]
        s["x"], s["table"] = x.to(dt), table.to(dt)
        if case["op"] == "loss_step":
            valid = s["targets"] >= 0
            s["dloss"] = valid.float() / valid.sum().clamp(min=1)
    else:
        t, k, e = case["tokens"], case["top_k"], case["experts"]
        # a router's choice: some experts are more popular than others
        logits = _randn(g, t, e) + 0.5 * _randn(g, e)
        top, ids = logits.topk(k, dim=1)
        if case["dropped"]:
            gone = torch.rand(t, k, device="cuda", generator=g) < case["dropped"]
            ids = torch.where(gone, torch.full_like(ids, -1), ids)
        s["ids"] = ids.to(torch.int64 if case["idx"] == "i64" else torch.int32).contiguous()
        s["weights"] = torch.exp(top - top.logsumexp(dim=1, keepdim=True)).contiguous()
        if case["op"] in ("route", "route_step"):
            s["x"] = _randn(g, t, d).to(dt)
        if case["op"] in ("unroute", "route_step"):
            s["y"] = _randn(g, t * k, d).to(dt)
        if case["op"] == "unroute":  # the plan of the sort that came before
            s["undo"], s["offsets"] = _plan(s["ids"], e)[1:]
        if case["op"] == "route_step":
            s["dout"] = (_randn(g, t, d) * 1e-2).to(dt)
            s["dxs"] = (_randn(g, t * k, d) * 1e-2).to(dt)
    return s


# ---- the plain forms ------------------------------------------------------------
def _plan(ids, experts):
    """perm, undo and offsets of the stable order by expert, dropped entries last."""
    key = ids.reshape(-1).long()
    key = torch.where((key >= 0) & (key < experts), key, torch.full_like(key, experts))
    perm = torch.sort(key, stable=True).indices
    undo = torch.empty_like(perm)
    undo[perm] = torch.arange(perm.numel(), device=perm.device)
    count = torch.zeros(experts + 1, dtype=torch.int64, device=perm.device)
    count.index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)[:experts]])
    return perm.int(), undo.int().reshape(ids.shape), offsets.int()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "embed":
        there = (s["tokens"] >= 0) & (s["tokens"] < case["vocab"])
        rows = s["table"][torch.where(there, s["tokens"], 0).long()].float() * case["scale"]
        return torch.where(there[:, None], rows, 0.0).to(s["table"].dtype)
    if op == "embed_grad":
        there = (s["tokens"] >= 0) & (s["tokens"] < case["vocab"])
        sums = torch.zeros(case["vocab"] + 1, case["d"], device="cuda")
        sums.index_add_(0, torch.where(there, s["tokens"], case["vocab"]).long(), s["dout"].float())
        sums = sums[:-1] * case["scale"]
        if case["into"]:
            sums = sums + s["dtable0"].float()
        return sums.to(s["dout"].dtype)
    if op in ("loss", "loss_step"):
        x, table = s["x"].float(), s["table"].float()
        logits = (x @ table.T) * case["scale"]
        most = logits.amax(dim=1, keepdim=True)
        lse = most[:, 0] + torch.exp(logits - most).sum(dim=1).log()
        valid = (s["targets"] >= 0) & (s["targets"] < case["vocab"])
        at = torch.where(valid, s["targets"], 0).long()[:, None]
        loss = torch.where(valid, lse - logits.gather(1, at)[:, 0], 0.0)
        if op == "loss":
            return loss, lse
        g = torch.exp(logits - lse[:, None])
        del logits
        g.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=g.dtype))
        g *= torch.where(valid, s["dloss"] * case["scale"], 0.0)[:, None]
        return loss, lse, (g @ table).to(s["x"].dtype), (g.T @ x).to(s["table"].dtype)
    t, k, d = case["tokens"], case["top_k"], case["d"]
    if op == "unroute":
        undo, offsets = s["undo"].long(), s["offsets"]
        kept = undo < offsets[-1]
        w = torch.where(kept, s["weights"], 0.0)
        return (w[..., None] * s["y"][undo].float()).sum(dim=1).to(s["y"].dtype)
    perm, undo, offsets = _plan(s["ids"], case["experts"])
    kept_slots = torch.arange(t * k, device="cuda") < offsets[-1]
    token = torch.div(perm.long(), k, rounding_mode="floor")
    xs = torch.where(kept_slots[:, None], s["x"][token].float(), 0.0).to(s["x"].dtype)
    if op == "route":
        return perm, undo, offsets, xs
    at, kept = undo.long(), undo < offsets[-1]
    w = torch.where(kept, s["weights"], 0.0)
    y = s["y"][at].float()
    out = (w[..., None] * y).sum(dim=1).to(s["y"].dtype)
    dw = torch.where(kept, (s["dout"].float()[:, None] * y).sum(dim=2), 0.0)
    dy = (w.reshape(-1)[perm.long()][:, None] * s["dout"][token].float()).to(s["y"].dtype)
    dx = torch.where(kept[..., None], s["dxs"][at].float(), 0.0).sum(dim=1).to(s["x"].dtype)
    return perm, undo, offsets, xs, out, dy, dw, dx


def _own(s):
    import lsh_bucketed_sparse_b200 as lsh
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return lsh.lsh_attn_embed(s["tokens"], s["table"], scale=case["scale"])
    if op == "embed_grad":
        # a gradient that is there already (the tied table's from the loss) is added to
        return lsh.lsh_attn_embed_backward(s["tokens"], s["dout"], case["vocab"], scale=case["scale"],
                                           init=s.get("dtable0"))
    if op in ("loss", "loss_step"):
        loss, lse = lsh.lsh_attn_xent(s["x"], s["table"], s["targets"], scale=case["scale"])
        if op == "loss":
            return loss, lse
        dx, dtable = lsh.lsh_attn_xent_backward(s["x"], s["table"], s["targets"], lse, s["dloss"], scale=case["scale"])
        return loss, lse, dx, dtable
    if op == "unroute":
        return lsh.lsh_attn_route_combine(s["y"], s["weights"], s["undo"], s["offsets"])
    perm, undo, offsets = lsh.lsh_attn_route_sort(s["ids"], case["experts"])
    xs = lsh.lsh_attn_route_gather(s["x"], undo, offsets)
    if op == "route":
        return perm, undo, offsets, xs
    out = lsh.lsh_attn_route_combine(s["y"], s["weights"], undo, offsets)
    dy, dw = lsh.lsh_attn_route_combine_backward(s["dout"], s["y"], s["weights"], undo, offsets)
    dx = lsh.lsh_attn_route_gather_backward(s["dxs"], undo, offsets)
    return perm, undo, offsets, xs, out, dy, dw, dx


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e, d, i = SIZE[case["dtype"]], case["d"], 8 if case["idx"] == "i64" else 4
    op = case["op"]
    if op == "embed":
        n = case["rows"]
        # each distinct row of the table is read at least once
        return dict(bytes=n * i + min(n, case["vocab"]) * d * e + n * d * e, flops=n * d)
    if op == "embed_grad":
        n = case["rows"]
        table = case["vocab"] * d * e
        return dict(bytes=n * i + n * d * e + (2 * table if case["into"] else table), flops=n * d)
    if op in ("loss", "loss_step"):
        n, v = case["rows"], case["vocab"]
        ins = (n + v) * d * e + n * i
        if op == "loss":
            return dict(bytes=ins + 8 * n, flops=2 * n * v * d)
        return dict(bytes=ins + 12 * n + (n + v) * d * e, flops=6 * n * v * d)
    t, k, x = case["tokens"], case["top_k"], case["experts"]
    one, many, plan = t * d * e, t * k * d * e, t * k * i + 8 * t * k + 4 * (x + 1)
    if op == "route":
        return dict(bytes=plan + one + many, flops=0)
    if op == "unroute":
        return dict(bytes=8 * t * k + many + one, flops=2 * t * k * d)
    # sort and gather; combine and its gradient share y; the gather's gradient
    return dict(bytes=plan + 8 * t * k + 4 * one + 4 * many, flops=8 * t * k * d)


# ---- in 64 bits -------------------------------------------------------------------
def _exact_loss(s, case):
    """Blocks of rows; each row's definition written out."""
    x, table = s["x"].double(), s["table"].double()
    n, v, c = case["rows"], case["vocab"], case["scale"]
    loss, lse = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    dx, dtable = torch.zeros_like(x), torch.zeros_like(table)
    step = max(1, 2 ** 27 // v)
    for a in range(0, n, step):
        b = min(n, a + step)
        z = c * (x[a:b] @ table.T)
        lse[a:b] = torch.logsumexp(z, dim=1)
        t = s["targets"][a:b].long()
        rows = torch.nonzero((t >= 0) & (t < v))[:, 0]
        loss[a + rows] = lse[a + rows] - z[rows, t[rows]]
        if case["op"] == "loss_step":
            p = torch.softmax(z, dim=1)
            up = torch.zeros(b - a, dtype=torch.float64, device="cuda")
            up[rows] = s["dloss"][a + rows].double() * c
            p[rows, t[rows]] -= 1.0
            p *= up[:, None]
            dx[a:b] = p @ table
            dtable += p.T @ x[a:b]
    return (loss, lse) if case["op"] == "loss" else (loss, lse, dx, dtable)


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op in ("loss", "loss_step"):
        return _exact_loss(s, case)
    if op == "embed":
        out = torch.zeros(case["rows"], d, dtype=torch.float64, device="cuda")
        rows = torch.nonzero((s["tokens"] >= 0) & (s["tokens"] < case["vocab"]))[:, 0]
        out[rows] = case["scale"] * s["table"].double()[s["tokens"][rows].long()]
        return out
    if op == "embed_grad":
        out = torch.zeros(case["vocab"], d, dtype=torch.float64, device="cuda")
        rows = torch.nonzero((s["tokens"] >= 0) & (s["tokens"] < case["vocab"]))[:, 0]
        out.index_put_((s["tokens"][rows].long(),), case["scale"] * s["dout"][rows].double(), accumulate=True)
        return out + s["dtable0"].double() if case["into"] else out
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    ids = s["ids"].reshape(-1).long()
    there = (ids >= 0) & (ids < e)
    # entries of expert 0 in their order, then of expert 1, ..., dropped ones last
    place = (ids * (t * k) + torch.arange(t * k, device="cuda")).masked_fill(~there, e * t * k)
    place = torch.where(there, place, e * t * k + torch.arange(t * k, device="cuda"))
    perm = torch.argsort(place)
    kept = int(there.sum())
    entry = perm[:kept]                       # the entry in each kept slot
    token = torch.div(entry, k, rounding_mode="floor")
    if op in ("unroute", "route_step"):
        y = s["y"].double()
        w = s["weights"].double().reshape(-1)[entry]
        out = torch.zeros(t, d, dtype=torch.float64, device="cuda")
        out.index_add_(0, token, w[:, None] * y[:kept])
        if op == "unroute":
            return out
    xs = torch.zeros(t * k, d, dtype=torch.float64, device="cuda")
    xs[:kept] = s["x"].double()[token]
    if op == "route":
        return None, None, None, xs
    dout = s["dout"].double()
    dy = torch.zeros(t * k, d, dtype=torch.float64, device="cuda")
    dy[:kept] = w[:, None] * dout[token]
    dw = torch.zeros(t * k, dtype=torch.float64, device="cuda")
    dw[entry] = (dout[token] * y[:kept]).sum(dim=1)
    dx = torch.zeros(t, d, dtype=torch.float64, device="cuda")
    dx.index_add_(0, token, s["dxs"].double()[:kept])
    return None, None, None, xs, out, dy, dw.reshape(t, k), dx
