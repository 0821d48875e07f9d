"""Cases that measure the experts' routing, the embedding and the distillation loss.

``run`` computes a case in plain torch operations (``own`` false) or with the
calls of ``quantized_linear_layer_amd`` (``own`` true); ``exact`` is the same
from the definition in 64 bits.

Routing (op ``dispatch``, ``combine``, ``combine_backward``). Each of T tokens goes
to k experts: its slots t * k + j. The slots are sorted by expert, stably; those
whose expert lies outside [0, E) come last and carry nothing. ``dispatch`` gives
the tokens' rows in that order, the ends of the experts' rows and each slot's row;
``combine`` adds a token's rows again, each times its weight, and a residual.
Without weights it is the gradient of ``dispatch``.

Embedding (op ``embed``, ``embed_backward``): rows of a table times a scale, zeros
for a token outside the vocabulary, and the gradient of the whole table.

Distillation (op ``distill``, ``distill_train``): the divergence of the softmax of the
logits X W / temperature from the softmax of a teacher's top logits over its list
of indices, with the gradients of X and W in ``distill_train``. Entries whose index
lies outside the vocabulary are left out.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token on its way to its two experts: serving, where latency counts
        dict(name="dispatch 1 token", op="dispatch", dtype="bf16", T=1, k=2, E=8, H=2048, left=0.0),
        # the layer of a training step
        dict(name="dispatch 8192 tokens", op="dispatch", dtype="bf16", T=8192, k=2, E=8, H=4096, left=0.0),
        # the way back of 64 sequences' new tokens, the products in float32, the residual bfloat16
        dict(name="combine 64 tokens", op="combine", dtype="f32", out="bf16", T=64, k=2, E=8, H=4096, left=0.0,
             weighted=True, residual=True),
        # the same of a training step
        dict(name="combine 8192 tokens", op="combine", dtype="f32", out="bf16", T=8192, k=2, E=8, H=4096, left=0.0,
             weighted=True, residual=True),
        # its gradient: what goes into the down projection's products, and the router's part
        dict(name="combine backward 4096 tokens", op="combine_backward", dtype="f32", out="bf16", T=4096, k=2, E=16,
             H=2048, left=0.0),
        # float32, nothing a multiple of anything, a part of the tokens padding
        dict(name="combine backward odd f32", op="combine_backward", dtype="f32", out="f32", T=1001, k=3, E=5, H=515,
             left=0.1),
        # a step of 64 sequences, one new token each
        dict(name="embed 64 tokens", op="embed", dtype="bf16", T=64, H=4096, V=32000, left=0.0),
        # a training batch
        dict(name="embed 8192 tokens", op="embed", dtype="bf16", T=8192, H=4096, V=32000, left=0.0),
        # its gradient: a few tokens of a text are most of it
        dict(name="embed backward 8192 tokens", op="embed_backward", dtype="bf16", T=8192, H=4096, V=32000, left=0.0),
        # float32, odd sizes, padding
        dict(name="embed backward odd f32", op="embed_backward", dtype="f32", T=1001, H=515, V=5003, left=0.1),
        # scoring a student on the last tokens of 32 sequences
        dict(name="distill 32 rows", op="distill", dtype="bf16", T=32, H=4096, V=32000, k=64, temperature=1.0,
             by_vocab=False, left=0.0),
        # a training step of a small student
        dict(name="distill train 4096x2048", op="distill_train", dtype="bf16", T=4096, H=2048, V=32000, k=64,
             temperature=2.0, by_vocab=True, left=0.0),
    ]


def _log(rng, low, high):
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(max(v, low), high)


def draw(rng):
    op = rng.choice(("dispatch", "combine", "combine_backward", "embed", "embed_backward", "distill",
                     "distill_train"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    left = rng.choice((0.0, 0.0, 0.1, 0.5))
    T, H = _log(rng, 1, 8192), _log(rng, 64, 4096)
    if rng.random() < 0.5:
        H = 8 * (-(-H // 8))
    if op in ("dispatch", "combine", "combine_backward"):
        E = _log(rng, 2, 256)
        k = min(rng.choice((1, 2, 2, 4, 6, 8)), E)
        T = min(T, 16384 // k)
        case = dict(op=op, dtype=dtype, T=T, k=k, E=E, H=H, left=left)
        if op != "dispatch":
            case["out"] = rng.choice((dtype, "bf16"))
        if op == "combine":
            case["weighted"], case["residual"] = rng.random() < 0.7, rng.random() < 0.7
        return case
    V = _log(rng, 1000, 32000)
    if op in ("embed", "embed_backward"):
        return dict(op=op, dtype=dtype, T=T, H=H, V=V, left=left)
    if rng.random() < 0.5:
        V = 8 * (-(-V // 8))
    T, H = min(T, 4096), min(H, 2048)
    return dict(op=op, dtype=dtype, T=min(T, 2048) if dtype == "f32" else T, H=H, V=V, k=_log(rng, 1, 256),
                temperature=rng.choice((1.0, 2.0, 0.7)), by_vocab=rng.random() < 0.5, left=left)


# ---- inputs -------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _some(n, part, g):
    """Which of n are left out: about the given part, never the first."""
    out = torch.rand((n,), generator=g, device="cuda") < part
    out[0] = False
    return out


def _tokens(case, g):
    """Tokens of a text: the frequency of the r-th most frequent one falls as 1 / r."""
    V = case["V"]
    weight = 1.0 / (torch.arange(V, device="cuda", dtype=torch.float32) + 2.7)
    weight = weight[torch.randperm(V, generator=g, device="cuda")]
    t = torch.multinomial(weight, case["T"], replacement=True, generator=g).to(torch.int32)
    return torch.where(_some(case["T"], case["left"], g), -1, t)


def prepare(case, seed):
    g = _gen(seed)
    op, T, H = case["op"], case["T"], case["H"]
    dtype = DTYPES[case["dtype"]]
    s = dict(case=case)
    if op in ("dispatch", "combine", "combine_backward"):
        k, E = case["k"], case["E"]
        # a token's best experts by scores that favour some of them
        score = torch.randn((T, E), generator=g, device="cuda")
        score += 0.4 * torch.randn((E,), generator=g, device="cuda")
        best, expert = score.topk(k, dim=1)
        out = _some(T, case["left"], g).unsqueeze(1)
        s["expert"] = torch.where(out, -1, expert).to(torch.int32)
        if op == "dispatch":
            s["X"] = _randn((T, H), g, dtype)
            return s
        s["slot_row"], s["row_end"] = _sorted(s["expert"], E)
        s["Y"] = _randn((T * k, H), g, dtype)
        if op == "combine_backward" or case["weighted"]:
            s["weight"] = best.softmax(1)
        if op == "combine_backward":
            s["dout"] = _randn((T, H), g, DTYPES[case["out"]], 1e-3)
        elif case["residual"]:
            s["residual"] = _randn((T, H), g, DTYPES[case["out"]])
        return s
    if op in ("embed", "embed_backward"):
        s["tokens"] = _tokens(case, g)
        s["scale"] = math.sqrt(H)
        if op == "embed":
            s["table"] = _randn((case["V"], H), g, dtype, 0.02)
        else:
            s["dX"] = _randn((T, H), g, dtype, 1e-3)
        return s
    V, k = case["V"], case["k"]
    W = _randn((V, H), g, dtype, 0.02)
    # the teacher's best: a few tokens are among them almost everywhere
    score = -torch.log(torch.arange(V, device="cuda", dtype=torch.float32) + 2.7)
    score = score[torch.randperm(V, generator=g, device="cuda")]
    teacher, index = torch.randn((T, V), generator=g, device="cuda").mul_(2.0).add_(score).topk(k, dim=1)
    # a student that leans to its teacher's first choice in half of the rows
    X = _randn((T, H), g, torch.float32)
    lean = (torch.rand((T, 1), generator=g, device="cuda") < 0.5).float() * 5.0
    rows = W[index[:, 0]].float()
    X += lean * rows / rows.norm(dim=1, keepdim=True)
    out = _some(T, case["left"], g)
    s["X"] = X.to(dtype)
    s["W"] = W if case["by_vocab"] else W.t().contiguous()
    s["index"] = torch.where(out.unsqueeze(1), -1, index).to(torch.int32)
    s["teacher"] = teacher
    s["dloss"] = torch.where(out, 0.0, case["temperature"] ** 2 / (T - out.sum()).float())
    return s


# ---- the plain forms -------------------------------------------------------------
def _sorted(expert, E):
    """(row of each slot, ends of the experts' rows) of the slots sorted by expert."""
    key = expert.flatten().long()
    key = torch.where((key >= 0) & (key < E), key, E)
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=order.device)
    ends = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    return row.to(torch.int32).view(expert.shape), ends.to(torch.int32)


def _plain_dispatch(s):
    expert, X, E = s["expert"], s["X"], s["case"]["E"]
    row, ends = _sorted(expert, E)
    kept = (expert >= 0) & (expert < E)
    Xs = X.new_zeros((expert.numel(), X.shape[1]))
    Xs[row.flatten().long()] = torch.where(kept.unsqueeze(2), X.unsqueeze(1), 0).flatten(0, 1)
    return dict(Xs=Xs, row_end=ends, slot_row=row)


def _slots(s):
    """A token's rows of Y, in 32 bits, and which of them an expert has made."""
    row = s["slot_row"].long()
    kept = row < s["row_end"][-1]
    return torch.where(kept.unsqueeze(2), s["Y"][row].float(), 0.0), kept, row


def _plain_combine(s):
    rows, _, _ = _slots(s)
    if "weight" in s:
        rows *= s["weight"].unsqueeze(2)
    out = rows.sum(1)
    if "residual" in s:
        out += s["residual"].float()
    return out.to(DTYPES[s["case"]["out"]])


def _plain_combine_backward(s):
    rows, kept, row = _slots(s)
    d = s["dout"].float().unsqueeze(1)
    weight = torch.where(kept, s["weight"], 0.0)
    dY = torch.empty(s["Y"].shape, dtype=s["dout"].dtype, device=d.device)
    dY[row.flatten()] = (weight.unsqueeze(2) * d).flatten(0, 1).to(dY.dtype)
    return dict(dY=dY, dweight=(rows * d).sum(2))


def _plain_embed(s):
    case, t = s["case"], s["tokens"].long()
    kept = (t >= 0) & (t < case["V"])
    if case["op"] == "embed":
        rows = s["table"][torch.where(kept, t, 0)].float() * s["scale"]
        return torch.where(kept.unsqueeze(1), rows, 0.0).to(s["table"].dtype)
    d = torch.zeros((case["V"], case["H"]), dtype=torch.float32, device=t.device)
    d.index_add_(0, torch.where(kept, t, 0), torch.where(kept.unsqueeze(1), s["dX"].float(), 0.0))
    return (d * s["scale"]).to(s["dX"].dtype)


def _plain_distill(s):
    case, X, index = s["case"], s["X"].float(), s["index"].long()
    W = s["W"].float().t() if case["by_vocab"] else s["W"].float()
    tau = case["temperature"]
    kept = (index >= 0) & (index < case["V"])
    some = kept.any(1)
    at = torch.where(kept, index, 0)
    u = torch.where(kept, s["teacher"] / tau, -math.inf)
    u = u - torch.where(some, u.amax(1), 0.0).unsqueeze(1)
    logp = u - u.exp().sum(1, keepdim=True).log()
    p = torch.where(kept, logp.exp(), 0.0)
    z = X @ W / tau
    top = z.amax(1, keepdim=True)
    lse = top + (z - top).exp().sum(1, keepdim=True).log()
    loss = torch.where(kept, p * (logp - (z.gather(1, at) - lse)), 0.0).sum(1)
    if case["op"] == "distill":
        return dict(loss=loss, lse=lse.squeeze(1))
    G = (z - lse).exp()
    G.scatter_add_(1, at, -p)
    G *= torch.where(some, s["dloss"] / tau, 0.0).unsqueeze(1)
    dX = G @ W.t()
    dW = G.t() @ X if case["by_vocab"] else X.t() @ G
    return dict(loss=loss, lse=lse.squeeze(1), dX=dX.to(s["X"].dtype), dW=dW.to(s["W"].dtype))


PLAIN = dict(dispatch=_plain_dispatch, combine=_plain_combine, combine_backward=_plain_combine_backward,
             embed=_plain_embed, embed_backward=_plain_embed, distill=_plain_distill,
             distill_train=_plain_distill)


def _run_own(s):
    import quantized_linear_layer_amd as ql
    case, op = s["case"], s["case"]["op"]
    if op == "dispatch":
        Xs, row_end, slot_row = ql.experts_dispatch(s["X"], s["expert"], case["E"])
        return dict(Xs=Xs, row_end=row_end, slot_row=slot_row)
    if op == "combine":
        return ql.experts_combine(s["Y"], s["slot_row"], s["row_end"], weight=s.get("weight"),
                                  residual=s.get("residual"), out_dtype=DTYPES[case["out"]])
    if op == "combine_backward":
        dY, dweight = ql.experts_combine_backward(s["dout"], s["Y"], s["slot_row"], s["row_end"], s["weight"])
        return dict(dY=dY, dweight=dweight)
    if op == "embed":
        return ql.embed(s["table"], s["tokens"], scale=s["scale"])
    if op == "embed_backward":
        return ql.embed_backward(s["dX"], s["tokens"], case["V"], scale=s["scale"])
    by = dict(temperature=case["temperature"], by_vocab=case["by_vocab"])
    loss, lse = ql.head_distill(s["X"], s["W"], s["index"], s["teacher"], **by)
    if op == "distill":
        return dict(loss=loss, lse=lse)
    dX, dW = ql.head_distill_backward(s["X"], s["W"], s["index"], s["teacher"], lse, s["dloss"], **by)
    return dict(loss=loss, lse=lse, dX=dX, dW=dW)


def run(s):
    return _run_own(s) if own else PLAIN[s["case"]["op"]](s)


# ---- what a pass cannot do without --------------------------------------------------
def work(case):
    op, T, H = case["op"], case["T"], case["H"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op in ("dispatch", "combine", "combine_backward"):
        M = T * case["k"]
        if op == "dispatch":
            return dict(bytes=(T + M) * H * size + 8 * M + 4 * case["E"], flops=0)
        out = 2 if case["out"] == "bf16" else 4
        if op == "combine":
            return dict(bytes=M * (H * size + 4 + 4 * case["weighted"]) + (1 + case["residual"]) * T * H * out,
                        flops=(1 + case["weighted"]) * M * H)
        return dict(bytes=M * H * (size + out) + T * H * out + 12 * M, flops=3 * M * H)
    if op in ("embed", "embed_backward"):
        rows = T if op == "embed" else case["V"]
        return dict(bytes=(T + rows) * H * size + 4 * T, flops=T * H + (rows * H if op == "embed_backward" else 0))
    V, k = case["V"], case["k"]
    once = (T * H + H * V) * size
    if op == "distill":
        return dict(bytes=once + 8 * T * k + 8 * T, flops=2 * T * H * V)
    return dict(bytes=2 * once + 8 * T * k + 12 * T, flops=6 * T * H * V)


# ---- the same in 64 bits ------------------------------------------------------------
def _exact_routes(case, s):
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    expert = s["expert"].cpu().flatten().tolist()
    here = [[] for _ in range(E)]
    behind = []
    for slot, e in enumerate(expert):
        (here[e] if 0 <= e < E else behind).append(slot)
    order, ends = [], []
    for slots in here:
        order += slots
        ends.append(len(order))
    n = len(order)
    order = torch.tensor(order + behind, dtype=torch.int64, device="cuda")
    row = torch.zeros(T * k, dtype=torch.int64, device="cuda").scatter_(
        0, order, torch.arange(T * k, device="cuda")).view(T, k)
    if op == "dispatch":
        Xs = s["X"].double()[order // k]
        Xs[n:] = 0.0
        return dict(Xs=Xs, row_end=torch.tensor(ends, dtype=torch.int32, device="cuda"), slot_row=row.to(torch.int32))
    H = case["H"]
    if op == "combine":
        out = s["residual"].double() if "residual" in s else torch.zeros((T, H), dtype=torch.float64, device="cuda")
        for j in range(k):
            w = s["weight"][:, j].double() if "weight" in s else torch.ones(T, dtype=torch.float64, device="cuda")
            made = row[:, j] < n
            out[made] = out[made] + w[made, None] * s["Y"][row[made, j]].double()
        return out
    d = s["dout"].double()
    dY = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
    dweight = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        made = (row[:, j] < n).nonzero().squeeze(1)
        at = row[made, j]
        dY[at] = s["weight"][made, j].double()[:, None] * d[made]
        dweight[made, j] = torch.einsum("th,th->t", d[made], s["Y"][at].double())
    return dict(dY=dY, dweight=dweight)


def _exact_embed(case, s):
    tokens = s["tokens"].long()
    made = ((tokens >= 0) & (tokens < case["V"])).nonzero().squeeze(1)
    if case["op"] == "embed":
        out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
        out[made] = s["table"].double()[tokens[made]] * s["scale"]
        return out
    d = torch.zeros((case["V"], case["H"]), dtype=torch.float64, device="cuda")
    return d.index_add_(0, tokens[made], s["scale"] * s["dX"].double()[made])


def _exact_distill(case, s):
    X = s["X"].double()
    W = s["W"].double().t() if case["by_vocab"] else s["W"].double()
    T, V = case["T"], case["V"]
    z = (X @ W) / case["temperature"]
    lse = torch.logsumexp(z, 1)
    # the teacher's distribution over the whole vocabulary
    P = torch.zeros((T, V), dtype=torch.float64, device="cuda")
    made = (s["index"] >= 0) & (s["index"] < V)
    rows = torch.arange(T, device="cuda").unsqueeze(1).expand_as(made)[made]
    u = s["teacher"].double() / case["temperature"]
    e = torch.exp(u - u.max(dim=1, keepdim=True).values) * made
    some = made.any(1)
    p = e / torch.where(some, e.sum(1), 1.0).unsqueeze(1)
    P.index_put_((rows, s["index"][made].long()), p[made], accumulate=True)
    loss = (torch.special.xlogy(p, p).sum(1) - (P * z).sum(1) + lse) * some
    if case["op"] == "distill":
        return dict(loss=loss, lse=lse)
    G = torch.softmax(z, 1) - P
    G *= (s["dloss"].double() / case["temperature"] * some).unsqueeze(1)
    dW = X.t() @ G
    return dict(loss=loss, lse=lse, dX=G @ W.t(), dW=dW.t() if case["by_vocab"] else dW)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("embed", "embed_backward"):
        return _exact_embed(case, s)
    if case["op"] in ("distill", "distill_train"):
        return _exact_distill(case, s)
    return _exact_routes(case, s)
