"""Cases that measure the experts' products, the head loss and the gradient clipping.

``run`` computes a case in plain torch operations (``own`` false) or with the
calls of ``quantized_linear_layer_amd`` (``own`` true); ``exact`` is the same
from the definition in 64 bits.

Experts' products (op ``forward``, ``dgrad``, ``wgrad``, ``apply``). The rows of
the activations are sorted by expert; expert e owns the rows from
``row_end[e-1]`` (0 for e = 0) up to ``row_end[e]``. Every operand is
quantized in blocks of 32 values along the product's reduction to E2M1 with one
power-of-two scale 2^e, e the least integer with 6 * 2^e >= the block's max,
nearest value, ties away from zero. ``apply`` takes weights quantized before.

Head loss (op ``loss``, ``train``): the cross entropy of the logits X W
against one target a row, with the gradients of X and W in ``train``. Rows
whose target lies outside the vocabulary are left out.

Clipping (op ``clip``): out_i = g_i * min(1, max_norm / (norm + 1e-6)) with the
2-norm over all the tensors.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LEFT_OUT = -100


def listed():
    return [
        # one token through its two experts: serving, where latency counts
        dict(name="apply 1 token", op="apply", dtype="bf16", E=8, M=2, K=2048, N=5632, empty=0),
        # a batch of 64 sequences, one new token each, two experts a token
        dict(name="apply 64 tokens", op="apply", dtype="bf16", E=8, M=128, K=4096, N=11008, empty=0),
        # a training step's up projection: 4096 tokens, two experts each
        dict(name="forward 4096x11008", op="forward", dtype="bf16", E=8, M=8192, K=4096, N=11008, empty=0),
        # the same kind of layer with more, smaller experts: input gradient
        dict(name="dgrad 16 experts", op="dgrad", dtype="bf16", E=16, M=8192, K=2048, N=5632, empty=1),
        # the weight gradient of the large up projection
        dict(name="wgrad 4096x11008", op="wgrad", dtype="bf16", E=8, M=8192, K=4096, N=11008, empty=0),
        # float32, nothing a multiple of anything, one expert without rows
        dict(name="forward odd f32", op="forward", dtype="f32", E=5, M=777, K=515, N=1003, empty=1),
        # scoring the last token of 32 sequences
        dict(name="loss 32 rows", op="loss", dtype="bf16", T=32, H=4096, V=32000, by_vocab=False),
        # a training step of a small model
        dict(name="train 4096x2048", op="train", dtype="bf16", T=4096, H=2048, V=32000, by_vocab=False),
        # a training step of a larger one, the weight shared with the embedding
        dict(name="train 8192x4096 tied", op="train", dtype="bf16", T=8192, H=4096, V=32000, by_vocab=True),
        # float32 and odd sizes
        dict(name="train odd f32", op="train", dtype="f32", T=1001, H=515, V=5003, by_vocab=False),
        # the adapters of a small fine-tuning run: launches are what costs
        dict(name="clip adapters", op="clip", dtype="f32", H=256, F=8, layers=6, max_norm=1.0),
        # the gradients of eight layers of a 2048 x 5632 model
        dict(name="clip 8 layers", op="clip", dtype="bf16", H=2048, F=5632, layers=8, max_norm=1.0),
    ]


def _log(rng, low, high):
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = min(max(v, low), high)
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(("forward", "dgrad", "wgrad", "apply", "loss", "train", "train", "clip"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("forward", "dgrad", "wgrad", "apply"):
        E = _log(rng, 2, 64)
        K, N = _log(rng, 64, 5120), _log(rng, 64, 11008)
        if rng.random() < 0.5:
            K, N = 8 * (-(-K // 8)), 8 * (-(-N // 8))
        while E * K * N > 8 * 4096 * 11008:
            E = max(1, E // 2)
            N = max(64, N - 8) if E == 1 else N
        M = _log(rng, 1, 256) if op == "apply" else _log(rng, 16, 8192)
        return dict(op=op, dtype=dtype, E=E, M=M, K=K, N=N, empty=rng.randrange(0, E // 2 + 1))
    if op in ("loss", "train"):
        T, H, V = _log(rng, 1, 8192), _log(rng, 64, 4096), _log(rng, 1000, 32000)
        if rng.random() < 0.5:
            H, V = 8 * (-(-H // 8)), 8 * (-(-V // 8))
        if dtype == "f32":
            T = min(T, 2048)
        return dict(op=op, dtype=dtype, T=T, H=H, V=V, by_vocab=rng.random() < 0.5)
    return dict(op=op, dtype=dtype, H=_log(rng, 64, 2048), F=_log(rng, 4, 5632), layers=rng.randint(1, 8),
                max_norm=rng.choice((0.1, 1.0, 1000.0)))


# ---- inputs -------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _activations(rows, cols, g, dtype):
    """Normal values with a few far larger channels, as hidden activations have them."""
    x = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    loud = torch.randperm(cols, generator=g, device="cuda")[:max(1, cols // 1000)]
    x[:, loud] *= 50.0
    return x.to(dtype)


def _row_counts(case, seed):
    """Rows of each expert: a token picks experts of unequal popularity; `empty` of them get none."""
    g = torch.Generator()
    g.manual_seed(seed)
    E, M = case["E"], case["M"]
    weight = torch.exp(0.4 * torch.randn(E, generator=g))
    weight[torch.randperm(E, generator=g)[:case["empty"]]] = 0.0
    picks = torch.multinomial(weight, M, replacement=True, generator=g)
    return torch.bincount(picks, minlength=E)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    dtype = DTYPES[case["dtype"]]
    s = dict(case=case)
    if op in ("forward", "dgrad", "wgrad", "apply"):
        E, M, K, N = case["E"], case["M"], case["K"], case["N"]
        counts = _row_counts(case, seed)
        s["row_end"] = counts.cumsum(0).to(torch.int32).cuda()
        s["most"] = int(counts.max())
        if op in ("forward", "apply", "wgrad"):
            s["A"] = _activations(M, K, g, dtype)
        if op in ("dgrad", "wgrad"):
            s["dY"] = _randn((M, N), g, dtype, 1e-3)
        if op in ("forward", "dgrad"):
            s["W"] = _randn((E, K, N), g, dtype, 0.02)
        if op == "apply":  # the weights as a checkpoint of them holds them
            s["Wq"], s["Ws"] = _packed(_randn((E, K, N), g, dtype, 0.02))
        return s
    if op in ("loss", "train"):
        T, H, V = case["T"], case["H"], case["V"]
        W = _randn((V, H), g, dtype, 0.02)
        targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        # hidden states, half of them leaning to their target's row as in a trained model
        X = _randn((T, H), g, torch.float32)
        lean = (torch.rand((T, 1), generator=g, device="cuda") < 0.5).float() * 5.0
        rows = W[targets.long()].float()
        X += lean * rows / rows.norm(dim=1, keepdim=True)
        # a tenth of the rows carry no loss (prompt or padding), never all of them
        out = torch.rand((T,), generator=g, device="cuda") < 0.1
        out[0] = False
        s["X"] = X.to(dtype)
        s["W"] = W if case["by_vocab"] else W.t().contiguous()
        s["targets"] = torch.where(out, LEFT_OUT, targets)
        s["dloss"] = torch.where(out, 0.0, 1.0 / (T - out.sum()).float())
        return s
    H, F, layers = case["H"], case["F"], case["layers"]
    shapes = [(H, H), (H, F), (H, F), (F, H), (H,), (H,), (F,)] * layers
    s["grads"] = [_randn(shape, g, torch.float32 if len(shape) == 1 else dtype, 2e-3) for shape in shapes]
    s["out"] = [torch.empty_like(t) for t in s["grads"]]
    return s


# ---- the plain forms -------------------------------------------------------------
def _blocks(x, n):
    """x with its last axis cut in blocks of 32, zeros added to a multiple of n."""
    pad = -x.shape[-1] % n
    x = torch.nn.functional.pad(x.float(), (0, pad))
    return x.unflatten(-1, (-1, 32))


def _quantized(x, n=32):
    """(index, exponent) of each value and block along the last axis of x."""
    b = _blocks(x, n)
    mantissa, power = torch.frexp(b.abs().amax(-1))
    e = torch.where(mantissa <= 0.75, power - 3, power - 2)
    e = torch.where(mantissa == 0, -127, e).clamp(min=-127).int()
    y = b.abs() * _power(-e).unsqueeze(-1)
    index = torch.bucketize(y, torch.tensor(MIDS, device=x.device), right=True)
    return index + 8 * torch.signbit(b), e


def _power(e):
    """2^e in 32 bits."""
    bits = torch.where(e > -127, (e + 127) << 23, 1 << 22)
    return bits.int().view(torch.float32)


def _values(index, e):
    grid = torch.tensor(GRID, device=index.device)
    v = torch.cat((grid, -grid))[index] * _power(e).unsqueeze(-1)
    return v.flatten(-2)


def _q(x):
    """x quantized along its last axis, as the values that the codes stand for."""
    return _values(*_quantized(x))[..., :x.shape[-1]]


def _packed(W):
    """W (E, K, N) as codes (E, N, K/2 rounded up to 64) and scale bytes (K/128 rounded up, E, N, 4)."""
    index, e = _quantized(W.transpose(1, 2), 128)
    index = index.flatten(-2).to(torch.uint8)
    codes = index[..., 0::2] | (index[..., 1::2] << 4)
    scales = (e + 127).to(torch.uint8).unflatten(-1, (-1, 4)).permute(2, 0, 1, 3)
    return codes.contiguous(), scales.contiguous()


def _unpacked(Wq, Ws, K):
    index = torch.stack((Wq & 15, Wq >> 4), -1).flatten(-2).unflatten(-1, (-1, 32)).long()
    e = Ws.permute(1, 2, 0, 3).flatten(-2).int() - 127
    return _values(index, e)[..., :K]


def _by_expert(x, row_end, most):
    """x's rows as (expert, place, column), with zeros after an expert's last row; and where each row is."""
    E = row_end.numel()
    row = torch.arange(x.shape[0], device=x.device)
    expert = torch.bucketize(row, row_end.long(), right=True)
    begin = torch.nn.functional.pad(row_end.long(), (1, -1))
    place = row - begin[expert]
    out = torch.zeros((E, most, x.shape[1]), dtype=torch.float32, device=x.device)
    out[expert, place] = x.float()
    return out, (expert, place)


def _plain_experts(s):
    op, row_end, most = s["case"]["op"], s["row_end"], s["most"]
    if op == "wgrad":
        A, _ = _by_expert(s["A"], row_end, most)
        dY, _ = _by_expert(s["dY"], row_end, most)
        return torch.bmm(_q(A.transpose(1, 2)), _q(dY.transpose(1, 2)).transpose(1, 2).contiguous())
    x = s["dY"] if op == "dgrad" else s["A"]
    if op == "apply":
        B = _unpacked(s["Wq"], s["Ws"], s["case"]["K"])
    else:
        B = _q(s["W"] if op == "dgrad" else s["W"].transpose(1, 2))
    x, at = _by_expert(_q(x), row_end, most)
    return torch.bmm(x, B.transpose(1, 2).contiguous())[at]


def _plain_head(s):
    case, X, targets = s["case"], s["X"].float(), s["targets"].long()
    W = s["W"].float().t() if case["by_vocab"] else s["W"].float()
    keep = (targets >= 0) & (targets < case["V"])
    at = torch.where(keep, targets, 0).unsqueeze(1)
    logits = X @ W
    top = logits.amax(1, keepdim=True)
    lse = top + (logits - top).exp().sum(1, keepdim=True).log()
    loss = torch.where(keep, (lse - logits.gather(1, at)).squeeze(1), 0.0)
    if case["op"] == "loss":
        return dict(loss=loss, lse=lse.squeeze(1))
    G = (logits - lse).exp()
    G.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    G *= torch.where(keep, s["dloss"], 0.0).unsqueeze(1)
    dX = G @ W.t()
    dW = G.t() @ X if case["by_vocab"] else X.t() @ G
    return dict(loss=loss, lse=lse.squeeze(1), dX=dX.to(s["X"].dtype), dW=dW.to(s["W"].dtype))


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    c = (s["case"]["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return dict(norm=norm, grads=[(g.float() * c).to(g.dtype) for g in s["grads"]])


def _run_own(s):
    import quantized_linear_layer_amd as ql
    case, op = s["case"], s["case"]["op"]
    if op == "forward":
        return ql.experts_forward_mx(s["A"], s["W"], s["row_end"])
    if op == "dgrad":
        return ql.experts_dgrad_mx(s["dY"], s["W"], s["row_end"])
    if op == "wgrad":
        return ql.experts_wgrad_mx(s["A"], s["dY"], s["row_end"])
    if op == "apply":
        return ql.experts_apply_mx(s["A"], s["Wq"], s["Ws"], s["row_end"])
    if op in ("loss", "train"):
        loss, lse = ql.head_loss(s["X"], s["W"], s["targets"], by_vocab=case["by_vocab"])
        if op == "loss":
            return dict(loss=loss, lse=lse)
        dX, dW = ql.head_loss_backward(s["X"], s["W"], s["targets"], lse, s["dloss"], by_vocab=case["by_vocab"])
        return dict(loss=loss, lse=lse, dX=dX, dW=dW)
    norm = ql.clip_grads(s["grads"], case["max_norm"], out=s["out"])
    return dict(norm=norm, grads=s["out"])


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op in ("loss", "train"):
        return _plain_head(s)
    return _plain_clip(s) if op == "clip" else _plain_experts(s)


# ---- what a pass cannot do without --------------------------------------------------
def work(case):
    op = case["op"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op in ("forward", "dgrad", "wgrad", "apply"):
        E, M, K, N = case["E"], case["M"], case["K"], case["N"]
        busy = min(E - case["empty"], M)
        flops = 2 * M * K * N
        if op == "apply":  # codes and scales of the experts that can have rows
            return dict(bytes=busy * K * N * 17 / 32 + M * K * size + 4 * M * N, flops=flops)
        if op == "wgrad":
            return dict(bytes=M * (K + N) * size + 4 * E * K * N, flops=flops)
        rows, cols = (K, N) if op == "forward" else (N, K)
        return dict(bytes=busy * K * N * size + M * rows * size + 4 * M * cols, flops=flops)
    if op in ("loss", "train"):
        T, H, V = case["T"], case["H"], case["V"]
        once = (T * H + H * V) * size
        if op == "loss":
            return dict(bytes=once + 12 * T, flops=2 * T * H * V)
        return dict(bytes=2 * once + 16 * T, flops=6 * T * H * V)
    H, F, layers = case["H"], case["F"], case["layers"]
    big, small = layers * (H * H + 3 * H * F), layers * (2 * H + F)
    return dict(bytes=2 * (size * big + 4 * small), flops=3 * (big + small))


# ---- the same in 64 bits ------------------------------------------------------------
def _q64(x, dim):
    """x quantized in blocks of 32 along dim, from the definition."""
    x = x.double().movedim(dim, -1)
    n = x.shape[-1]
    whole = torch.zeros(x.shape[:-1] + (32 * (-(-n // 32)),), dtype=torch.float64, device=x.device)
    whole[..., :n] = x
    b = whole.reshape(whole.shape[:-1] + (-1, 32))
    most = b.abs().max(dim=-1, keepdim=True).values
    # the least e >= -127 with 6 * 2^e >= most: the power of two at or above most / 6
    m, p = torch.frexp(most / 6.0)
    e = torch.where(m == 0.5, p - 1, p).double()
    scale = torch.where(most > 0, torch.ldexp(torch.ones_like(most), e.clamp(min=-127.0)), 2.0 ** -127)
    y = b.abs() / scale
    level = torch.zeros_like(y)
    for low, high in zip(GRID[:-1], GRID[1:]):
        level += (y >= (low + high) / 2) * (high - low)
    return (torch.sign(b) * level * scale).reshape(whole.shape)[..., :n].movedim(-1, dim)


def _exact_experts(case, s):
    op = case["op"]
    ends = s["row_end"].tolist()
    begins = [0] + ends[:-1]
    out = []
    for e, (b, n) in enumerate(zip(begins, ends)):
        if op == "wgrad":
            out.append(_q64(s["A"][b:n], 0).t() @ _q64(s["dY"][b:n], 0) if n > b else
                       torch.zeros((case["K"], case["N"]), dtype=torch.float64, device="cuda"))
        elif n > b:
            if op == "dgrad":
                out.append(_q64(s["dY"][b:n], 1) @ _q64(s["W"][e], 1).t())
            else:
                B = _unpacked64(s["Wq"][e], s["Ws"][:, e], case["K"]) if op == "apply" else _q64(s["W"][e], 0)
                out.append(_q64(s["A"][b:n], 1) @ B)
    return torch.stack(out) if op == "wgrad" else torch.cat(out)


def _unpacked64(codes, scales, K):
    """Codes (N, bytes) and scale bytes (steps, N, 4) of one expert as its K x N weight."""
    rows = codes.shape[0]
    code = torch.empty((rows, 2 * codes.shape[1]), dtype=torch.int64, device="cuda")
    code[:, 0::2] = codes.long() % 16
    code[:, 1::2] = codes.long() // 16
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    value = grid[code % 8] * (1 - 2 * (code // 8)).double()
    power = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), scales.permute(1, 0, 2).reshape(rows, -1).double() - 127.0)
    return (value * power.repeat_interleave(32, dim=1))[:, :K].t()


def _exact_head(case, s):
    X = s["X"].double()
    W = s["W"].double().t() if case["by_vocab"] else s["W"].double()
    T, V = case["T"], case["V"]
    logits = X @ W
    lse = torch.logsumexp(logits, 1)
    keep = (s["targets"] >= 0) & (s["targets"] < V)
    rows = keep.nonzero().squeeze(1)
    cols = s["targets"][rows].long()
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    loss[rows] = lse[rows] - logits[rows, cols]
    if case["op"] == "loss":
        return dict(loss=loss, lse=lse)
    P = torch.softmax(logits, 1)
    P[rows, cols] -= 1.0
    P *= (s["dloss"].double() * keep).unsqueeze(1)
    dW = X.t() @ P
    return dict(loss=loss, lse=lse, dX=P @ W.t(), dW=dW.t() if case["by_vocab"] else dW)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("loss", "train"):
        return _exact_head(case, s)
    if case["op"] != "clip":
        return _exact_experts(case, s)
    norm = math.sqrt(math.fsum(float(g.double().square().sum()) for g in s["grads"]))
    c = min(1.0, case["max_norm"] / (norm + 1e-6))
    return dict(norm=torch.tensor(norm, dtype=torch.float64, device="cuda"), grads=[g.double() * c for g in s["grads"]])
