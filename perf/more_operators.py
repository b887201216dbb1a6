"""Operators of a routed layer whose matrices are served in 8-bit integers: a router by groups of experts with its
gradient, the quantiser of the rows, and the products with scales for each row (token) and column (channel), dense and
of experts.

  route        logits (T, E) -> scores by sigmoid or softmax, a bias that only the choice sees, the best groups of
               experts kept, the k best experts among them, weights; and the pairs' order by expert
  route_grad   the gradient of the weights with respect to the logits
  quant        rows (M, K) -> codes in -127 .. 127 and a scale for each row
  gemm         A's codes times B's, summed as whole numbers, times A's row scale and B's row scale
  up           gathered rows times their expert's gate and up matrices, silu(gate) * up applied on the way out
  product      gathered rows times their expert's matrix

Where `own` is false, `run` computes them in elementary torch operations.
"""
import math

import torch

own = False

# ---------------------------------------------------------------- the cases


def listed():
    return [
        # one token of one user: everything is latency
        dict(name="route_token", op="route", T=1, E=256, k=8, groups=8, kept=4, best=2, scores="sigmoid", dtype="f32",
             bias=True, renorm=True, scale=2.5, pad=0.0),
        # a training step's tokens, a sixteenth of them padding that no expert takes
        dict(name="route_train", op="route", T=16384, E=256, k=8, groups=8, kept=4, best=2, scores="sigmoid",
             dtype="f32", bias=True, renorm=True, scale=2.5, pad=0.0625),
        # the way back, an expert count that is no power of two, logits as a bf16 product leaves them
        dict(name="route_grad", op="route_grad", T=16384, E=160, k=6, groups=8, kept=3, best=1, scores="sigmoid",
             dtype="bf16", bias=False, renorm=True, scale=1.0, pad=0.0),
        # the rows of a decoding batch, in front of every product
        dict(name="quant_decode", op="quant", M=48, K=4096, dtype="bf16"),
        # the rows of a long prompt
        dict(name="quant_prompt", op="quant", M=32768, K=4096, dtype="bf16"),
        # one token: the matrix is read once
        dict(name="gemm_token", op="gemm", M=1, N=8192, K=8192, dtype="bf16"),
        # a decoding batch
        dict(name="gemm_decode", op="gemm", M=48, N=8192, K=4096, dtype="bf16"),
        # a prompt and a matrix of no round sizes, fp32 results (a head's logits)
        dict(name="gemm_prompt", op="gemm", M=2047, N=4102, K=4112, dtype="f32"),
        # the square product of the benchmark
        dict(name="gemm_8192", op="gemm", M=8192, N=8192, K=8192, dtype="bf16"),
        # one token's experts: the matrices of k experts are read once
        dict(name="up_token", op="up", T=1, E=64, k=8, K=2048, F=1408, skew=0.5, pad=0.0),
        # a decoding batch: a few rows for most of the experts
        dict(name="up_decode", op="up", T=48, E=128, k=8, K=4096, F=768, skew=0.5, pad=0.0),
        # a prompt of no round length over the experts' way back
        dict(name="product_prompt", op="product", T=8191, E=32, k=4, K=4096, N=2056, skew=0.3, pad=0.0),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


# the largest listed case's products and bytes
_MOST_FLOPS = 2 * 8192 ** 3
_MOST_BYTES = 7e8


def draw(rng):
    while True:
        op = rng.choice(["route", "route", "route_grad", "quant", "quant", "gemm", "gemm", "gemm", "up", "up", "product",
                         "product"])
        skew, pad = round(rng.uniform(0.0, 1.0), 2), rng.choice([0.0, 0.0, 0.1])
        if op in ("route", "route_grad"):
            groups = rng.choice([1, 2, 4, 8])
            E = groups * _log_int(rng, 4, 512 // groups)
            kept = rng.randint(1, groups)
            scores = rng.choice(["sigmoid", "sigmoid", "softmax"])
            case = dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, min(8, kept * E // groups)), groups=groups,
                        kept=kept, best=rng.randint(1, 2), scores=scores, dtype=rng.choice(["f32", "bf16"]),
                        bias=rng.random() < 0.7, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), pad=pad)
        elif op == "quant":
            case = dict(op=op, M=_log_int(rng, 1, 65536), K=_log_int(rng, 64, 16384, 16),
                        dtype=rng.choice(["bf16", "bf16", "f32"]))
        elif op == "gemm":
            case = dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 64, 16384), K=_log_int(rng, 128, 16384, 16),
                        dtype=rng.choice(["bf16", "bf16", "f32"]))
        else:
            E = _log_int(rng, 4, 256)
            case = dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)), K=_log_int(rng, 256, 4096, 16),
                        skew=skew, pad=pad)
            if op == "up":
                case["F"] = _log_int(rng, 128, 2048)
            else:
                case["N"] = _log_int(rng, 256, 4096)
        w = work(case)
        if w["flops"] <= _MOST_FLOPS and w["bytes"] <= _MOST_BYTES:
            return case


# --------------------------------------------------------------- the inputs


def _type(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _logits(case, g):
    """Router logits, some experts liked better than others, padded tokens closed to every expert."""
    T, E = case["T"], case["E"]
    x = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    if case["pad"]:
        x[torch.rand(T, generator=g, device="cuda") < case["pad"]] = -math.inf
    return x.to(_type(case["dtype"]))


def _order(experts, E):
    """offsets (E + 1), rows (pairs), slots (T, k) of the stable order of the pairs by expert; pairs without an
    expert (-1) have no place in it."""
    T, k = experts.shape
    e = experts.reshape(-1).long()
    key = torch.where(e < 0, E, e)
    order = torch.argsort(key, stable=True)
    count = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=e.device)
    offsets[1:] = count.cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=e.device)
    slots = torch.where(e < 0, -1, place).to(torch.int32).view(T, k)
    rows = torch.where(key[order] < E, order // k, -1).to(torch.int32)
    return offsets, rows, slots


def _codes(g, *shape):
    """Codes as a quantiser leaves them: normal values whose row's largest lies about four deviations out."""
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x.mul_(127 / 4).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda") * 0.02 + 0.005


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("route", "route_grad"):
        s["logits"] = _logits(case, g)
        s["bias"] = torch.randn(case["E"], generator=g, device="cuda") * 0.1 if case["bias"] else None
        if op == "route_grad":
            s["experts"] = _choose(s, case)[0]
            s["dweights"] = torch.randn(case["T"], case["k"], generator=g, device="cuda")
    elif op == "quant":
        x = torch.randn(case["M"], case["K"], generator=g, device="cuda", dtype=_type(case["dtype"]))
        # some channels are far larger than the others, as they are in a model's hidden states
        x[:, torch.rand(case["K"], generator=g, device="cuda") < 0.01] *= 8
        s["x"] = x
    elif op == "gemm":
        s["A"], s["sA"] = _codes(g, case["M"], case["K"]), _scales(g, case["M"])
        s["B"], s["sB"] = _codes(g, case["N"], case["K"]), _scales(g, case["N"])
    else:
        N = 2 * case["F"] if op == "up" else case["N"]
        logits = torch.randn(case["T"], case["E"], generator=g, device="cuda")
        logits += case["skew"] * torch.randn(case["E"], generator=g, device="cuda")
        if case["pad"]:
            logits[torch.rand(case["T"], generator=g, device="cuda") < case["pad"]] = -math.inf
        value, index = logits.sort(dim=1, descending=True, stable=True)
        value, index = value[:, : case["k"]], index[:, : case["k"]]
        s["offsets"], s["rows"], _ = _order(torch.where(value > -math.inf, index, -1), case["E"])
        s["X"], s["sX"] = _codes(g, case["T"], case["K"]), _scales(g, case["T"])
        s["W"] = _codes(g, case["E"], N, case["K"])
        s["sW"] = _scales(g, case["E"], N) * (0.2 / math.sqrt(case["K"]))
    return s


# ----------------------------------------------------------- the operators


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import dense_block_scaled_amd as dbs

    c = s["case"]
    op = c["op"]
    if op == "route":
        return tuple(dbs.moe_route_grouped(s["logits"], c["k"], bias=s["bias"], groups=c["groups"], kept_groups=c["kept"],
                                           group_best=c["best"], scores=c["scores"], renormalize=c["renorm"],
                                           scale=c["scale"]))
    if op == "route_grad":
        return dbs.moe_route_grouped_backward(s["logits"], s["experts"], s["dweights"], scores=c["scores"],
                                              renormalize=c["renorm"], scale=c["scale"])
    if op == "quant":
        return dbs.quant_i8(s["x"])
    if op == "gemm":
        return dbs.gemm_i8(s["A"], s["sA"], s["B"], s["sB"], out_dtype=_type(c["dtype"]))
    if op == "up":
        return dbs.gemm_moe_swiglu_i8(s["X"], s["sX"], s["W"], s["sW"], s["offsets"], s["rows"])
    return dbs.gemm_moe_i8(s["X"], s["sX"], s["W"], s["sW"], s["offsets"], s["rows"])


def _plain(s):
    c = s["case"]
    return globals()["_plain_" + c["op"]](s, c)


def _choose(s, c):
    """experts (T, k; -1: none) and their scores.  In 64 bits: neighbours in the order may be close."""
    x = s["logits"].double()
    T, E, G = c["T"], c["E"], c["groups"]
    open_ = x > -math.inf
    if c["scores"] == "sigmoid":
        score = torch.sigmoid(x)
    else:
        top = torch.where(open_, x, -math.inf).amax(1, keepdim=True)
        part = torch.where(open_, (x - torch.where(top > -math.inf, top, 0.0)).exp(), 0.0)
        score = part / part.sum(1, keepdim=True).clamp(min=1e-300)
    by = score if s["bias"] is None else score + s["bias"].double()
    by = torch.where(open_, by, -math.inf).view(T, G, E // G)
    if c["kept"] < G:
        best = by.sort(dim=2, descending=True).values[:, :, : c["best"]]
        there = best > -math.inf
        group = torch.where(there.any(2), torch.where(there, best, 0.0).sum(2), -math.inf)
        order = group.sort(dim=1, descending=True, stable=True).indices[:, : c["kept"]]
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, order, True)
        by = torch.where(keep[:, :, None], by, -math.inf)
    value, index = by.reshape(T, E).sort(dim=1, descending=True, stable=True)
    value, index = value[:, : c["k"]], index[:, : c["k"]]
    chosen = value > -math.inf
    return torch.where(chosen, index, -1).to(torch.int32).contiguous(), torch.where(chosen, score.gather(1, index), 0.0)


def _plain_route(s, c):
    experts, w = _choose(s, c)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    offsets, rows, slots = _order(experts, c["E"])
    return experts, (w * c["scale"]).float(), offsets, rows, slots


def _plain_route_grad(s, c):
    x = s["logits"].float()
    chosen = s["experts"] >= 0
    index = s["experts"].long().clamp(min=0)
    u = torch.where(chosen, s["dweights"], 0.0) * c["scale"]
    at = torch.gather(x, 1, index)
    if c["scores"] == "sigmoid":
        score = torch.where(chosen, torch.sigmoid(at), 0.0)
        if c["renorm"]:
            w = score / score.sum(1, keepdim=True).clamp(min=1e-30)
            d = w * (u - (w * u).sum(1, keepdim=True)) * torch.sigmoid(-at)
        else:
            d = u * score * torch.sigmoid(-at)
        dx = torch.zeros_like(x).scatter_add_(1, index, torch.where(chosen, d, 0.0))
    elif c["renorm"]:
        top = torch.where(chosen, at, -math.inf).amax(1, keepdim=True)
        part = torch.where(chosen, (at - torch.where(top > -math.inf, top, 0.0)).exp(), 0.0)
        w = torch.where(chosen, part / part.sum(1, keepdim=True), 0.0)
        dx = torch.zeros_like(x).scatter_add_(1, index, w * (u - (w * u).sum(1, keepdim=True)))
    else:
        top = x.amax(1, keepdim=True)
        open_ = top > -math.inf
        part = (x - torch.where(open_, top, 0.0)).exp()
        p = torch.where(open_, part / part.sum(1, keepdim=True), 0.0)
        dense = torch.zeros_like(x).scatter_add_(1, index, u)
        dx = p * (dense - (p * dense).sum(1, keepdim=True))
    return dx.to(s["logits"].dtype)


def _plain_quant(s, c):
    # in 64 bits: codes next to a border between two
    x = s["x"].double()
    most = x.abs().amax(1, keepdim=True)
    codes = torch.where(most > 0, (x * 127 / most).round(), 0.0)
    return codes.to(torch.int8), (most[:, 0] / 127).float()


def _plain_gemm(s, c):
    sums = s["A"].float() @ s["B"].float().t()
    return (sums * s["sA"][:, None] * s["sB"]).to(_type(c["dtype"]))


def _sums(s):
    """Every sorted row's whole-number product with its expert's matrix times the scales, fp32, and which rows an
    expert owns: the groups padded to the longest of them, so that one batched product does."""
    off = s["offsets"].long()
    count = off.diff()
    longest = int(count.max())
    line = torch.arange(longest, device=off.device)
    taken = line < count[:, None]
    at = torch.where(taken, off[:-1, None] + line, 0)
    rows = s["rows"].long()[at].clamp(min=0)
    x = s["X"][rows].float() * s["sX"][rows][..., None]
    h = torch.bmm(x, s["W"].float().transpose(1, 2)) * s["sW"][:, None, :]
    return h[taken], at[taken]


def _plain_up(s, c):
    h, at = _sums(s)
    gate, up = h[:, : c["F"]], h[:, c["F"]:]
    out = torch.zeros(c["T"] * c["k"], c["F"], dtype=torch.bfloat16, device="cuda")
    out[at] = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16)
    return out


def _plain_product(s, c):
    h, at = _sums(s)
    out = torch.zeros(c["T"] * c["k"], c["N"], dtype=torch.bfloat16, device="cuda")
    out[at] = h.to(torch.bfloat16)
    return out


# -------------------------------------------------------- what a pass needs


def work(case):
    op = case["op"]
    item = {"f32": 4, "bf16": 2}[case.get("dtype", "bf16")]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        if op == "route":
            return dict(bytes=T * E * item + T * k * 16 + (E + 1) * 4, flops=T * E * 5)
        # the sigmoid's gradient and the renormalised softmax's need the chosen logits alone
        read = T * k * item if case["scores"] == "sigmoid" or case["renorm"] else T * E * item
        return dict(bytes=read + T * E * item + T * k * 8, flops=T * k * 10)
    if op == "quant":
        n = case["M"] * case["K"]
        return dict(bytes=n * (item + 1) + 4 * case["M"], flops=3 * n)
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=M * K + N * K + 4 * (M + N) + item * M * N, flops=2 * M * N * K)
    T, E, k, K = case["T"], case["E"], case["k"], case["K"]
    tokens = T * (1 - case["pad"])
    pairs = tokens * k
    met = E * (1 - (1 - k / E) ** tokens)      # experts that some token goes to
    N = 2 * case["F"] if op == "up" else case["N"]
    out = case["F"] if op == "up" else N
    return dict(bytes=T * K + met * N * (K + 4) + 2 * T * k * out + 8 * T * k, flops=2 * pairs * N * K)


# ------------------------------------------------- the definition, 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x = s["logits"].double()
        T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
        low = torch.where(x > -math.inf, x, -1e4)
        if case["scores"] == "sigmoid":
            p = 1 / (1 + torch.exp(-low))
        else:
            p = torch.softmax(low, dim=1)
        c = p.clone() if s["bias"] is None else p + s["bias"].double()
        c[x == -math.inf] = -math.inf
        if case["kept"] < G:
            left = c.clone()
            total = torch.zeros(T, G, dtype=torch.float64, device=x.device)
            for j in range(case["best"]):
                m = left.view(T, G, E // G).max(2)
                total += torch.where(m.values > -math.inf, m.values, 0.0 if j else -math.inf)
                left.view(T, G, E // G).scatter_(2, m.indices[..., None], -math.inf)
            closed = torch.ones(T, G, dtype=torch.bool, device=x.device)
            for j in range(case["kept"]):
                closed.scatter_(1, torch.where(closed, total, -math.inf).max(1).indices[:, None], False)
            c.view(T, G, E // G)[closed] = -math.inf
        mass = torch.zeros(T, k, dtype=torch.float64, device=x.device)
        for j in range(k):
            best = c.max(1)
            mass[:, j] = torch.where(best.values > -math.inf, p.gather(1, best.indices[:, None])[:, 0], 0.0)
            c.scatter_(1, best.indices[:, None], -math.inf)
        if case["renorm"]:
            total = mass.sum(1, keepdim=True)
            mass = torch.where(total > 0, mass / total, 0.0)
        return (None, mass * case["scale"], None, None, None)
    if op == "route_grad":
        x = s["logits"].double()
        e, dw = s["experts"].long(), s["dweights"].double() * case["scale"]
        sel = torch.zeros_like(x, dtype=torch.bool)
        up = torch.zeros_like(x)
        for j in range(case["k"]):
            t = torch.nonzero(e[:, j] >= 0).flatten()
            sel[t, e[t, j]] = True
            up[t, e[t, j]] = dw[t, j]
        grad = torch.zeros_like(x)
        live = sel.any(1)
        z, u, on = x[live], up[live], sel[live]
        if case["scores"] == "softmax":
            p = torch.softmax(z.masked_fill(~on, -math.inf) if case["renorm"] else z, dim=1)
            grad[live] = p * (u - (p * u).sum(1, keepdim=True))
        else:
            p = torch.where(on, 1 / (1 + torch.exp(-z)), 0.0)
            slope = torch.where(on, torch.exp(-z) / (1 + torch.exp(-z)) ** 2, 0.0)
            if case["renorm"]:
                total = p.sum(1, keepdim=True)
                u = u / total - (u * p).sum(1, keepdim=True) / total ** 2
            grad[live] = u * slope
        return grad
    if op == "quant":
        x = s["x"]
        return None, torch.maximum(x.amax(1), -x.amin(1)).double() / 127
    if op == "gemm":
        d = torch.matmul(s["A"].double(), s["B"].double().t())
        return d.mul_(s["sA"].double()[:, None]).mul_(s["sB"].double())
    counts = s["offsets"].diff().tolist()
    width = case["F"] if op == "up" else case["N"]
    out = torch.zeros(case["T"] * case["k"], width, dtype=torch.float64, device="cuda")
    start = 0
    for e, n in enumerate(counts):
        if n:
            at = s["rows"][start:start + n].long()
            x = s["X"].index_select(0, at).double()
            h = torch.matmul(s["W"][e].double(), x.t().contiguous()).t()
            h = h * s["sX"][at].double()[:, None] * s["sW"][e].double()
            if op == "up":
                h = h[:, :width] * h[:, width:] / (1 + torch.exp(-h[:, :width]))
            out[start:start + n] = h
        start += n
    return out
