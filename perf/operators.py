"""Mixture-of-experts operators on the calls a routed feed-forward layer makes of them, in serving and in training.

A layer of E experts sends every token to its k best experts.  Its operators, in the order of a pass:

  route          logits (T, E) -> experts, weights (T, k), and the order that sorts the T k pairs by expert
  up             gathered rows times their expert's gate and up matrices, silu(gate) * up applied on the way out
  product        gathered rows times their expert's matrix (training keeps the gate's inputs)
  gate           silu(h[:, :F]) * h[:, F:]
  combine        every token's k rows, weighted and summed

and, going back: combine_grad, gate_grad, dx (rows times the transposed matrices), dw (the matrices' gradients) and
route_grad.  Where `own` is false, `run` computes them in elementary torch operations.
"""
import math

import torch

own = False

# ---------------------------------------------------------------- the cases


def listed():
    return [
        # one token of one user: everything is latency
        dict(name="route_token", op="route", T=1, E=64, k=6, dtype="f32", renorm=True, pad=0.0),
        # a training step's tokens, a sixteenth of them padding that no expert takes
        dict(name="route_train", op="route", T=32768, E=128, k=8, dtype="f32", renorm=True, pad=0.0625),
        # the router's gradient, an expert count that is no power of two, weights as the softmax leaves them
        dict(name="route_grad", op="route_grad", T=16384, E=160, k=6, dtype="bf16", renorm=False, pad=0.0),
        # one token's experts: the weights of k experts are read once
        dict(name="up_token", op="up", T=1, E=64, k=8, K=2048, F=1408, skew=0.5, pad=0.0),
        # a decoding batch: a few rows for most of the experts
        dict(name="up_decode", op="up", T=48, E=128, k=8, K=4096, F=768, skew=0.5, pad=0.0),
        # a prompt of no round length, widths that end inside a tile
        dict(name="product_prompt", op="product", T=4099, E=64, k=6, K=2048, N=1416, skew=0.7, pad=0.0),
        # a training step's products: the rows' gradient and the matrices' gradient
        dict(name="dx_train", op="dx", T=8192, E=32, k=4, K=4096, N=2048, skew=0.3, pad=0.0),
        dict(name="dw_train", op="dw", T=8192, E=32, k=4, N=4096, K=2048, dtype="bf16", skew=0.3, pad=0.0),
        # the gate between the products of a training step, and its gradient
        dict(name="gate_train", op="gate", M=32768, F=2048),
        dict(name="gate_grad_train", op="gate_grad", M=49999, F=1416),
        # the tokens' sums of a training step and their gradient, padding among them
        dict(name="combine_train", op="combine", T=8192, E=64, k=8, H=4096, skew=0.5, pad=0.0, weighted=True),
        dict(name="combine_grad_train", op="combine_grad", T=8191, E=64, k=6, H=2056, skew=0.5, pad=0.0625),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    n = max(lo, min(hi, int(round(v / step)) * step))
    return n + step if n == 3072 else n


# the largest listed case's products and bytes
_MOST_FLOPS = 2 * 32768 * 4096 * 2048
_MOST_BYTES = 1.2e9


def draw(rng):
    while True:
        op = rng.choice(["route", "route_grad", "up", "up", "product", "product", "dx", "dw", "dw", "gate", "gate_grad",
                         "combine", "combine_grad"])
        E = _log_int(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        case = dict(op=op, T=_log_int(rng, 1, 32768), E=E, k=k)
        pad = rng.choice([0.0, 0.0, 0.1])
        skew = round(rng.uniform(0.0, 1.0), 2)
        if op in ("route", "route_grad"):
            case.update(dtype=rng.choice(["f32", "bf16"]), renorm=rng.random() < 0.5, pad=pad)
        elif op == "up":
            case.update(T=_log_int(rng, 1, 4096), K=_log_int(rng, 256, 4096, 8), F=_log_int(rng, 128, 2048, 8),
                        skew=skew, pad=pad)
        elif op in ("product", "dx"):
            case.update(T=_log_int(rng, 1, 16384), K=_log_int(rng, 256, 4096, 8), N=_log_int(rng, 256, 4096, 8),
                        skew=skew, pad=pad)
        elif op == "dw":
            case.update(T=_log_int(rng, 16, 16384), N=_log_int(rng, 256, 4096, 8), K=_log_int(rng, 256, 4096, 8),
                        dtype=rng.choice(["bf16", "f32"]), skew=skew, pad=pad)
        elif op in ("gate", "gate_grad"):
            case = dict(op=op, M=_log_int(rng, 1, 65536), F=_log_int(rng, 128, 2048, 8))
        else:
            case.update(H=_log_int(rng, 256, 4096, 8), skew=skew, pad=pad)
            if op == "combine":
                case["weighted"] = rng.random() < 0.7
        w = work(case)
        if w["flops"] <= _MOST_FLOPS and w["bytes"] <= _MOST_BYTES:
            return case


# --------------------------------------------------------------- the inputs


def _type(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _logits(case, g, dtype, skew=0.0):
    """Router logits: some experts liked better than others, padded tokens closed to every expert."""
    T, E = case["T"], case["E"]
    x = torch.randn(T, E, generator=g, device="cuda")
    if skew:
        x += skew * torch.randn(E, generator=g, device="cuda")
    if case["pad"]:
        x[torch.rand(T, generator=g, device="cuda") < case["pad"]] = -math.inf
    return x.to(dtype)


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


def _routed(case, g):
    logits = _logits(case, g, torch.float32, case["skew"])
    value, index = logits.sort(dim=1, descending=True, stable=True)
    value, index = value[:, : case["k"]], index[:, : case["k"]]
    return _order(torch.where(value > -math.inf, index, -1), case["E"])


def _randn(g, *shape, scale=1.0):
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x.mul_(scale) if scale != 1.0 else x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "route":
        s["logits"] = _logits(case, g, _type(case["dtype"]))
    elif op == "route_grad":
        s["logits"] = _logits(case, g, _type(case["dtype"]))
        value, index = s["logits"].float().sort(dim=1, descending=True, stable=True)
        value, index = value[:, : case["k"]], index[:, : case["k"]]
        s["experts"] = torch.where(value > -math.inf, index, -1).to(torch.int32).contiguous()
        s["dweights"] = torch.randn(case["T"], case["k"], generator=g, device="cuda")
    elif op in ("up", "product"):
        N = 2 * case["F"] if op == "up" else case["N"]
        s["offsets"], s["rows"], _ = _routed(case, g)
        s["X"] = _randn(g, case["T"], case["K"])
        s["W"] = _randn(g, case["E"], N, case["K"], scale=case["K"] ** -0.5)
    elif op == "dx":
        # the gradient of rows that met W (E, K, N): it comes in sorted order already
        s["offsets"], _, _ = _routed(case, g)
        s["X"] = _randn(g, case["T"] * case["k"], case["K"])
        s["W"] = _randn(g, case["E"], case["K"], case["N"], scale=case["K"] ** -0.5)
    elif op == "dw":
        s["offsets"], s["rows"], _ = _routed(case, g)
        s["dY"] = _randn(g, case["T"] * case["k"], case["N"], scale=0.1)
        s["X"] = _randn(g, case["T"], case["K"])
    elif op == "gate":
        s["H"] = _randn(g, case["M"], 2 * case["F"])
    elif op == "gate_grad":
        s["H"] = _randn(g, case["M"], 2 * case["F"])
        s["dA"] = _randn(g, case["M"], case["F"])
    else:
        T, k = case["T"], case["k"]
        s["offsets"], _, s["slots"] = _routed(case, g)
        s["Y"] = _randn(g, T * k, case["H"])
        w = torch.rand(T, k, generator=g, device="cuda") + 0.05
        s["weights"] = w / w.sum(1, keepdim=True) if case.get("weighted", True) else None
        if op == "combine_grad":
            s["dO"] = _randn(g, T, case["H"])
    return s


# ----------------------------------------------------------- the operators


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import dense_block_scaled_amd as dbs

    c = s["case"]
    op = c["op"]
    if op == "route":
        return tuple(dbs.moe_route(s["logits"], c["k"], renormalize=c["renorm"]))
    if op == "route_grad":
        return dbs.moe_route_backward(s["logits"], s["experts"], s["dweights"], renormalize=c["renorm"])
    if op == "up":
        return dbs.gemm_moe_swiglu_bf16(s["X"], s["W"], s["offsets"], s["rows"])
    if op == "product":
        return dbs.gemm_moe_bf16(s["X"], s["W"], s["offsets"], s["rows"])
    if op == "dx":
        return dbs.gemm_moe_bf16(s["X"], s["W"], s["offsets"], lw=dbs.MN_MAJOR)
    if op == "dw":
        return dbs.gemm_moe_dw_bf16(s["dY"], s["X"], s["offsets"], s["rows"], out_dtype=_type(c["dtype"]))
    if op == "gate":
        return dbs.swiglu(s["H"])
    if op == "gate_grad":
        return dbs.swiglu_backward(s["dA"], s["H"])
    if op == "combine":
        return dbs.moe_combine(s["Y"], s["slots"], s["weights"])
    return dbs.moe_combine_backward(s["dO"], s["Y"], s["slots"], s["weights"], s["offsets"])


def _plain(s):
    c = s["case"]
    return globals()["_plain_" + c["op"]](s, c)


def _plain_route(s, c):
    x = s["logits"].float()
    value, index = x.sort(dim=1, descending=True, stable=True)
    value, index = value[:, : c["k"]], index[:, : c["k"]]
    chosen = value > -math.inf
    top = torch.where(chosen[:, :1], value[:, :1], 0.0)
    part = torch.where(chosen, (value - top).exp(), 0.0)
    whole = part.sum(1, keepdim=True) if c["renorm"] else (x - top).exp().sum(1, keepdim=True)
    weights = torch.where(chosen, part / whole, 0.0)
    experts = torch.where(chosen, index, -1).to(torch.int32)
    offsets, rows, slots = _order(experts, c["E"])
    return experts, weights, offsets, rows, slots


def _plain_route_grad(s, c):
    x = s["logits"].float()
    chosen = s["experts"] >= 0
    index = s["experts"].long().clamp(min=0)
    dw = torch.where(chosen, s["dweights"], 0.0)
    at = torch.gather(x, 1, index)
    if c["renorm"]:
        top = torch.where(chosen, at, -math.inf).amax(1, keepdim=True)
        part = torch.where(chosen, (at - torch.where(top > -math.inf, top, 0.0)).exp(), 0.0)
        w = torch.where(chosen, part / part.sum(1, keepdim=True), 0.0)
        dx = torch.zeros_like(x)
        dx.scatter_add_(1, index, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        top = x.amax(1, keepdim=True)
        open_ = top > -math.inf
        part = (x - torch.where(open_, top, 0.0)).exp()
        p = torch.where(open_, part / part.sum(1, keepdim=True), 0.0)
        dense = torch.zeros_like(x)
        dense.scatter_add_(1, index, dw)
        dx = p * (dense - (p * dense).sum(1, keepdim=True))
    return dx.to(s["logits"].dtype)


def _groups(s):
    off = s["offsets"].tolist()
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e + 1] > off[e]]


def _plain_up(s, c):
    F = c["F"]
    out = torch.zeros(c["T"] * c["k"], F, dtype=torch.bfloat16, device="cuda")
    for e, lo, hi in _groups(s):
        h = s["X"][s["rows"][lo:hi]].float() @ s["W"][e].float().t()
        gate, up = h[:, :F], h[:, F:]
        out[lo:hi] = gate * torch.sigmoid(gate) * up
    return out


def _plain_product(s, c):
    out = torch.zeros(c["T"] * c["k"], c["N"], dtype=torch.bfloat16, device="cuda")
    for e, lo, hi in _groups(s):
        out[lo:hi] = s["X"][s["rows"][lo:hi]].float() @ s["W"][e].float().t()
    return out


def _plain_dx(s, c):
    out = torch.zeros(c["T"] * c["k"], c["N"], dtype=torch.bfloat16, device="cuda")
    for e, lo, hi in _groups(s):
        out[lo:hi] = s["X"][lo:hi].float() @ s["W"][e].float()
    return out


def _plain_dw(s, c):
    out = torch.zeros(c["E"], c["N"], c["K"], dtype=_type(c["dtype"]), device="cuda")
    for e, lo, hi in _groups(s):
        out[e] = s["dY"][lo:hi].float().t() @ s["X"][s["rows"][lo:hi]].float()
    return out


def _plain_gate(s, c):
    gate, up = s["H"][:, : c["F"]].float(), s["H"][:, c["F"]:].float()
    return (gate * torch.sigmoid(gate) * up).to(torch.bfloat16)


def _plain_gate_grad(s, c):
    gate, up, da = s["H"][:, : c["F"]].float(), s["H"][:, c["F"]:].float(), s["dA"].float()
    sig = torch.sigmoid(gate)
    dgate = da * up * sig * (1 + gate * (1 - sig))
    return torch.cat([dgate, da * gate * sig], dim=1).to(torch.bfloat16)


def _plain_combine(s, c):
    taken = s["slots"] >= 0
    w = taken.float() if s["weights"] is None else torch.where(taken, s["weights"], 0.0)
    y = s["Y"][s["slots"].clamp(min=0)].float()
    return (w[..., None] * y).sum(1).to(torch.bfloat16)


def _plain_combine_grad(s, c):
    taken = s["slots"] >= 0
    at = s["slots"].clamp(min=0)
    do = s["dO"].float()[:, None, :]
    dweights = torch.where(taken, (do * s["Y"][at].float()).sum(-1), 0.0)
    dY = torch.zeros_like(s["Y"])
    dY[at[taken]] = (s["weights"][..., None] * do).to(torch.bfloat16)[taken]
    return dY, dweights


# -------------------------------------------------------- what a pass needs


def work(case):
    op = case["op"]
    if op in ("gate", "gate_grad"):
        n = case["M"] * case["F"]
        return dict(bytes=2 * n * (3 if op == "gate" else 5), flops=n * (5 if op == "gate" else 10))
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        item = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=T * E * item + T * k * 16 + (E + 1) * 4, flops=T * E * 3)
    if op == "route_grad":
        item = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=2 * T * E * item + T * k * 8, flops=T * E * 6)
    tokens = T * (1 - case["pad"])
    pairs = tokens * k
    if op in ("combine", "combine_grad"):
        H = case["H"]
        if op == "combine":
            return dict(bytes=2 * H * (pairs + T) + 8 * T * k, flops=2 * pairs * H)
        return dict(bytes=2 * H * (T + pairs + T * k) + 12 * T * k, flops=3 * pairs * H)
    met = E * (1 - (1 - k / E) ** tokens)      # experts that some token goes to
    K, N = case["K"], 2 * case["F"] if op == "up" else case["N"]
    if op == "dw":
        item = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=2 * (pairs * N + T * K) + item * E * N * K + 4 * T * k, flops=2 * pairs * N * K)
    out = case["F"] if op == "up" else N
    first = pairs if op == "dx" else T
    return dict(bytes=2 * (first * K + met * N * K + T * k * out) + 4 * T * k, flops=2 * pairs * N * K)


# ------------------------------------------------- the definition, 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x = s["logits"].double()
        T, E = x.shape
        k = case["k"]
        left = x.clone()
        experts = torch.full((T, k), -1, dtype=torch.int32, device=x.device)
        mass = torch.zeros(T, k, dtype=torch.float64, device=x.device)
        high = x.max(1).values
        line = torch.arange(E, device=x.device)
        for j in range(k):
            best = left.max(1).values
            first = torch.where(left == best[:, None], line, E).min(1).values    # ties: the lowest index
            there = best > -math.inf
            experts[there, j] = first[there].to(torch.int32)
            mass[there, j] = torch.exp(best[there] - high[there])
            left[there, first[there]] = -math.inf
        if case["renorm"]:
            total = mass.sum(1)
        else:
            total = torch.where(high > -math.inf, torch.exp(x - high[:, None]).sum(1), 0.0)
        weights = torch.where(experts >= 0, mass / total[:, None], 0.0)
        return (None, weights, None, None, None)
    if op == "route_grad":
        x = s["logits"].double()
        grad = torch.zeros_like(x)
        e, dw = s["experts"].long(), s["dweights"].double()
        sel = torch.zeros_like(x, dtype=torch.bool)
        up = torch.zeros_like(x)
        for j in range(case["k"]):
            t = torch.nonzero(e[:, j] >= 0).flatten()
            sel[t, e[t, j]] = True
            up[t, e[t, j]] = dw[t, j]
        live = sel.any(1)
        z = x.masked_fill(~sel, -math.inf) if case["renorm"] else x
        p = torch.softmax(z[live], dim=1)
        u = up[live]
        grad[live] = p * (u - (p * u).sum(1, keepdim=True))
        return grad
    if op in ("gate", "gate_grad"):
        F = case["F"]
        a, b = s["H"].double().split(F, dim=1)
        e = 1 + torch.exp(-a)
        if op == "gate":
            return a * b / e
        d = s["dA"].double()
        return torch.cat([d * b * (e + a * (e - 1)) / (e * e), d * a / e], 1)
    if op in ("combine", "combine_grad"):
        T, k, H = case["T"], case["k"], case["H"]
        Y, at = s["Y"], s["slots"].long()
        if op == "combine":
            out = torch.zeros(T, H, dtype=torch.float64, device=Y.device)
            for j in range(k):
                t = torch.nonzero(at[:, j] >= 0).flatten()
                w = 1.0 if s["weights"] is None else s["weights"][t, j].double()[:, None]
                out[t] += w * Y[at[t, j]].double()
            return out
        dY = torch.zeros(T * k, H, dtype=torch.float64, device=Y.device)
        dw = torch.zeros(T, k, dtype=torch.float64, device=Y.device)
        for j in range(k):
            t = torch.nonzero(at[:, j] >= 0).flatten()
            do = s["dO"][t].double()
            dY[at[t, j]] = s["weights"][t, j].double()[:, None] * do
            dw[t, j] = (do * Y[at[t, j]].double()).sum(1)
        return dY, dw
    counts = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    start = 0
    if op == "dw":
        out = torch.zeros(case["E"], case["N"], case["K"], dtype=torch.float64, device="cuda")
        for e, n in enumerate(counts):
            if n:
                x = s["X"].index_select(0, s["rows"][start:start + n]).double()
                out[e] = torch.matmul(x.t().contiguous(), s["dY"][start:start + n].double()).t()
            start += n
        return out
    width = case["F"] if op == "up" else case["N"]
    out = torch.zeros(case["T"] * case["k"], width, dtype=torch.float64, device="cuda")
    for e, n in enumerate(counts):
        if n:
            if op == "dx":
                out[start:start + n] = torch.matmul(s["X"][start:start + n].double(), s["W"][e].double())
            else:
                x = s["X"].index_select(0, s["rows"][start:start + n]).double()
                h = torch.matmul(s["W"][e].double(), x.t().contiguous()).t()
                if op == "up":
                    h = h[:, :width] * h[:, width:] / (1 + torch.exp(-h[:, :width]))
                out[start:start + n] = h
        start += n
    return out
