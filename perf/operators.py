"""Cases of the operators around the expert-parallel shuffle that a Mixture-of-Experts layer computes.

router        gate logits -> the k experts of each token and their combine weights (and the
              gradient of the logits)
dispatch_grad the gradient of the dispatch: a token's row is the sum of its receive rows' gradients
combine_grad  the gradient of the combine: of the expert outputs and of the combine weights
experts       every expert's matrix product on its segment of the receive rows, with bias,
              activation (plain or gated) and residual in the epilogue
experts_grad  its gradient: of the rows, the weights and the bias

A case holds the sizes T (tokens), E (experts), k (experts a token), R (virtual ranks), G (ranks a
node), H (row width) and, for the experts, N (output width).  Receive rows are ordered by (expert,
token), so an expert's rows are consecutive.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GATED = ("swiglu", "geglu")


def listed():
    return [
        # One decode step of 16 sequences under node-limited sigmoid routing with a balancing
        # bias (the DeepSeek-V3-like workload's experts, nodes and top-k): launch latency.
        dict(name="router decode", op="router", T=16, E=256, k=8, R=64, G=8, score="sigmoid",
             renormalise=True, scale=2.5, bias=True, nodes=4, dtype="f32", grad=False),
        # The DeepSeek-V3-like training batch's router, forward and gradient.
        dict(name="router train", op="router", T=16384, E=256, k=8, R=64, G=8, score="softmax",
             renormalise=True, scale=1.0, bias=False, nodes=4, dtype="f32", grad=True),
        # The non-divisible workload's experts with bf16 logits (ties are common) and weights
        # normalised over all experts; an odd number of tokens.
        dict(name="router ragged bf16", op="router", T=4099, E=100, k=6, R=7, G=7, score="softmax",
             renormalise=False, scale=1.0, bias=False, nodes=0, dtype="bf16", grad=True),
        # The tiny shuffle's gradient: latency.
        dict(name="dispatch grad tiny", op="dispatch_grad", T=128, E=8, k=2, R=2, G=2, H=256,
             zipf=0.0, dtype="bf16"),
        # The non-divisible expert-parallel batch (100 experts on 7 ranks).
        dict(name="dispatch grad nondiv", op="dispatch_grad", T=32768, E=100, k=6, R=7, G=7, H=2048,
             zipf=0.0, dtype="bf16"),
        # The OLMoE-like batch's combine gradient, with the float32 output's gradient.
        dict(name="combine grad f32", op="combine_grad", T=4096, E=64, k=8, R=4, G=4, H=2048,
             zipf=0.0, dtype="f32"),
        # The DeepSeek-V3-like batch's.
        dict(name="combine grad large", op="combine_grad", T=16384, E=256, k=8, R=64, G=64, H=7168,
             zipf=0.0, dtype="bf16"),
        # One decode step of 16 sequences through the gated first product of OLMoE-like experts:
        # bound by reading the weights.
        dict(name="experts decode", op="experts", T=16, E=64, k=8, R=4, G=4, H=2048, N=1024,
             act="swiglu", bias=False, residual=False, pre=False, zipf=0.0),
        # The same product on the OLMoE-like prefill batch, keeping what the gradient needs.
        dict(name="experts prefill", op="experts", T=4096, E=64, k=8, R=4, G=4, H=2048, N=1024,
             act="swiglu", bias=False, residual=False, pre=True, zipf=0.0),
        # The second product on the Qwen3-like batch under Zipf popularity (one expert takes
        # nearly every token, others a handful), with bias and residual.
        dict(name="experts zipf", op="experts", T=8192, E=128, k=8, R=8, G=8, H=1024, N=4096,
             act="none", bias=True, residual=True, pre=False, zipf=1.2),
        # The gradient of the prefill product: one training step's backward.
        dict(name="experts grad", op="experts_grad", T=4096, E=64, k=8, R=4, G=4, H=2048, N=1024,
             act="swiglu", bias=False, zipf=0.0, dtype="bf16"),
        # Odd sizes: rows that end inside every tile, widths that no tile divides.
        dict(name="experts grad ragged", op="experts_grad", T=1021, E=30, k=4, R=8, G=2, H=776, N=1000,
             act="gelu", bias=True, zipf=0.0, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "dispatch_grad", "combine_grad", "experts", "experts_grad"])
    E = _log_int(rng, 4, 256)
    c = dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, min(8, E)))
    c["R"] = rng.randint(1, min(E, 16))
    c["G"] = c["R"]
    if op == "router":
        score = rng.choice(["softmax", "sigmoid"])
        c["k"] = max(c["k"], 2)  # the renormalised weight of a single expert is a constant
        c.update(score=score, renormalise=rng.random() < 0.6, scale=round(rng.uniform(0.5, 2.5), 3),
                 bias=rng.random() < 0.5, nodes=0, dtype=rng.choice(["f32", "bf16"]),
                 grad=rng.random() < 0.6)
        if E % 4 == 0 and rng.random() < 0.4:  # four nodes, at most two a token
            c.update(R=4, G=1, k=min(c["k"], E // 2), nodes=2)
        return c
    c.update(H=8 * _log_int(rng, 8, 896), zipf=rng.choice([0.0, 0.0, 0.6, 1.2]))
    if op in ("dispatch_grad", "combine_grad"):
        c["dtype"] = rng.choice(["f32", "bf16"])
    else:
        act = rng.choice(["none", "relu", "silu", "gelu", "swiglu", "geglu"])
        c.update(N=8 * _log_int(rng, 8, 512), act=act, bias=rng.random() < 0.5)
        if op == "experts":
            c.update(residual=rng.random() < 0.4, pre=act != "none" and rng.random() < 0.5)
        else:
            # float32 weight gradients where the rows' gradient is not rounded on the way
            c["dtype"] = rng.choice(["f32", "bf16"]) if act == "none" else "bf16"
    most = {}
    for x in listed():
        w = work(x)
        most = {m: max(most.get(m, 0), w[m]) for m in w}
    while c["T"] > 1 or c["H"] > 64:  # a batch that costs no more than the largest listed one
        w = work(c)
        if all(w[m] <= most[m] for m in w):
            break
        if c["T"] > 1:
            c["T"] = (c["T"] * 3) // 4
        else:
            c["H"] = 8 * max(8, c["H"] // 16)
    return c


def _device():
    return torch.device("cuda", torch.cuda.current_device())


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * scale).to(dtype)


def _routing(s, c, g):
    """A routing as a router gives it, and the receive layout that it implies."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = _normal(g, (T, E))
    if c["zipf"]:
        logits = logits - c["zipf"] * torch.log(torch.arange(1, E + 1, device=g.device))
    top = torch.topk(logits, k, dim=1)
    s["topk_idx"] = top.indices.to(torch.int32).contiguous()
    s["topk_w"] = torch.softmax(top.values, 1).contiguous()
    order = torch.sort(s["topk_idx"].reshape(-1), stable=True).indices
    s["slot_of"] = torch.empty_like(order)
    s["slot_of"][order] = torch.arange(T * k, device=g.device)
    s["slot_of"] = s["slot_of"].reshape(T, k)
    s["rows_of"] = torch.bincount(s["topk_idx"].reshape(-1).long(), minlength=E).tolist()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    s = dict(c)
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "router":
        s["logits"] = _normal(g, (T, E), DTYPES[c["dtype"]], 1.5)
        s["bias"] = _normal(g, (E,), scale=0.3) if c["bias"] else None
        s["grad_w"] = _normal(g, (T, k)) if c["grad"] else None
    else:
        _routing(s, c, g)
        rows, H = T * k, c["H"]
        if c["op"] == "dispatch_grad":
            s["grad_recv"] = _normal(g, (rows, H), torch.bfloat16)
        elif c["op"] == "combine_grad":
            s["y"] = _normal(g, (rows, H), torch.bfloat16)
            s["grad_out"] = _normal(g, (T, H), DTYPES[c["dtype"]])
        else:
            N = c["N"]
            Z = 2 * N if c["act"] in GATED else N   # width of the product itself
            s["x"] = _normal(g, (rows, H), torch.bfloat16)
            s["w"] = torch.empty((E, Z, H), dtype=torch.bfloat16, device=g.device)
            s["w"].normal_(0.0, 1.0 / math.sqrt(H), generator=g)
            s["b"] = _normal(g, (E, Z), torch.float32, 0.5) if c["bias"] else None
            if c["op"] == "experts":
                s["residual"] = _normal(g, (rows, N), torch.bfloat16) if c["residual"] else None
            else:
                s["grad_y"] = _normal(g, (rows, N), torch.bfloat16)
                s["pre"] = _normal(g, (rows, Z), torch.bfloat16) if c["act"] != "none" else None
    if own:
        # The plan is the handle that a program keeps for a routing: the shuffle's calls need it too.
        import combine_shuffling_amd as cs

        s["plan"] = cs.Plan(T, c.get("H", 8), E, k, c["R"], c["G"])
        if c["op"] != "router":
            s["plan"].route(s["topk_idx"])
    return s


# ---- the framework's calls

def _run_own(s):
    p = s["plan"]
    if s["op"] == "router":
        how = dict(score=s["score"], renormalise=s["renormalise"], scale=s["scale"])
        idx, w = p.router(s["logits"], bias=s["bias"], nodes_per_token=s["nodes"], **how)
        if s["grad_w"] is None:
            return {"idx": idx, "w": w}
        return {"idx": idx, "w": w,
                "grad_logits": p.router_backward(s["logits"], idx, s["grad_w"], **how)}
    if s["op"] == "dispatch_grad":
        return {"grad_x": p.dispatch_backward(s["grad_recv"], out_dtype=DTYPES[s["dtype"]])}
    if s["op"] == "combine_grad":
        grad_y, grad_w = p.combine_backward(s["grad_out"], s["y"], s["topk_w"])
        return {"grad_y": grad_y, "grad_w": grad_w}
    if s["op"] == "experts":
        y, pre = p.expert_linear(s["x"], s["w"], bias=s["b"], residual=s["residual"],
                                 activation=s["act"], save_pre=s["pre"])
        return {"y": y, "pre": pre}
    grad_x, grad_w, grad_b = p.expert_linear_backward(
        s["grad_y"], s["x"], s["w"], pre=s["pre"], activation=s["act"],
        bias_grad=s["b"] is not None, grad_w_dtype=DTYPES[s["dtype"]])
    return {"grad_x": grad_x, "grad_w": grad_w, "grad_b": grad_b}


# ---- the plain form

def _select(s, key):
    """The k largest keys of a row, the lowest index first among equal ones; only experts of the
    `nodes` best nodes (by the sum of a node's two largest keys) where that is limited."""
    if s["nodes"]:
        per = s["E"] // (s["R"] // s["G"])
        by_node = key.reshape(s["T"], -1, per)
        best = torch.sort(by_node, dim=2, descending=True).values[:, :, :2].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : s["nodes"]]
        out = torch.ones_like(best, dtype=torch.bool).scatter_(1, kept, False)
        key = by_node.masked_fill(out[:, :, None], -math.inf).reshape(key.shape)
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, : s["k"]]


def _router(s):
    x = s["logits"].float()
    ids = _select(s, x if s["bias"] is None else x + s["bias"])
    if s["score"] == "softmax":
        p = torch.exp(x - x.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    q = p.gather(1, ids)
    total = q.sum(1, keepdim=True) if s["renormalise"] else torch.ones_like(q[:, :1])
    w = s["scale"] * q / total
    out = {"idx": ids.to(torch.int32), "w": w}
    if s["grad_w"] is not None:
        d = s["grad_w"] * s["scale"] / total       # of the selected scores
        if s["renormalise"]:
            d = d - (d * q / total).sum(1, keepdim=True)
        d = torch.zeros_like(p).scatter(1, ids, d)  # of all scores
        if s["score"] == "softmax":
            d = p * (d - (p * d).sum(1, keepdim=True))
        else:
            d = d * p * (1 - p)
        out["grad_logits"] = d.to(s["logits"].dtype)
    return out


def _erf_cdf(z):
    return 0.5 * (1 + torch.erf(z / math.sqrt(2.0)))


def _act(kind, z):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind in ("silu", "swiglu"):
        return z / (1 + torch.exp(-z))
    if kind in ("gelu", "geglu"):
        return z * _erf_cdf(z)
    return z


def _act_slope(kind, z):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind in ("silu", "swiglu"):
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if kind in ("gelu", "geglu"):
        return _erf_cdf(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _parts(s, t):
    return torch.split(t, s["rows_of"])


def _run_plain(s):
    if s["op"] == "router":
        return _router(s)
    rows = s["slot_of"]
    if s["op"] == "dispatch_grad":
        g = s["grad_recv"][rows.reshape(-1)].float().reshape(s["T"], s["k"], -1)
        return {"grad_x": g.sum(1).to(DTYPES[s["dtype"]])}
    if s["op"] == "combine_grad":
        g = s["grad_out"].float()
        token = torch.empty_like(rows.reshape(-1))
        weight = torch.empty_like(s["topk_w"].reshape(-1))
        token[rows.reshape(-1)] = torch.arange(rows.numel(), device=rows.device) // s["k"]
        weight[rows.reshape(-1)] = s["topk_w"].reshape(-1)
        by_row = g[token]
        dots = (by_row * s["y"].float()).sum(1)
        grad_y = (by_row * weight[:, None]).to(torch.bfloat16)
        return {"grad_y": grad_y, "grad_w": dots[rows]}
    if s["op"] == "experts":
        z = torch.cat([a.float() @ w.float().t() for a, w in zip(_parts(s, s["x"]), s["w"])])
        if s["b"] is not None:
            z = z + torch.cat([b.expand(n, -1) for b, n in zip(s["b"], s["rows_of"])])
        if s["act"] in GATED:
            y = _act(s["act"], z[:, : s["N"]]) * z[:, s["N"]:]
        else:
            y = _act(s["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(torch.bfloat16), "pre": z.to(torch.bfloat16) if s["pre"] else None}
    g = s["grad_y"].float()
    if s["act"] in GATED:
        gate, up = s["pre"].float().split(s["N"], 1)
        g = torch.cat([g * up * _act_slope(s["act"], gate), g * _act(s["act"], gate)], 1)
    elif s["act"] != "none":
        g = g * _act_slope(s["act"], s["pre"].float())
    gs = _parts(s, g)
    grad_x = torch.cat([a @ w.float() for a, w in zip(gs, s["w"])]).to(torch.bfloat16)
    grad_w = torch.stack([(a.t() @ x.float()).to(DTYPES[s["dtype"]])
                          for a, x in zip(gs, _parts(s, s["x"]))])
    grad_b = torch.stack([a.sum(0) for a in gs]) if s["b"] is not None else None
    return {"grad_x": grad_x, "grad_w": grad_w, "grad_b": grad_b}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without

def work(case):
    c = case
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "router":
        size = 4 if c["dtype"] == "f32" else 2
        b = T * E * size + T * k * 8 + (4 * E if c["bias"] else 0)
        f = T * E * (4 + k)
        if c["grad"]:
            b += T * k * 4 + T * E * size
            f += 6 * T * E
        return {"bytes": b, "flops": f}
    rows, H = T * k, c["H"]
    if c["op"] == "dispatch_grad":
        return {"bytes": rows * H * 2 + T * H * (4 if c["dtype"] == "f32" else 2) + rows * 4,
                "flops": rows * H}
    if c["op"] == "combine_grad":
        return {"bytes": 2 * rows * H * 2 + T * H * (4 if c["dtype"] == "f32" else 2) + rows * 12,
                "flops": 3 * rows * H}
    N = c["N"]
    Z = 2 * N if c["act"] in GATED else N
    hit = min(E, rows) if c["zipf"] else E * (1 - (1 - k / E) ** T)  # experts with rows, on average
    bias = 4 * E * Z if c["bias"] else 0
    if c["op"] == "experts":
        b = rows * H * 2 + hit * Z * H * 2 + rows * N * 2 + bias
        b += (rows * N * 2 if c["residual"] else 0) + (rows * Z * 2 if c["pre"] else 0)
        return {"bytes": b, "flops": 2.0 * rows * H * Z}
    b = rows * N * 2 + 2 * rows * H * 2 + hit * Z * H * 2 + bias
    b += E * Z * H * (4 if c["dtype"] == "f32" else 2) + (rows * Z * 2 if c["act"] != "none" else 0)
    return {"bytes": b, "flops": 4.0 * rows * H * Z}


# ---- the definition, in 64 bits

def _exact_router(s):
    x = s["logits"].double()
    key = s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]  # float32 by definition
    T, E, k = s["T"], s["E"], s["k"]
    index = torch.arange(E, device=x.device)
    ids = torch.empty((T, k), dtype=torch.long, device=x.device)
    for t0 in range(0, T, 512):
        q = key[t0: t0 + 512].clone()
        if s["nodes"]:
            n = s["R"] // s["G"]
            v = q.reshape(q.shape[0], n, E // n)
            m1 = v.max(2)
            rest = v.scatter(2, m1.indices[:, :, None], -math.inf).max(2).values
            best = m1.values + (rest if E // n > 1 else 0)
            at = torch.arange(n, device=x.device)
            ahead = (best[:, None, :] > best[:, :, None]) | \
                ((best[:, None, :] == best[:, :, None]) & (at[None, None, :] < at[None, :, None]))
            q = torch.where((ahead.sum(2) < s["nodes"]).repeat_interleave(E // n, 1), q, -math.inf)
        ahead = (q[:, None, :] > q[:, :, None]) | \
            ((q[:, None, :] == q[:, :, None]) & (index[None, None, :] < index[None, :, None]))
        place = ahead.sum(2)
        for j in range(k):
            ids[t0: t0 + 512, j] = (place == j).to(torch.uint8).argmax(1)
    if s["score"] == "softmax":
        p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    else:
        p = torch.sigmoid(x)
    one = torch.zeros_like(p).scatter(1, ids, 1.0)
    S = (p * one).sum(1, keepdim=True) if s["renormalise"] else torch.ones_like(p[:, :1])
    w = s["scale"] * p.gather(1, ids) / S
    out = {"idx": None, "w": w}
    if s["grad_w"] is not None:
        gw = torch.zeros_like(p).scatter(1, ids, s["grad_w"].double())
        if s["score"] == "softmax":
            # dw_i / dx_e = w_i (delta_ie - r_e), r the distribution that w is drawn from
            r = p * one / S if s["renormalise"] else p
            a = gw * s["scale"] * p * one / S
            out["grad_logits"] = a - r * a.sum(1, keepdim=True)
        else:
            a = gw * s["scale"] / S
            if s["renormalise"]:
                a = a - (gw * s["scale"] * p * one).sum(1, keepdim=True) / S ** 2
            out["grad_logits"] = one * a * p * (1 - p)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "router":
        return _exact_router(s)
    T, E, k = s["T"], s["E"], s["k"]
    expert = s["topk_idx"].long()
    if s["op"] == "dispatch_grad":
        total = torch.zeros((T, s["H"]), dtype=torch.float64, device=expert.device)
        for j in range(k):
            total += s["grad_recv"][s["slot_of"][:, j]]
        return {"grad_x": total}
    if s["op"] == "combine_grad":
        g = s["grad_out"].double()
        grad_y = torch.empty(s["y"].shape, dtype=torch.float64, device=g.device)
        grad_w = torch.empty((T, k), dtype=torch.float64, device=g.device)
        for j in range(k):
            at = s["slot_of"][:, j]
            grad_y[at] = s["topk_w"][:, j: j + 1].double() * g
            grad_w[:, j] = torch.linalg.vecdot(g, s["y"][at].double())
        return {"grad_y": grad_y, "grad_w": grad_w}
    of_row = torch.sort(expert.reshape(-1)).values
    N, H, dev = s["N"], s["H"], of_row.device
    Z = s["w"].shape[1]
    Phi = lambda z: torch.special.ndtr(z)  # noqa: E731
    sig = torch.sigmoid
    f = {"none": lambda z: z, "relu": torch.relu, "silu": lambda z: z * sig(z),
         "gelu": lambda z: z * Phi(z)}
    df = {"none": torch.ones_like, "relu": lambda z: torch.heaviside(z, torch.zeros_like(z)),
          "silu": lambda z: sig(z) + z * sig(z) * sig(-z),
          "gelu": lambda z: Phi(z) + z * torch.exp(-z.square() / 2) / (2 * np.pi) ** 0.5}
    kind = {"swiglu": "silu", "geglu": "gelu"}.get(s["act"], s["act"])
    if s["op"] == "experts":
        z = torch.zeros((T * k, Z), dtype=torch.float64, device=dev)
        for e in range(E):
            at = (of_row == e).nonzero()[:, 0]
            z[at] = torch.mm(s["x"][at].double(), s["w"][e].double().t().contiguous())
            if s["b"] is not None:
                z[at] += s["b"][e].double()
        y = f[kind](z[:, :N]) * z[:, N:] if Z > N else f[kind](z)
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, "pre": z if s["pre"] else None}
    gy = s["grad_y"].double()
    if s["pre"] is None:
        gz = gy
    else:
        z = s["pre"].double()
        gz = torch.empty((T * k, Z), dtype=torch.float64, device=dev)
        gz[:, :N] = gy * df[kind](z[:, :N]) * (z[:, N:] if Z > N else 1.0)
        if Z > N:
            gz[:, N:] = gy * f[kind](z[:, :N])
    grad_x = torch.zeros((T * k, H), dtype=torch.float64, device=dev)
    grad_w = torch.zeros((E, Z, H), dtype=torch.float64, device=dev)
    grad_b = torch.zeros((E, Z), dtype=torch.float64, device=dev)
    for e in range(E):
        at = (of_row == e).nonzero()[:, 0]
        grad_x[at] = torch.mm(gz[at], s["w"][e].double())
        grad_w[e] = torch.mm(gz[at].t().contiguous(), s["x"][at].double())
        grad_b[e] = gz[at].sum(0)
    return {"grad_x": grad_x, "grad_w": grad_w, "grad_b": grad_b if s["b"] is not None else None}
