"""Measured cases of the experts' products in 16 bits and of low-rank adapters.

Five operators, each as a user's program calls it:

  gated        rows times their expert's gate and up matrices, the activation and the product:
               h = act(x Wg^T, x Wu^T), where the program trains with the pre-activations beside it
  gated_grad   its gradients: of the rows and of the matrices, from the gradient of h
  linear       rows times their expert's matrix (the down projection)
  linear_grad  its gradients
  adapter      low-rank products of many requests beside a shared projection, each row with its
               request's adapter: out = base + scale (x A^T) B^T

Rows lie in expert order (the rows of expert e from offsets[e] on); one matrix for all rows is the
shared expert, or any dense projection. Adapters take their rows where they are, through the maps
that sort them.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one token of a decode step through the shared expert
        _experts("gated one token", "gated", 1, 1, 1, 1, 7168, 2048, "bf16", limit=7.0),
        # a 64-token decode step through its experts
        _experts("gated decode", "gated", 64, 896, 896, 16, 3584, 384, "bf16"),
        # the forward pass of a training batch on a quarter of the experts, pre-activations kept
        _experts("gated batch quarter", "gated", 8192, 64, 256, 8, 7168, 2048, "fp16", limit=7.0, save=True),
        # the backward pass of a micro-batch on one half of many small experts, some of them crowded
        _experts("gated grad half", "gated_grad", 4096, 448, 896, 16, 3584, 384, "bf16", act="situ", skew=True),
        # the shared expert's backward pass
        _experts("gated grad shared", "gated_grad", 8192, 1, 1, 1, 7168, 2048, "bf16"),
        # a small model's micro-batch, odd sizes
        _experts("gated grad odd", "gated_grad", 333, 60, 60, 4, 1000, 424, "fp16", limit=7.0),
        # the down projection of the decode step
        _experts("linear decode", "linear", 64, 896, 896, 16, 384, 3584, "bf16"),
        # a long prompt through a dense projection
        _experts("linear prompt", "linear", 8191, 1, 1, 1, 2048, 7168, "fp16"),
        # the down projection's backward pass on a quarter of the experts, matrices' gradients in 32 bits
        _experts("linear grad quarter", "linear_grad", 8192, 64, 256, 8, 2048, 7168, "bf16", out="fp32"),
        # one token with its request's adapter
        _adapters("adapter one token", 1, 4, 16, 7168, 2048, "bf16"),
        # a decode batch, hardly two of whose requests share an adapter
        _adapters("adapter decode", 64, 128, 16, 7168, 7168, "bf16", out="fp32"),
        # prompts of a few requests in one batch
        _adapters("adapter prompts", 8191, 8, 64, 3584, 7168, "bf16", runs=True),
    ]


def _experts(name, op, T, E, experts, topk, K, N, dtype, act="swiglu", limit=0.0, save=False, skew=False, out=None):
    """K: elements of a row; N: those of a row of the result (the gated products have 2 N weight rows).
    out: the type of the result, and in a backward pass that of the matrices' gradients."""
    return {"name": name, "op": op, "T": T, "E": E, "experts": experts, "topk": topk, "K": K, "N": N, "dtype": dtype, "act": act,
            "limit": limit, "save": save, "skew": skew, "out": out or dtype}


def _adapters(name, M, adapters, R, K, N, dtype, runs=False, out=None):
    """runs: a request's rows follow each other (prompts); else every row is a request of its own."""
    return {"name": name, "op": "adapter", "M": M, "adapters": adapters, "R": R, "K": K, "N": N, "dtype": dtype, "runs": runs,
            "out": out or dtype}


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "gated_grad", "linear", "linear_grad", "adapter", "adapter"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    K = 8 * _log(rng, 8, 896)
    if op == "adapter":
        case = _adapters("", _log(rng, 1, 8192), _log(rng, 1, 128), rng.choice([8, 16, 32, 64, 128]), K, rng.choice([_log(rng, 16, 8192), 8 * _log(rng, 8, 896)]),
                         dtype, runs=rng.random() < 0.4, out=rng.choice([dtype, dtype, "fp32"]))
    else:
        N = 8 * _log(rng, 6, 256 if op.startswith("gated") else 896)
        dense = rng.random() < 0.35
        experts = 1 if dense else _log(rng, 4, 896)
        topk = 1 if dense else rng.randint(1, min(16, experts))
        E = experts if experts < 8 else max(1, experts // rng.choice([1, 2, 4]))
        while E * K * N > 1_200_000_000:  # matrices no larger than the listed ones'
            E, experts = max(1, E // 2), max(topk, experts // 2)
        # operations and the plain form's padded rows no more than the listed ones'
        products = 2 * K * N * topk * (2 if op.startswith("gated") else 1) * (2 if op.endswith("grad") else 1)
        T = _log(rng, 1, max(1, min(8192, 900_000_000_000 // products, 8_000_000_000 // (E * (K + 2 * N)))))
        case = _experts("", op, T, E, experts, topk, K, N, dtype, act=rng.choice(["swiglu", "swiglu", "situ"]), limit=rng.choice([0.0, 7.0]),
                        save=op == "gated" and rng.random() < 0.5, skew=rng.random() < 0.4,
                        out=rng.choice([dtype, "fp32"]) if op.startswith("linear") else dtype)
    del case["name"]
    return case


_BETA, _LINEAR_BETA = 4.0, 25.0  # caps of the "situ" activation


def _route(case, g):
    """Distinct ids of each token's experts."""
    logits = torch.randn(case["T"], case["experts"], generator=g, device="cuda")
    if case["skew"]:
        rank = torch.randperm(case["experts"], generator=g, device="cuda").double() + 1
        logits = (logits.double() - 1.1 * rank.log()).float()
    return torch.topk(logits, case["topk"], dim=1).indices


def _normal(g, scale, dtype, *size):
    return (scale * torch.randn(*size, generator=g, device="cuda", dtype=dtype if dtype != torch.float16 else torch.float32)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, dtype, K, N = case["op"], _TYPES[case["dtype"]], case["K"], case["N"]
    st = {"case": case}
    if op == "adapter":
        M, n, R = case["M"], case["adapters"], case["R"]
        # one id of -1, a row without an adapter, for each sixteen others
        ids = torch.randint(0, n, (M,), generator=g, device="cuda")
        ids = torch.where(torch.rand(M, generator=g, device="cuda") < 1 / 16, torch.full_like(ids, -1), ids) if M > 16 else ids
        if case["runs"]:
            first = torch.rand(M, generator=g, device="cuda") < 4 * n / M
            ids = ids[torch.where(first, torch.arange(M, device="cuda"), torch.zeros_like(ids)).cummax(0).values]
        st["ids"] = ids
        st["x"] = _normal(g, 1.0, dtype, M, K)
        st["a"], st["b"] = _normal(g, K ** -0.5, dtype, n, R, K), _normal(g, R ** -0.5, dtype, n, N, R)
        st["scale"] = 0.5 + 1.5 * torch.rand(n, generator=g, device="cuda")
        st["base"] = _normal(g, 1.0, _TYPES[case["out"]], M, N)
        st["out"] = torch.zeros(M, N, dtype=_TYPES[case["out"]], device="cuda")
        # the maps that sort the rows by adapter, made once for a step's layers
        key = torch.where(ids < 0, torch.full_like(ids, n), ids)
        order = torch.argsort(key, stable=True)
        place = torch.empty_like(order)
        place[order] = torch.arange(M, device="cuda")
        st["offsets"] = torch.searchsorted(key[order], torch.arange(n + 1, device="cuda")).to(torch.int32)
        st["row_slot"] = order.to(torch.int32)
        st["slot_row"] = torch.where(ids < 0, torch.full_like(place, -1), place).to(torch.int32)
    else:
        E, gated = case["E"], op.startswith("gated")
        M, rows = case["T"] * case["topk"], (2 if gated else 1) * N
        st["w"] = _normal(g, K ** -0.5, dtype, E, rows, K)
        st["x"] = _normal(g, 1.0, dtype, M, K)
        st["offsets"], st["most"] = None, M
        if case["experts"] > 1:
            local = _route(case, g).reshape(-1) - (case["experts"] - E)
            local = torch.sort(local[local >= 0]).values
            st["offsets"] = torch.searchsorted(local, torch.arange(E + 1, device="cuda")).to(torch.int32)
            st["most"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())  # for the plain form alone
        if op.endswith("grad"):
            st["dout"] = _normal(g, 1.0, dtype, M, N)
            st["dx"] = torch.zeros(M, K, dtype=dtype, device="cuda")
            st["dw"] = torch.zeros(E, rows, K, dtype=_TYPES[case["out"]], device="cuda")
            if gated:  # pre-activations as the forward pass kept them
                st["gu"] = _normal(g, 1.5, dtype, M, 2 * N)
                st["dgu"] = torch.zeros(M, 2 * N, dtype=dtype, device="cuda")
        else:
            st["out"] = torch.zeros(M, N, dtype=_TYPES[case["out"]], device="cuda")
            if gated:
                st["gu"] = torch.zeros(M, 2 * N, dtype=dtype, device="cuda") if case["save"] else None
    if own:
        st.update(_plan(st))
    return st


def _plan(st):
    """What a program of this library's user makes once for a shape."""
    import mxfp4_weight_expert_amd as moe

    c = st["case"]
    if c["op"] == "adapter":
        shape = moe.AdapterShape(M=c["M"], N=c["N"], K=c["K"], R=c["R"], A=c["adapters"], dtype=c["dtype"], out_dtype=c["out"])
        return {"shape": shape, "workspace": torch.empty(moe.adapter_query(shape), dtype=torch.uint8, device="cuda")}
    M = c["T"] * c["topk"]
    if c["op"].startswith("gated"):
        return {"shape": moe.GatedShape(M=M, I=c["N"], H=c["K"], E=c["E"], dtype=c["dtype"], activation=c["act"], swiglu_limit=c["limit"],
                                        act_beta=_BETA, act_linear_beta=_LINEAR_BETA)}
    return {"shape": moe.LinearShape(M=M, N=c["N"], K=c["K"], E=c["E"], dtype=c["dtype"], out_dtype=c["out"])}


def run(st):
    return _own(st) if own else _PLAIN[st["case"]["op"]](st)


def _own(st):
    import mxfp4_weight_expert_amd as moe

    op, shape = st["case"]["op"], st["shape"]
    if op == "gated":
        h = moe.gated_linear(st["x"], st["offsets"], st["w"], shape, out=st["out"], gu=st["gu"])
        return h if st["gu"] is None else (h, st["gu"])
    if op == "gated_grad":
        return moe.gated_linear_backward(st["dout"], st["x"], st["offsets"], st["gu"], st["w"], shape, dx=st["dx"], dw=st["dw"], dgu=st["dgu"])
    if op == "linear":
        return moe.grouped_linear(st["x"], st["offsets"], st["w"], shape, out=st["out"])
    if op == "linear_grad":
        return moe.grouped_linear_backward(st["dout"], st["x"], st["offsets"], st["w"], shape, dx=st["dx"], dw=st["dw"])
    return moe.adapter_linear(st["x"], st["offsets"], st["row_slot"], st["slot_row"], st["a"], st["b"], st["scale"], shape, base=st["base"],
                              out=st["out"], workspace=st["workspace"])


# ------------------------------------------------------------------------------------------ plain forms


def _places(st):
    """(rows' places in [E, most] as one number, one more for rows without an expert; which rows have one)."""
    case, M, most = st["case"], st["x"].shape[0], st["most"]
    row = torch.arange(M, device="cuda")
    if st["offsets"] is None:
        return row, row >= 0
    first = st["offsets"].long()
    expert = (torch.searchsorted(first, row, right=True) - 1).clamp_max(case["E"] - 1)
    live = row < first[-1]
    return torch.where(live, expert * most + row - first[expert], torch.full_like(row, case["E"] * most)), live


def _padded(st, t, at, live):
    """Rows by expert in 32 bits, [E, most, width]; zeros where an expert has fewer."""
    E, most = st["case"]["E"], st["most"]
    out = torch.zeros(E * most + 1, t.shape[1], device="cuda")
    out[at] = torch.where(live[:, None], t.float(), torch.zeros((), device="cuda"))
    return out[:-1].view(E, most, t.shape[1])


def _unpadded(t, at, live, like):
    """Back to rows; rows without an expert stay as they are in `like`."""
    flat = t.reshape(-1, t.shape[2])
    return torch.where(live[:, None], flat[at.clamp_max(flat.shape[0] - 1)].to(like.dtype), like)


def _times_matrices(st, t, at, live):
    return torch.bmm(_padded(st, t, at, live), st["w"].float().transpose(1, 2).contiguous())


def _plain_linear(st):
    at, live = _places(st)
    return _unpadded(_times_matrices(st, st["x"], at, live), at, live, st["out"])


def _activation(case, g, u):
    if case["act"] == "situ":
        return _BETA * torch.tanh(g / _BETA) * torch.sigmoid(g) * (_LINEAR_BETA * torch.tanh(u / _LINEAR_BETA))
    if case["limit"] > 0:
        g, u = g.clamp_max(case["limit"]), u.clamp(-case["limit"], case["limit"])
    return g * torch.sigmoid(g) * u


def _plain_gated(st):
    at, live = _places(st)
    N = st["case"]["N"]
    gu = _times_matrices(st, st["x"], at, live)
    h = _unpadded(_activation(st["case"], gu[..., :N], gu[..., N:]), at, live, st["out"])
    return h if st["gu"] is None else (h, _unpadded(gu, at, live, st["gu"]))


def _gradients(st, dout, at, live):
    """dx and dw of a product from the gradient of its result in 32 bits."""
    d = _padded(st, dout, at, live)
    dx = _unpadded(torch.bmm(d, st["w"].float()), at, live, st["dx"])
    return dx, torch.bmm(d.transpose(1, 2).contiguous(), _padded(st, st["x"], at, live)).to(st["dw"].dtype)


def _plain_linear_grad(st):
    at, live = _places(st)
    return _gradients(st, st["dout"], at, live)


def _plain_gated_grad(st):
    case, N = st["case"], st["case"]["N"]
    at, live = _places(st)
    g, u, dh = st["gu"][:, :N].float(), st["gu"][:, N:].float(), st["dout"].float()
    if case["act"] == "situ":
        s, tg, tu = torch.sigmoid(g), torch.tanh(g / _BETA), torch.tanh(u / _LINEAR_BETA)
        dg = dh * _LINEAR_BETA * tu * s * ((1 - tg * tg) + _BETA * tg * (1 - s))
        du = dh * _BETA * tg * s * (1 - tu * tu)
    else:
        limit = case["limit"] if case["limit"] > 0 else math.inf
        inside_g, inside_u = g <= limit, u.abs() <= limit
        g, u = g.clamp_max(limit), u.clamp(-limit, limit)
        s, zero = torch.sigmoid(g), torch.zeros((), device="cuda")
        dg = torch.where(inside_g, dh * u * s * (1 + g * (1 - s)), zero)
        du = torch.where(inside_u, dh * g * s, zero)
    return _gradients(st, torch.cat([dg, du], 1), at, live)


def _plain_adapter(st):
    case, ids = st["case"], st["ids"]
    n, R = case["adapters"], case["R"]
    t = (st["x"].float() @ st["a"].view(n * R, -1).float().t()).view(-1, n, R)
    mine = torch.arange(n, device="cuda") == ids[:, None]
    t = torch.where(mine[..., None], t * st["scale"][:, None], torch.zeros((), device="cuda"))
    b = st["b"].float().transpose(0, 1).reshape(case["N"], n * R)
    return (st["base"].float() + t.view(-1, n * R) @ b.t()).to(st["out"].dtype)


_PLAIN = {"gated": _plain_gated, "gated_grad": _plain_gated_grad, "linear": _plain_linear, "linear_grad": _plain_linear_grad,
          "adapter": _plain_adapter}


# ------------------------------------------------------------------------------------ work and 64 bits


def work(case):
    op, K, N, size, out = case["op"], case["K"], case["N"], _SIZE[case["dtype"]], _SIZE[case["out"]]
    if op == "adapter":
        M, R, n = case["M"], case["R"], case["adapters"]
        touched = n * (1 - (1 - 1 / n) ** (min(M, 4 * n) if case["runs"] else M))
        return {"bytes": M * (K * size + 2 * N * out + 4) + touched * R * (K + N) * size, "flops": 2 * M * R * (K + N)}
    slots = case["T"] * case["topk"]
    here = slots * case["E"] / case["experts"]  # rows with a local expert, on average
    touched = case["E"] * (1 - (1 - case["topk"] / case["experts"]) ** case["T"])
    matrix = (2 if op.startswith("gated") else 1) * N * K
    if op == "gated":
        return {"bytes": touched * matrix * size + here * (K + (3 if case["save"] else 1) * N) * size, "flops": 2 * here * matrix}
    if op == "linear":
        return {"bytes": touched * matrix * size + here * (K * size + N * out), "flops": 2 * here * matrix}
    rows = here * size * (2 * K + (3 if op == "gated_grad" else 1) * N)  # x, dx, dout, pre-activations
    return {"bytes": touched * matrix * size + case["E"] * matrix * out + rows, "flops": 4 * here * matrix}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adapter":
        return _exact_adapter(case, st)
    E, N, op = case["E"], case["N"], case["op"]
    first = [0, st["x"].shape[0]] if st["offsets"] is None else st["offsets"].tolist()
    zeros = {n: torch.zeros(st[n].shape, dtype=torch.float64, device="cuda") for n in ("out", "gu", "dx", "dw") if st.get(n) is not None}
    for e in range(E):
        lo, hi = first[e], first[e + 1]
        if lo == hi:
            continue
        x, w = st["x"][lo:hi].double(), st["w"][e].double()
        if op == "linear":
            zeros["out"][lo:hi] = x @ w.t()
        elif op == "gated":
            g, u = x @ w[:N].t(), x @ w[N:].t()
            if "gu" in zeros:
                zeros["gu"][lo:hi, :N], zeros["gu"][lo:hi, N:] = g, u
            zeros["out"][lo:hi] = _exact_activation(case, g, u)
        else:
            d = st["dout"][lo:hi].double()
            if op == "gated_grad":
                # the derivative by torch's own differentiation, in 64 bits
                g, u = (st["gu"][lo:hi, i * N : (i + 1) * N].double().requires_grad_() for i in (0, 1))
                d = torch.cat(torch.autograd.grad(_exact_activation(case, g, u), (g, u), d), 1)
            zeros["dx"][lo:hi] = d @ w
            zeros["dw"][e] = d.t() @ x
    if op == "linear":
        return zeros["out"]
    if op == "gated":
        return (zeros["out"], zeros["gu"]) if "gu" in zeros else zeros["out"]
    return zeros["dx"], zeros["dw"]


def _exact_activation(case, g, u):
    if case["act"] == "situ":
        return _BETA * torch.tanh(g / _BETA) / (1 + torch.exp(-g)) * _LINEAR_BETA * torch.tanh(u / _LINEAR_BETA)
    if case["limit"] > 0:
        # values on the border count as inside, for the gradient too
        limit = torch.tensor(case["limit"], dtype=torch.float64, device="cuda")
        g = torch.where(g > limit, limit, g)
        u = torch.where(u > limit, limit, torch.where(u < -limit, -limit, u))
    return g / (1 + torch.exp(-g)) * u


def _exact_adapter(case, st):
    out = st["base"].double()
    for i in range(case["adapters"]):
        rows = (st["ids"] == i).nonzero()[:, 0]
        if rows.numel():
            out[rows] += st["scale"][i].double() * ((st["x"][rows].double() @ st["a"][i].double().t()) @ st["b"][i].double().t())
    return out
