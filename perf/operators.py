"""Measured cases of the expert-routing and 4-bit weight operators.

Four operators, each as a user's program calls it:

  dispatch / dispatch_grad  tokens copied into expert order with the maps there and back, and the
                            gradient of the tokens from the gradient of the sorted rows
  combine / combine_grad    expert rows weighted and summed back to token order, and the gradients
                            of the rows and of the routing weights
  linear                    a few tokens times one 4-bit weight matrix with group scales
  grouped                   the sorted rows times their expert's 4-bit weight matrix

Weights lie in the library's packed layout (blocks of 16 rows x 64 bytes); the two formats are
MXFP4 (E2M1 codes, an E8M0 byte for 32 weights) and INT4 (codes 0..15, a scale in the tokens' type and
optionally a zero point for each group of 32, 64 or 128 weights).
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one decode step of the 64-token layer: maps for 896 experts, where latency counts
        _routing("dispatch decode", "dispatch", 64, 896, 896, 16, 3584, "bf16"),
        # a long prompt through the same layer
        _routing("dispatch prefill", "dispatch", 8192, 896, 896, 16, 3584, "bf16"),
        # the backward of a training micro-batch on one half of the experts
        _routing("dispatch grad half", "dispatch_grad", 4096, 448, 896, 16, 3584, "bf16", skew=True),
        # one decode step, half of the experts elsewhere (their slots hold nothing)
        _routing("combine decode half", "combine", 256, 448, 896, 16, 3584, "bf16", skew=True),
        # a long prompt, wide tokens
        _routing("combine prefill", "combine", 8191, 256, 256, 8, 7168, "fp16"),
        # a small training batch held in 32 bits, an odd width
        _routing("combine grad odd", "combine_grad", 333, 60, 60, 4, 1023, "fp32"),
        # a training micro-batch
        _routing("combine grad batch", "combine_grad", 4096, 256, 256, 8, 7168, "bf16"),
        # a single token through a down projection
        _weights("linear one token", "linear", 1, 1, 7168, 2048, "mxfp4", 32, "bf16"),
        # a batch of sixteen on a square projection, zero points and a bias
        _weights("linear batch", "linear", 16, 1, 8192, 8192, "int4", 128, "fp16", zeros=True, bias=True),
        # a vocabulary's worth of rows for five tokens, scores in 32 bits
        _weights("linear vocabulary", "linear", 5, 1, 129279, 7168, "mxfp4", 32, "bf16", out="fp32"),
        # the gate and up projection of a 64-token decode step
        _weights("grouped decode", "grouped", 64, 896, 768, 3584, "mxfp4", 32, "bf16", topk=16, experts=896),
        # a quarter of 256 wide experts on this GPU, 4-bit integers in groups of 64
        _weights("grouped quarter", "grouped", 128, 64, 4096, 7168, "int4", 64, "bf16", topk=8, experts=256),
    ]


def _routing(name, op, T, E, experts, topk, H, dtype, skew=False):
    return {"name": name, "op": op, "T": T, "E": E, "experts": experts, "topk": topk, "H": H, "dtype": dtype, "skew": skew}


def _weights(name, op, T, E, N, K, fmt, group, dtype, zeros=False, bias=False, out=None, topk=1, experts=1):
    return {"name": name, "op": op, "T": T, "E": E, "N": N, "K": K, "format": fmt, "group": group, "dtype": dtype,
            "zeros": zeros, "bias": bias, "out": out or dtype, "topk": topk, "experts": experts}


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "linear", "linear", "grouped", "grouped"])
    if op in ("linear", "grouped"):
        fmt = rng.choice(["mxfp4", "int4"])
        group = 32 if fmt == "mxfp4" else rng.choice([32, 64, 128])
        dtype = rng.choice(["bf16", "fp16"])
        zeros = fmt == "int4" and rng.random() < 0.5
        more = {"zeros": zeros, "bias": rng.random() < 0.3, "out": rng.choice([dtype, dtype, "fp32"])}
        if op == "linear":
            K = 128 * _log(rng, 1, 64)
            case = _weights("", op, _log(rng, 1, 64), 1, _log(rng, 16, min(129279, 900_000_000 // K)), K, fmt, group, dtype, **more)
        else:
            K = 128 * _log(rng, 1, 56)
            E = _log(rng, 4, 896)
            N = _log(rng, 16, max(16, min(4096, 3_000_000_000 // (K * E))))
            experts = min(896, E * rng.choice([1, 2, 4])) if E > 16 else E
            topk = rng.randint(1, min(16, experts))
            case = _weights("", op, _log(rng, 1, 128), E, N, K, fmt, group, dtype, topk=topk, experts=experts, **more)
    else:
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        experts = _log(rng, 4, 896)
        topk = rng.randint(1, min(16, experts))
        H = rng.choice([_log(rng, 64, 7168), 64 * _log(rng, 1, 112)])
        T = _log(rng, 1, min(8192, 900_000_000 // (topk * H * _SIZE[dtype])))
        case = _routing("", op, T, rng.choice([experts, max(1, experts // 2)]), experts, topk, H, dtype, skew=rng.random() < 0.5)
    del case["name"]
    return case


def _offset(case):
    """Global id of the first local expert: the last share of the experts."""
    return case["experts"] - case["E"]


def _route(case, g):
    """Distinct ids of each token's experts, and weights that sum to one."""
    logits = torch.randn(case["T"], case["experts"], generator=g, device="cuda")
    if case.get("skew"):
        rank = torch.randperm(case["experts"], generator=g, device="cuda").double() + 1
        logits = (logits.double() - 1.1 * rank.log()).float()
    top, ids = torch.topk(logits, case["topk"], dim=1)
    return ids.to(torch.int32), torch.softmax(top, 1)


def _maps(ids, case):
    """For each slot t * topk + k: its row in expert order, or -1; for each row its slot; the experts' first rows."""
    E, slots = case["E"], ids.numel()
    local = ids.reshape(-1).long() - _offset(case)
    here = (local >= 0) & (local < E)
    key = torch.where(here, local, torch.full_like(local, E))
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(slots, device=ids.device)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), counts[:E].cumsum(0)])
    return order, torch.where(here, row, torch.full_like(row, -1)), offsets


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, T, topk, dtype = case["op"], case["T"], case["topk"], _TYPES[case["dtype"]]
    st = {"case": case}
    if op in ("linear", "grouped"):
        E, N, K, group = case["E"], case["N"], case["K"], case["group"]
        up = (N + 15) // 16 * 16
        st["w"] = torch.randint(0, 256, (E, up, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        if case["format"] == "mxfp4":
            st["scales"] = torch.randint(118, 128, (E, N, K // group), generator=g, device="cuda", dtype=torch.uint8)
        else:
            st["scales"] = (0.002 + 0.02 * torch.rand(E, N, K // group, generator=g, device="cuda")).to(dtype)
        st["zeros"] = torch.randint(4, 12, (E, N, K // group), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        st["bias"] = torch.randn(E, N, generator=g, device="cuda").to(dtype) if case["bias"] else None
        rows = T * topk if op == "grouped" else T
        st["x"] = torch.randn(rows, K, generator=g, device="cuda").to(dtype)
        st["out"] = torch.zeros(rows, N, dtype=_TYPES[case["out"]], device="cuda")
        if op == "grouped":
            _, _, offsets = _maps(_route(case, g)[0], case)
            st["offsets"] = offsets.to(torch.int32)
            st["most"] = int((offsets[1:] - offsets[:-1]).max())  # for the plain form alone
    else:
        ids, w = _route(case, g)
        H, slots = case["H"], T * topk
        order, row, _ = _maps(ids, case)
        st["ids"], st["topk_w"], st["slot_row"] = ids, w, row.to(torch.int32).view(T, topk)
        if op == "dispatch":
            st["x"] = torch.randn(T, H, generator=g, device="cuda").to(dtype)
            st["out"] = torch.zeros(slots, H, dtype=dtype, device="cuda")
            st["offsets"] = torch.zeros(case["E"] + 1, dtype=torch.int32, device="cuda")
            st["row_slot"] = torch.zeros(slots, dtype=torch.int32, device="cuda")
            st["slot_row"] = torch.zeros(T, topk, dtype=torch.int32, device="cuda")
        else:
            st["rows"] = torch.randn(slots, H, generator=g, device="cuda").to(dtype)
            if op == "combine_grad":
                st["dout"] = torch.randn(T, H, generator=g, device="cuda").to(dtype)
                st["out"] = torch.zeros(slots, H, dtype=dtype, device="cuda")
                st["dw"] = torch.zeros(T, topk, dtype=torch.float32, device="cuda")
            else:
                st["out"] = torch.zeros(T, H, dtype=dtype, device="cuda")
    if own:
        st.update(_plan(st))
    return st


def _plan(st):
    """What a program of this library's user makes once for a shape."""
    import mxfp4_weight_expert_amd as moe

    c = st["case"]
    if c["op"] in ("linear", "grouped"):
        rows = c["T"] * c["topk"] if c["op"] == "grouped" else c["T"]
        return {"shape": moe.W4Shape(M=rows, N=c["N"], K=c["K"], E=c["E"], format=c["format"], group=c["group"],
                                     dtype=c["dtype"], out_dtype=c["out"])}
    shape = moe.DispatchShape(T=c["T"], E=c["E"], topk=c["topk"], H=c["H"], dtype=c["dtype"], expert_offset=_offset(c))
    if c["op"] != "dispatch":
        return {"shape": shape}
    return {"shape": shape, "workspace": torch.empty(moe.dispatch_query(shape), dtype=torch.uint8, device="cuda")}


def run(st):
    return _own(st) if own else _PLAIN[st["case"]["op"]](st)


def _own(st):
    import mxfp4_weight_expert_amd as moe

    op, shape = st["case"]["op"], st["shape"]
    if op == "dispatch":
        return moe.dispatch(st["x"], st["ids"], shape, out=st["out"], offsets=st["offsets"], row_slot=st["row_slot"],
                            slot_row=st["slot_row"], workspace=st["workspace"])
    if op == "dispatch_grad":
        return moe.dispatch_backward(st["rows"], st["slot_row"], shape, out=st["out"])
    if op == "combine":
        return moe.combine(st["rows"], st["slot_row"], st["topk_w"], shape, out=st["out"])
    if op == "combine_grad":
        return moe.combine_backward(st["dout"], st["rows"], st["slot_row"], st["topk_w"], shape, dy=st["out"], dw=st["dw"])
    if op == "linear":
        return moe.w4_linear(st["x"], st["w"], st["scales"], shape, zeros=st["zeros"], bias=st["bias"], out=st["out"])
    return moe.w4_grouped_linear(st["x"], st["offsets"], st["w"], st["scales"], shape, zeros=st["zeros"], bias=st["bias"],
                                 out=st["out"])


# ------------------------------------------------------------------------------------------ plain forms


def _plain_dispatch(st):
    case = st["case"]
    order, row, offsets = _maps(st["ids"], case)
    live = torch.arange(order.numel(), device=order.device) < offsets[-1]  # rows behind the last expert stay as they are
    rows = torch.where(live[:, None], st["x"][order // case["topk"]], st["out"])
    slot = torch.where(live, order, st["row_slot"].long())
    return rows, offsets.to(torch.int32), slot.to(torch.int32), row.to(torch.int32).view(case["T"], case["topk"])


def _gathered(st):
    """Each slot's row in 32 bits, [T, topk, H]; zeros where the slot has none."""
    at = st["slot_row"].long()
    return torch.where((at >= 0)[..., None], st["rows"][at.clamp_min(0)].float(), torch.zeros((), device=at.device))


def _plain_dispatch_grad(st):
    return _gathered(st).sum(1).to(st["out"].dtype)


def _plain_combine(st):
    return (_gathered(st) * st["topk_w"][..., None]).sum(1).to(st["out"].dtype)


def _plain_combine_grad(st):
    case, at = st["case"], st["slot_row"].long().view(-1)
    slots = at.numel()
    dw = (_gathered(st) * st["dout"].float()[:, None, :]).sum(2)
    slot = torch.full((slots + 1,), -1, dtype=torch.int64, device=at.device)
    slot[torch.where(at >= 0, at, torch.full_like(at, slots))] = torch.arange(slots, device=at.device)
    slot = slot[:slots]
    s = slot.clamp_min(0)
    dy = st["topk_w"].view(-1)[s][:, None] * st["dout"].float()[s // case["topk"]]
    return torch.where((slot >= 0)[:, None], dy.to(st["out"].dtype), st["out"]), dw


def _dequantised(st):
    """The weights in 32 bits, [E, N, K]."""
    case, w = st["case"], st["w"]
    E, N, K, group = case["E"], case["N"], case["K"], case["group"]
    up = w.shape[1]
    w = w.view(E, up // 16, K // 128, 16, 64).transpose(2, 3).reshape(E, up, K // 2)[:, :N]
    code = torch.stack([w & 15, w >> 4], -1).view(E, N, K // group, group)
    if case["format"] == "mxfp4":
        m = (code & 7).float()
        v = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))
        v = torch.where(code >= 8, -v, v)
        scale = torch.exp2(st["scales"].float() - 127)
    else:
        zero = st["zeros"].float()[..., None] if st["zeros"] is not None else 8.0
        v, scale = code.float() - zero, st["scales"].float()
    return (v * scale[..., None]).view(E, N, K)


def _plain_linear(st):
    out = st["x"].float() @ _dequantised(st)[0].t()
    if st["bias"] is not None:
        out = out + st["bias"][0].float()
    return out.to(st["out"].dtype)


def _plain_grouped(st):
    case, first = st["case"], st["offsets"].long()
    rows = torch.arange(st["x"].shape[0], device=first.device)
    expert = (torch.searchsorted(first, rows, right=True) - 1).clamp_max(case["E"] - 1)
    live = rows < first[-1]
    at = torch.where(live, expert * st["most"] + rows - first[expert], torch.full_like(rows, case["E"] * st["most"]))
    x = torch.zeros(case["E"] * st["most"] + 1, case["K"], device=rows.device)
    x[at] = torch.where(live[:, None], st["x"].float(), torch.zeros((), device=rows.device))
    x = x[:-1].view(case["E"], st["most"], case["K"]).transpose(1, 2).contiguous()
    out = torch.bmm(_dequantised(st), x)  # [E, N, most]
    if st["bias"] is not None:
        out = out + st["bias"].float()[..., None]
    out = out.transpose(1, 2).reshape(-1, case["N"])[at.clamp_max(case["E"] * st["most"] - 1)]
    return torch.where(live[:, None], out.to(st["out"].dtype), st["out"])


_PLAIN = {"dispatch": _plain_dispatch, "dispatch_grad": _plain_dispatch_grad, "combine": _plain_combine,
          "combine_grad": _plain_combine_grad, "linear": _plain_linear, "grouped": _plain_grouped}


# ------------------------------------------------------------------------------------ work and 64 bits


def work(case):
    op, T, topk, size = case["op"], case["T"], case["topk"], _SIZE[case["dtype"]]
    slots = T * topk
    here = slots * case["E"] / case["experts"]  # slots with a local expert, on average
    if op in ("linear", "grouped"):
        N, K, group = case["N"], case["K"], case["group"]
        rows, touched = T, 1.0
        if op == "grouped":
            rows, touched = here, case["E"] * (1 - (1 - topk / case["experts"]) ** T)
        scale = 1 if case["format"] == "mxfp4" else size + case["zeros"]
        weights = touched * N * (K / 2 + K / group * scale + case["bias"] * size)
        return {"bytes": weights + rows * (K * size + N * _SIZE[case["out"]]), "flops": 2 * rows * N * K}
    H = case["H"]
    if op == "dispatch":
        return {"bytes": (T + here) * H * size + 4 * (2 * slots + here + case["E"] + 1), "flops": 0}
    if op == "combine_grad":
        return {"bytes": (T + 2 * here) * H * size + 12 * slots, "flops": 3 * here * H}
    weighted = op == "combine"
    return {"bytes": (T + here) * H * size + (4 + 4 * weighted) * slots, "flops": (1 + weighted) * here * H}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "grouped"):
        return _exact_product(case, st)
    T, topk, E = case["T"], case["topk"], case["E"]
    if op == "dispatch":
        # one whole number for a slot: its expert, then its place; sorted, they are the rows
        slots = T * topk
        place = torch.arange(slots, device="cuda")
        expert = st["ids"].view(-1).to(torch.int64) - _offset(case)
        away = (expert < 0) | (expert >= E)
        ordered = torch.sort(torch.where(away, E, expert) * slots + place).values
        slot, owner = ordered % slots, ordered // slots
        live = owner < E
        offsets = torch.searchsorted(owner, torch.arange(E + 1, device="cuda"))
        rows = st["x"].double()[slot // topk].mul_(live[:, None])
        back = torch.argsort(slot).masked_fill(away, -1)
        return rows, offsets.to(torch.int32), (slot * live).to(torch.int32), back.to(torch.int32).view(T, topk)
    H, at = case["H"], st["slot_row"].long()
    w = st["topk_w"].double()
    if op == "combine_grad":
        dy = torch.zeros(T * topk, H, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, topk, dtype=torch.float64, device="cuda")
        dout = st["dout"].double()
        for k in range(topk):
            has = (at[:, k] >= 0).nonzero()[:, 0]
            rows = at[has, k]
            dy[rows] = w[has, k, None] * dout[has]
            dw[has, k] = (st["rows"][rows].double() * dout[has]).sum(1)
        return dy, dw
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for k in range(topk):
        has = (at[:, k] >= 0).nonzero()[:, 0]
        rows = st["rows"][at[has, k]].double()
        out[has] += rows * w[has, k, None] if op == "combine" else rows
    return out


def _exact_product(case, st):
    E, N, K, group = case["E"], case["N"], case["K"], case["group"]
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    table = torch.cat([table, -table]) if case["format"] == "mxfp4" else torch.arange(16, dtype=torch.float64, device="cuda")
    first = [0, case["T"]] if case["op"] == "linear" else st["offsets"].tolist()
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    column = torch.arange(K, device="cuda")
    byte, high = column // 2, column % 2
    for e in range(E):
        lo, hi = first[e], first[e + 1]
        if lo == hi:
            continue
        x = st["x"][lo:hi].double()
        flat = st["w"][e].reshape(-1)
        for n in range(0, N, 8192):
            row = torch.arange(n, min(N, n + 8192), device="cuda")[:, None]
            where = (row // 16 * (K // 128) + byte // 64) * 1024 + row % 16 * 64 + byte % 64
            code = flat[where].long() >> (4 * high) & 15
            v = table[code]
            s = st["scales"][e, n : n + 8192].double()
            if case["format"] == "mxfp4":
                s = torch.pow(2.0, s - 127)
            else:
                z = 8 if st["zeros"] is None else st["zeros"][e, n : n + 8192].double().repeat_interleave(group, 1)
                v = v - z
            out[lo:hi, n : n + 8192] = x @ (v * s.repeat_interleave(group, 1)).t()
        if st["bias"] is not None:
            out[lo:hi] += st["bias"][e].double()
    return out
