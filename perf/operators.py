"""Cases of the 4-bit weight products and of the mixture-of-experts (MoE)
token routing: what each is timed and compared on.

`run` computes a case either in its plain form (elementary torch operations
in fp32) or, with `own` set, through the calls a user makes of
int8_gemm_linear_amd.  The kinds of case:

  linear    Y = X W^T with 4-bit weights W = s (q - z), a scale (and zero
            point) per group of 32, 64 or 128 along K; bf16 X and Y
  experts   the same product for tokens sorted by expert, one weight per expert
  dispatch  tokens sorted by expert: offsets, rows, and a copy of each
            token's row (and scales) for each of its experts
  combine   the experts' rows brought back: a weighted sum for each token
  gradient  of combine (rows and weights) and of dispatch (tokens)

Layer sizes are those of the 1.7B- and 32B-class decoder linears and of the
128-expert layers (hidden 2048, top-8, width 768) the benchmark uses.
"""
import math

import torch

own = False

SCALES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ROWS = {"bf16": torch.bfloat16, "fp32": torch.float32, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # one token through a small layer (1.7B class): the call's latency counts
        {"name": "linear 1 token small", "kind": "linear", "M": 1, "N": 2048, "K": 2048, "group": 128,
         "scale": "bf16", "zero": False},
        # one token through the largest decoder layer (32B class gate_up): the weights' bytes count
        {"name": "linear 1 token large", "kind": "linear", "M": 1, "N": 51200, "K": 5120, "group": 128,
         "scale": "bf16", "zero": False},
        # a decode batch with zero points and short groups on the longest K (32B class down)
        {"name": "linear 32 tokens", "kind": "linear", "M": 32, "N": 5120, "K": 25600, "group": 64,
         "scale": "fp16", "zero": True},
        # a prompt of odd length (32B class qkv): the products count
        {"name": "linear prompt", "kind": "linear", "M": 1000, "N": 10240, "K": 5120, "group": 128,
         "scale": "fp32", "zero": False},
        # a decode batch of 32 tokens through 128 experts' gate_up: about two rows per expert
        {"name": "experts 32 tokens", "kind": "experts", "T": 32, "topk": 8, "E": 128, "N": 1536, "K": 2048,
         "group": 128, "scale": "bf16", "zero": False},
        # a prompt through 128 experts' down, ragged experts of 40 to 250 rows
        {"name": "experts prompt", "kind": "experts", "T": 2000, "topk": 8, "E": 128, "N": 2048, "K": 768,
         "group": 64, "scale": "bf16", "zero": True},
        # a decode batch: int8 codes with a scale per token, the latency of the routing
        {"name": "dispatch 16 tokens", "kind": "dispatch", "T": 16, "topk": 8, "E": 128, "K": 2048,
         "rows": "int8", "scales": 1, "drop": 0.0},
        # a long prompt in e4m3 with a scale per 128 values; a twentieth of the slots is for experts elsewhere
        {"name": "dispatch prompt", "kind": "dispatch", "T": 8191, "topk": 8, "E": 128, "K": 2048,
         "rows": "e4m3", "scales": 16, "drop": 0.05},
        # a decode batch's rows brought back
        {"name": "combine 16 tokens", "kind": "combine", "T": 16, "topk": 8, "E": 128, "K": 2048,
         "rows": "bf16", "drop": 0.0},
        # a long prompt's rows brought back
        {"name": "combine prompt", "kind": "combine", "T": 8191, "topk": 8, "E": 128, "K": 2048,
         "rows": "bf16", "drop": 0.05},
        # a training step on few tokens, in fp32 and an odd width that no wide load divides
        {"name": "gradient small", "kind": "gradient", "T": 333, "topk": 2, "E": 16, "K": 1027,
         "rows": "fp32", "drop": 0.0},
        # a training step on a long batch
        {"name": "gradient large", "kind": "gradient", "T": 8192, "topk": 8, "E": 128, "K": 2048,
         "rows": "bf16", "drop": 0.02},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["linear", "experts", "dispatch", "combine", "gradient"])
    if kind == "linear":
        group = rng.choice([32, 64, 128])
        K = group * _log_int(rng, 2, 25600 // group)
        N = _log_int(rng, 16, 51200)
        M = _log_int(rng, 1, 1024)
        while N * K > 51200 * 5120 or M * N * K > 1000 * 10240 * 5120:
            N, M = max(16, N // 2), max(1, M // 2)
        return {"kind": kind, "M": M, "N": N, "K": K, "group": group,
                "scale": rng.choice(sorted(SCALES)), "zero": rng.random() < 0.5}
    E = rng.choice([8, 16, 60, 64, 128])
    topk = rng.randint(1, 8)
    if kind == "experts":
        group = rng.choice([32, 64, 128])
        K = group * _log_int(rng, 2, 4096 // group)
        N = _log_int(rng, 64, 2048)
        T = _log_int(rng, 1, 2000)
        while E * N * K > 128 * 1536 * 2048:
            N //= 2
        while T * topk * N * K > 2000 * 8 * 2048 * 768:
            T //= 2
        return {"kind": kind, "T": T, "topk": topk, "E": E, "N": N, "K": K, "group": group,
                "scale": rng.choice(sorted(SCALES)), "zero": rng.random() < 0.5}
    T = _log_int(rng, 1, 8192)
    drop = rng.choice([0.0, 0.0, 0.1, 0.5]) if T >= 16 else 0.0
    if kind == "dispatch":
        rows = rng.choice(["bf16", "int8", "e4m3"])
        K = 128 * rng.randint(1, 16) if rows != "bf16" else _log_int(rng, 64, 2048)
        scales = {"bf16": 0, "int8": 1, "e4m3": rng.choice([1, K // 128])}[rows]
        while T * topk * K * ROWS[rows].itemsize > 8191 * 8 * 2048:
            T //= 2
        return {"kind": kind, "T": T, "topk": topk, "E": E, "K": K, "rows": rows, "scales": scales, "drop": drop}
    rows = rng.choice(["bf16", "fp32"])
    K = _log_int(rng, 64, 2048)
    while T * topk * K * ROWS[rows].itemsize > 8191 * 8 * 2048 * 2:
        T //= 2
    return {"kind": kind, "T": T, "topk": topk, "E": E, "K": K, "rows": rows, "drop": drop}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * int(seed) + 17)


def _codes(shape, group, scale, zero, g):
    """Codes, scales and zero points of weights ~ N(0, 0.02): symmetric around 8, or with a zero point
    near 8 that differs by group (an asymmetric quantizer's)."""
    *lead, N, K = shape
    w = torch.randn((*lead, N, K), generator=g, device="cuda").mul_(2.4).add_(8).round_().clamp_(0, 15).to(torch.uint8)
    q = w[..., 0::2] | (w[..., 1::2] << 4)
    s = 0.02 / 2.4 * (0.5 + torch.rand((*lead, N, K // group), generator=g, device="cuda"))
    z = torch.randint(6, 11, (*lead, N, K // group), generator=g, device="cuda", dtype=torch.uint8) if zero else None
    return q, s.to(SCALES[scale]), z


def _routing(T, topk, E, drop, g):
    """Experts [T, topk] (distinct for each token, some experts liked more) and fp32 weights that sum to one;
    a share `drop` of the slots goes nowhere (-1)."""
    liking = torch.randn((1, E), generator=g, device="cuda") * 0.3
    p = torch.softmax(torch.randn((T, E), generator=g, device="cuda") + liking, dim=1)
    w, ids = torch.topk(p, min(topk, E), dim=1)
    w = w / w.sum(dim=1, keepdim=True)
    if drop:
        ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < drop, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32).contiguous(), w.contiguous()


def _sort(ids, E):
    """Offsets [E + 1] and the row of each slot (-1: none), rows sorted by (expert, slot index)."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    _, order = torch.sort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=order.device)
    row = torch.where(key < E, row, torch.full_like(row, -1))
    offsets = torch.searchsorted(key[order].contiguous(), torch.arange(E + 1, device=flat.device))
    return offsets.to(torch.int32), row.to(torch.int32).view(ids.shape), order


def prepare(case, seed):
    g = _generator(seed)
    kind = case["kind"]
    s = {"case": case}
    if kind in ("linear", "experts"):
        K = case["K"]
        if kind == "linear":
            s["x"] = torch.randn((case["M"], K), generator=g, device="cuda").to(torch.bfloat16)
            shape = (case["N"], K)
        else:
            ids, _ = _routing(case["T"], case["topk"], case["E"], 0.0, g)
            s["offsets"], _, _ = _sort(ids, case["E"])
            s["x"] = torch.randn((ids.numel(), K), generator=g, device="cuda").to(torch.bfloat16)
            shape = (case["E"], case["N"], K)
            s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["q"], s["scale"], s["zero"] = _codes(shape, case["group"], case["scale"], case["zero"], g)
        return s
    T, topk, K = case["T"], case["topk"], case["K"]
    dt = ROWS[case["rows"]]
    s["ids"], s["weights"] = _routing(T, topk, case["E"], case["drop"], g)
    R = s["ids"].numel()
    if kind == "dispatch":
        x = torch.randn((T, K), generator=g, device="cuda")
        s["x"] = (x * 40).round().clamp(-127, 127).to(dt) if dt == torch.int8 else \
            (x * 100).to(dt) if dt == torch.float8_e4m3fn else x.to(dt)
        n = case["scales"]
        s["scale"] = None if n == 0 else 0.01 + torch.rand((T,) if n == 1 else (T, n), generator=g, device="cuda")
        # the rows behind the last expert's stay as they are: the caller's buffers, cleared once
        s["rows"] = torch.zeros((R, K), dtype=dt, device="cuda")
        s["row_scale"] = None if n == 0 else torch.zeros((R,) if n == 1 else (R, n), device="cuda")
        return s
    _, s["slot_row"], _ = _sort(s["ids"], case["E"])
    s["y"] = torch.randn((R, K), generator=g, device="cuda").to(dt)
    if kind == "gradient":
        s["dout"] = torch.randn((T, K), generator=g, device="cuda").to(dt)
        s["drows"] = torch.randn((R, K), generator=g, device="cuda").to(dt)
        s["dy"] = torch.zeros((R, K), dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the plain forms, fp32
# ---------------------------------------------------------------------------
def _weights(q, scale, zero, dtype):
    """s (q - z) as [..., N, K] of `dtype`."""
    K = 2 * q.shape[-1]
    groups = scale.shape[-1]
    v = torch.stack((q & 15, q >> 4), dim=-1).to(dtype).view(*q.shape[:-1], groups, K // groups)
    z = 8.0 if zero is None else zero.to(dtype).unsqueeze(-1)
    return ((v - z) * scale.to(dtype).unsqueeze(-1)).view(*q.shape[:-1], K)


def _grouped(s, dtype):
    """The experts' products on rows padded to the fullest expert's, then taken out again."""
    x, off, most = s["x"], s["offsets"].long(), s["most"]
    E, K = s["q"].shape[0], x.shape[1]
    w = _weights(s["q"], s["scale"], s["zero"], dtype)
    row = torch.arange(x.shape[0], device=x.device)
    e = torch.searchsorted(off[1:].contiguous(), row, right=True)
    at = row - off[e]
    padded = torch.zeros((E, K, most), dtype=dtype, device=x.device)
    padded[e, :, at] = x.to(dtype)
    return torch.matmul(w, padded)[e, :, at].contiguous()


def _gather(y, slot_row, dtype):
    """y's row for each slot, [T, topk, K]; zeros where the slot has none."""
    there = slot_row >= 0
    v = y[slot_row.clamp(min=0).long().reshape(-1)].view(*slot_row.shape, y.shape[1]).to(dtype)
    return torch.where(there.unsqueeze(-1), v, torch.zeros((), dtype=dtype, device=y.device)), there


def _combine(s, dtype):
    v, _ = _gather(s["y"], s["slot_row"], dtype)
    return (v * s["weights"].to(dtype).unsqueeze(-1)).sum(dim=1)


def _gradient(s, dtype):
    """dy (rows behind the last expert's as they were), dweights, dx."""
    v, there = _gather(s["y"], s["slot_row"], dtype)
    d = s["dout"].to(dtype).unsqueeze(1)
    dweights = (v * d).sum(dim=2)
    dx = _gather(s["drows"], s["slot_row"], dtype)[0].sum(dim=1)
    slots = torch.where(there, s["slot_row"], there.numel()).reshape(-1)
    _, order = torch.sort(slots, stable=True)                     # the slot of each row
    has = (torch.arange(order.numel(), device=order.device) < there.sum()).unsqueeze(1)
    dy = s["dout"].to(dtype)[order // there.shape[1]] * s["weights"].to(dtype).reshape(-1)[order].unsqueeze(1)
    return torch.where(has, dy, s["dy"].to(dtype)), dweights, dx


def _plain(s):
    kind = s["case"]["kind"]
    if kind == "linear":
        return torch.matmul(s["x"].float(), _weights(s["q"], s["scale"], s["zero"], torch.float32).t()).to(torch.bfloat16)
    if kind == "experts":
        return _grouped(s, torch.float32).to(torch.bfloat16)
    if kind == "dispatch":
        E, topk = s["case"]["E"], s["ids"].shape[1]
        off, slot_row, order = _sort(s["ids"], E)
        # the order's slots without an expert come last: those rows keep what the buffers hold
        has = (torch.arange(order.numel(), device=order.device) < off[E]).unsqueeze(1)
        token = order // topk
        rows = s["rows"].view(torch.uint8)
        rows.copy_(torch.where(has, s["x"].view(torch.uint8)[token], rows))
        scale = s["row_scale"]
        if scale is not None:
            scale.copy_(torch.where(has if scale.dim() == 2 else has.squeeze(1), s["scale"][token], scale))
        return {"rows": s["rows"], "scale": scale, "offsets": off, "slot_row": slot_row}
    if kind == "combine":
        return _combine(s, torch.float32).to(s["y"].dtype)
    dy, dweights, dx = _gradient(s, torch.float32)
    return {"dy": s["dy"].copy_(dy), "dweights": dweights, "dx": dx.to(s["dy"].dtype)}


def _own(s):
    import int8_gemm_linear_amd as q
    kind = s["case"]["kind"]
    if kind == "linear":
        return q.w4_mm(s["x"], s["q"], s["scale"], s["zero"])
    if kind == "experts":
        # a token takes an expert once, so no expert has more rows than there are tokens
        return q.grouped_w4_mm(s["x"], s["q"], s["scale"], s["offsets"], s["case"]["T"], s["zero"])
    if kind == "dispatch":
        rows, scale, off, slot_row = q.moe_dispatch(s["x"], s["ids"], s["case"]["E"], scale=s["scale"],
                                                    out=s["rows"], out_scale=s["row_scale"])
        return {"rows": rows, "scale": scale, "offsets": off, "slot_row": slot_row}
    if kind == "combine":
        return q.moe_combine(s["y"], s["slot_row"], s["weights"])
    dy, dweights = q.moe_combine_backward(s["dout"], s["y"], s["slot_row"], s["weights"], dy=s["dy"])
    return {"dy": dy, "dweights": dweights, "dx": q.moe_permute_backward(s["drows"], s["slot_row"])}


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    """The outputs from the definitions in fp64."""
    kind = case["kind"]
    s = prepare(case, seed)
    if kind == "dispatch":
        floating = s["x"].dtype != torch.int8
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda") if floating else None
        scale = None if s["scale"] is None else torch.zeros(s["row_scale"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for e in range(case["E"]):
            token = torch.nonzero(s["ids"] == e)[:, 0]
            end = at + token.numel()
            if floating:
                rows[at:end] = s["x"].double()[token]
            if scale is not None:
                scale[at:end] = s["scale"].double()[token]
            at = end
        return {"rows": rows, "scale": scale, "offsets": None, "slot_row": None}
    if kind == "combine":
        out = torch.zeros((case["T"], case["K"]), dtype=torch.float64, device="cuda")
        for j in range(s["slot_row"].shape[1]):
            r = s["slot_row"][:, j].long()
            at = torch.nonzero(r >= 0).squeeze(1)
            out[at] += s["weights"][at, j].double().unsqueeze(1) * s["y"][r[at]].double()
        return out
    if kind == "gradient":
        dy = s["dy"].double()
        dweights = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
        dx = torch.zeros((case["T"], case["K"]), dtype=torch.float64, device="cuda")
        for j in range(s["slot_row"].shape[1]):
            r = s["slot_row"][:, j].long()
            at = torch.nonzero(r >= 0).squeeze(1)
            d = s["dout"][at].double()
            dy[r[at]] = s["weights"][at, j].double().unsqueeze(1) * d
            dweights[at, j] = (d * s["y"][r[at]].double()).sum(dim=1)
            dx[at] += s["drows"][r[at]].double()
        return {"dy": dy, "dweights": dweights, "dx": dx}
    group = case["group"]

    def product(x, codes, scale, zero):
        out = torch.zeros((x.shape[0], codes.shape[0]), dtype=torch.float64, device="cuda")
        x = x.double()
        step = max(1, (1 << 26) // case["K"])
        for n in range(0, codes.shape[0], step):
            c = codes[n:n + step]
            w = torch.empty((c.shape[0], case["K"]), dtype=torch.float64, device="cuda")
            w[:, 0::2] = (c % 16).double()
            w[:, 1::2] = torch.div(c, 16, rounding_mode="floor").double()
            w -= 8.0 if zero is None else zero[n:n + step].double().repeat_interleave(group, dim=1)
            w *= scale[n:n + step].double().repeat_interleave(group, dim=1)
            out[:, n:n + step] = x @ w.t()
        return out

    if kind == "linear":
        return product(s["x"], s["q"], s["scale"], s["zero"])
    off = s["offsets"].tolist()
    out = torch.zeros((s["x"].shape[0], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        if off[e + 1] > off[e]:
            out[off[e]:off[e + 1]] = product(s["x"][off[e]:off[e + 1]], s["q"][e], s["scale"][e],
                                             None if s["zero"] is None else s["zero"][e])
    return out


def work(case):
    kind = case["kind"]
    if kind in ("linear", "experts"):
        N, K = case["N"], case["K"]
        one = N * K / 2 + N * (K // case["group"]) * (SCALES[case["scale"]].itemsize + case["zero"])
        if kind == "linear":
            rows, weights = case["M"], one
        else:
            # experts that get a row when each token takes its experts evenly
            T, E, topk = case["T"], case["E"], min(case["topk"], case["E"])
            rows, weights = T * topk, one * E * (1 - (1 - topk / E) ** T)
        return {"bytes": weights + 2 * rows * (K + N), "flops": 2 * rows * N * K}
    T, K = case["T"], case["K"]
    slots = T * min(case["topk"], case["E"])
    moved = slots * (1 - case["drop"])
    row = K * ROWS[case["rows"]].itemsize
    if kind == "dispatch":
        return {"bytes": (T + moved) * (row + 4 * case["scales"]) + 8 * slots, "flops": 0}
    if kind == "combine":
        return {"bytes": (T + moved) * row + 8 * slots, "flops": 2 * moved * K}
    # dout, y and drows read, dy and dx written
    return {"bytes": (2 * T + 3 * moved) * row + 12 * slots, "flops": 4 * moved * K}
