"""Cases of the low-rank adapters, the tokens' log probabilities and the
embedding: what each is timed and compared on.

`run` computes a case either in its plain form (elementary torch operations
in fp32) or, with `own` set, through the calls a user makes of
int8_gemm_linear_amd.  The kinds of case:

  adapter            Y = base + s_i (X A_i^T) B_i^T beside a shared projection,
                     the adapter i of each token by its request
  adapter gradient   dX, dA and dB of the same
  logprobs           of each row's given token, with the row's entropy, log of
                     the sum of exponentials and best alternatives
  logprobs gradient  of the log probabilities and entropies: the logits'
  embedding          rows of a table (plain, or codes with scales) by token
  embedding gradient summed over the positions of each token: the table's

Layer sizes are those of the 1.7B- and 32B-class decoder linears the benchmark
uses; the vocabularies are generic.
"""
import math

import torch

own = False

FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TABLES = {**FLOATS, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # one token of one request through a small layer (1.7B class): the call's latency counts
        {"name": "adapter 1 token", "kind": "adapter", "T": 1, "K": 2048, "N": 2048, "R": 16, "L": 8,
         "requests": 1, "runs": False, "drop": 0.0},
        # a decode batch, every token another request with an adapter of its own, some without (32B class qkv)
        {"name": "adapter 32 requests", "kind": "adapter", "T": 32, "K": 5120, "N": 10240, "R": 16, "L": 64,
         "requests": 28, "runs": False, "drop": 0.1},
        # a large decode batch whose requests share adapters of a high rank (32B class gate_up): the adapters' bytes
        {"name": "adapter wide", "kind": "adapter", "T": 128, "K": 5120, "N": 51200, "R": 64, "L": 32,
         "requests": 24, "runs": False, "drop": 0.0},
        # prompts of ragged lengths in one batch: the tokens' bytes
        {"name": "adapter prompts", "kind": "adapter", "T": 4001, "K": 5120, "N": 5120, "R": 32, "L": 8,
         "requests": 6, "runs": True, "drop": 0.05},
        # a training step on few tokens and sizes that no tile divides
        {"name": "adapter gradient small", "kind": "adapter gradient", "T": 333, "K": 1032, "N": 1001, "R": 8,
         "L": 3, "requests": 3, "runs": False, "drop": 0.0},
        # a training step of eight adapters at once (32B class qkv)
        {"name": "adapter gradient", "kind": "adapter gradient", "T": 8192, "K": 5120, "N": 10240, "R": 16,
         "L": 8, "requests": 8, "runs": True, "drop": 0.0},
        # one sampled token with its alternatives: a single long row
        {"name": "logprobs 1 row", "kind": "logprobs", "T": 1, "V": 131072, "type": "bf16", "top": 20,
         "banned": 0.0, "drop": 0.0},
        # a decode batch under a grammar that bans tokens (-inf), fp32 logits of an odd vocabulary
        {"name": "logprobs 48 rows", "kind": "logprobs", "T": 48, "V": 100003, "type": "fp32", "top": 5,
         "banned": 0.3, "drop": 0.0},
        # a prompt's tokens scored, with the best alternative of each
        {"name": "logprobs prompt", "kind": "logprobs", "T": 2047, "V": 131072, "type": "bf16", "top": 1,
         "banned": 0.0, "drop": 0.02},
        # a training step on an odd vocabulary: loss and entropy bonus
        {"name": "logprobs gradient", "kind": "logprobs gradient", "T": 4096, "V": 100003, "type": "bf16",
         "entropy": True, "drop": 0.05},
        # a decode batch's tokens from a table of codes with a scale per 128 values
        {"name": "embedding 16 tokens", "kind": "embedding", "T": 16, "V": 131072, "H": 5120, "type": "e4m3",
         "scales": 40, "drop": 0.0},
        # a training step: a few tokens make up much of any text
        {"name": "embedding gradient", "kind": "embedding gradient", "T": 16384, "V": 131072, "H": 2048,
         "type": "bf16", "drop": 0.05},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["adapter", "adapter", "adapter gradient", "logprobs", "logprobs gradient",
                       "embedding", "embedding gradient"])
    if kind.startswith("adapter"):
        gradient = kind != "adapter"
        c = {"kind": kind, "K": 8 * _log_int(rng, 16, 25600 // 8), "N": _log_int(rng, 16, 51200),
             "R": rng.choice([8, 16, 24, 32, 64]), "L": _log_int(rng, 1, 64), "runs": gradient or rng.random() < 0.5}
        c["T"] = _log_int(rng, 1, 8192 if gradient else 4096) if c["runs"] else _log_int(rng, 1, 256)
        c["requests"] = min(c["T"], _log_int(rng, 1, c["L"]))
        c["drop"] = rng.choice([0.0, 0.1]) if c["T"] >= 16 else 0.0
        most = listed()[5 if gradient else 2]
        while work(c)["bytes"] > work(most)["bytes"] or c["L"] * c["R"] * (c["K"] + c["N"]) > 32 * 64 * 56320:
            key = "T" if 2 * c["T"] > c["L"] * c["R"] and c["T"] > 1 else "L" if c["L"] > 1 else "N"
            c[key] = max(1, c[key] // 2)
            c["requests"] = min(c["requests"], c["T"], c["L"])
            c["drop"] = c["drop"] if c["T"] >= 16 else 0.0
        return c
    T, drop = _log_int(rng, 1, 16384), rng.choice([0.0, 0.1])
    if kind.startswith("logprobs"):
        V, dt = _log_int(rng, 128, 200000), rng.choice(sorted(FLOATS))
        while T * V * FLOATS[dt].itemsize > 2047 * 131072 * 2:
            T = max(1, T // 2)
        drop = drop if T >= 16 else 0.0
        if kind == "logprobs":
            return {"kind": kind, "T": T, "V": V, "type": dt, "top": rng.choice([0, 1, 5, 20, 32]),
                    "banned": rng.choice([0.0, 0.5]), "drop": drop}
        return {"kind": kind, "T": T, "V": V, "type": dt, "entropy": rng.random() < 0.5, "drop": drop}
    V, drop = _log_int(rng, 256, 131072), drop if T >= 16 else 0.0
    if kind == "embedding":
        dt = rng.choice(sorted(TABLES))
        H = 128 * rng.randint(1, 40) if dt in ("int8", "e4m3") else _log_int(rng, 64, 5120)
        while V * H > 131072 * 5120 // 2:
            V //= 2
        return {"kind": kind, "T": T, "V": V, "H": H, "type": dt,
                "scales": rng.choice([1, H // 128]) if dt in ("int8", "e4m3") else 0, "drop": drop}
    dt, H = rng.choice(sorted(FLOATS)), _log_int(rng, 64, 5120)
    while (V + T) * H * FLOATS[dt].itemsize > (131072 + 16384) * 2048 * 2:
        V, T = max(1, V // 2), max(1, T // 2)
    return {"kind": kind, "T": T, "V": V, "H": H, "type": dt, "drop": drop if T >= 16 else 0.0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * int(seed) + 29)


def _requests(case, g):
    """The adapter of each token, int32 [T]: `requests` different ones, in runs of ragged lengths (prompts)
    or mixed (a decode batch); a share `drop` of the tokens has none (-1)."""
    T, n = case["T"], case["requests"]
    chosen = torch.randperm(case["L"], generator=g, device="cuda")[:n]
    none = int(case["drop"] * T)
    # every request has a token, the others are spread over them
    more = torch.randint(0, n, (T - n - none,), generator=g, device="cuda") if T - n - none > 0 else chosen[:0]
    which = torch.cat((torch.arange(n, device="cuda"), more))[:T]
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    if case["runs"]:
        ids[:which.numel()] = chosen[torch.sort(which).values].to(torch.int32)
        return ids.roll(none // 2)
    at = torch.randperm(T, generator=g, device="cuda")[:which.numel()]
    ids[at] = chosen[which].to(torch.int32)
    return ids


def _normal(shape, dtype, g, sigma=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(sigma).to(dtype)


def _tokens(T, V, drop, g):
    """Tokens [T] int64 as text has them: the n-th commonest about as often as 1/n; -1 (padding) for a share."""
    rank = torch.exp(torch.rand((T,), generator=g, device="cuda", dtype=torch.float64) * math.log(V)).long() - 1
    ids = torch.randperm(V, generator=g, device="cuda")[rank.clamp(0, V - 1)]
    return torch.where(torch.rand((T,), generator=g, device="cuda") < drop, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    g = _generator(seed)
    kind = case["kind"]
    s = {"case": case}
    if kind.startswith("adapter"):
        T, K, N, R, L = (case[k] for k in ("T", "K", "N", "R", "L"))
        bf16 = torch.bfloat16
        s["x"] = _normal((T, K), bf16, g)
        s["a"], s["b"] = _normal((L, R, K), bf16, g, K ** -0.5), _normal((L, N, R), bf16, g, 0.1)
        s["ids"] = _requests(case, g)
        s["scale"] = 0.5 + 1.5 * torch.rand((L,), generator=g, device="cuda")        # alpha / rank
        if kind == "adapter":
            s["base"] = _normal((T, N), bf16, g)                                     # the shared projection's output
        else:
            s["dy"], s["base"] = _normal((T, N), bf16, g), _normal((T, K), bf16, g)  # its gradient of x
        return s
    if kind.startswith("logprobs"):
        T, V = case["T"], case["V"]
        s["logits"] = _normal((T, V), FLOATS[case["type"]], g, 2.0)
        s["target"] = torch.randint(0, V, (T,), generator=g, device="cuda")
        likely = torch.rand((T, 1), generator=g, device="cuda").mul_(16).to(s["logits"].dtype)
        s["logits"].scatter_add_(1, s["target"].unsqueeze(1), likely)
        if case.get("banned"):
            step = max(1, (1 << 27) // V)
            for t in range(0, T, step):
                part = s["logits"][t:t + step]
                ban = torch.rand(part.shape, generator=g, device="cuda") < case["banned"]
                ban.scatter_(1, s["target"][t:t + step].unsqueeze(1), False)
                part.masked_fill_(ban, -math.inf)
        s["target"][torch.rand((T,), generator=g, device="cuda") < case["drop"]] = -1
        if kind == "logprobs gradient":
            lse, entropy = [], []                                   # the forward pass's
            step = max(1, (1 << 26) // V)
            for t in range(0, T, step):
                z = s["logits"][t:t + step].double()
                z = z - z.logsumexp(dim=1, keepdim=True)
                entropy.append(-(z.exp() * z).sum(dim=1))
                lse.append(s["logits"][t:t + step].double().logsumexp(dim=1))
            s["lse"], s["entropy"] = torch.cat(lse).float(), torch.cat(entropy).float()
            s["dlogprob"] = -torch.rand((T,), generator=g, device="cuda")
            s["dentropy"] = -0.1 * torch.rand((T,), generator=g, device="cuda") if case["entropy"] else None
        return s
    T, V, H = case["T"], case["V"], case["H"]
    s["ids"] = _tokens(T, V, case["drop"], g)
    if kind == "embedding":
        dt = TABLES[case["type"]]
        s["table"] = torch.empty((V, H), dtype=dt, device="cuda")
        step = max(1, (1 << 27) // H)
        for v in range(0, V, step):
            x = torch.randn((min(step, V - v), H), generator=g, device="cuda")
            s["table"][v:v + step] = x.mul_(40).round_().clamp_(-127, 127).to(dt) if dt == torch.int8 else \
                x.mul_(100).clamp_(-448, 448).to(dt) if dt == torch.float8_e4m3fn else x.to(dt)
        n = case["scales"]
        s["row_scale"] = None if n == 0 else \
            0.01 + torch.rand((V,) if n == 1 else (V, n), generator=g, device="cuda")
        s["factor"] = math.sqrt(H)
    else:
        s["dout"] = _normal((T, H), FLOATS[case["type"]], g)
        s["factor"] = 1.0
    return s


# ---------------------------------------------------------------------------
# the plain forms, fp32
# ---------------------------------------------------------------------------
def _one_hot(s):
    """[T, L]: 1 where the token has the adapter."""
    return (s["ids"].unsqueeze(1) == torch.arange(s["a"].shape[0], device="cuda")).float()


def _factors(s):
    """Every adapter's rows as one matrix (A [L R, K] and B [N, L R]) and X A^T with zeros in the columns of
    adapters that a token does not have, [T, L, R]."""
    a, b = s["a"].float(), s["b"].float()
    a, b = a.flatten(0, 1), b.transpose(0, 1).reshape(b.shape[1], -1)
    hot = _one_hot(s).unsqueeze(2)
    v = torch.matmul(s["x"].float(), a.t()).view(hot.shape[0], hot.shape[1], -1) * hot
    return a, b, v, hot * s["scale"].unsqueeze(1)


def _adapter(s):
    if s["ids"].numel() <= 8:                       # few tokens take their adapter's rows one by one
        at = s["ids"].clamp(min=0).long()
        v = (s["a"][at].float() * s["x"].float().unsqueeze(1)).sum(dim=2)
        v = v * (s["scale"][at] * (s["ids"] >= 0)).unsqueeze(1)
        return (s["base"].float() + (s["b"][at].float() * v.unsqueeze(1)).sum(dim=2)).to(torch.bfloat16)
    _, b, v, _ = _factors(s)
    v = (v * s["scale"].unsqueeze(1)).flatten(1)
    return (s["base"].float() + torch.matmul(v, b.t())).to(torch.bfloat16)


def _adapter_gradient(s):
    a, b, v, hot = _factors(s)
    x, dy = s["x"].float(), s["dy"].float()
    u = (torch.matmul(dy, b).view(v.shape) * hot).flatten(1)
    dx = s["base"].float() + torch.matmul(u, a)
    db = torch.matmul(dy.t(), (v * hot).flatten(1)).view(b.shape[0], v.shape[1], -1)
    return {"dx": dx.to(torch.bfloat16), "da": torch.matmul(u.t(), x).view(s["a"].shape),
            "db": db.transpose(0, 1).contiguous()}


def _best(x, k):
    """The k largest of each row, ties to the lowest index: the values' bits as ordered integers, the index
    in the lower half."""
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    order = (order << 32) + (0xFFFFFFFF - torch.arange(x.shape[1], device=x.device))
    return 0xFFFFFFFF - (torch.topk(order, k, dim=1).values & 0xFFFFFFFF)


def _logprobs(s):
    x, target = s["logits"].float(), s["target"]
    m = x.amax(dim=1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    total = e.sum(dim=1, keepdim=True)
    log_total = torch.log(total)
    weighted = torch.where(e > 0, e * d, torch.zeros((), device=x.device)).sum(dim=1, keepdim=True)
    ids = _best(x, s["case"]["top"])
    at = target.clamp(min=0).unsqueeze(1)
    logprob = torch.where(target.unsqueeze(1) >= 0, d.gather(1, at) - log_total, torch.zeros((), device=x.device))
    return {"logprob": logprob.squeeze(1), "entropy": (log_total - weighted / total).squeeze(1),
            "lse": (m + log_total).squeeze(1), "top": d.gather(1, ids) - log_total, "ids": ids.to(torch.int32)}


def _logprobs_gradient(s):
    x, target = s["logits"].float(), s["target"]
    z = x - s["lse"].unsqueeze(1)
    p = torch.exp(z)
    there = target >= 0
    g = torch.where(there, s["dlogprob"], torch.zeros((), device=x.device)).unsqueeze(1)
    out = -p * g
    if s["dentropy"] is not None:
        out -= torch.where(p > 0, p * (z + s["entropy"].unsqueeze(1)), torch.zeros((), device=x.device)) \
            * s["dentropy"].unsqueeze(1)
    out.scatter_add_(1, target.clamp(min=0).unsqueeze(1), g)
    return out.to(s["logits"].dtype)


def _rows(table, ids):
    """Rows by index, of any type."""
    if table.dtype == torch.float8_e4m3fn:
        return table.view(torch.uint8)[ids].view(table.dtype).float()
    return table[ids].float()


def _embedding(s):
    ids = s["ids"].clamp(min=0)
    v = _rows(s["table"], ids)
    if s["row_scale"] is not None:
        sc = s["row_scale"][ids]
        v = (v.view(v.shape[0], s["case"]["scales"], -1) * sc.view(sc.shape[0], -1, 1)).view(v.shape)
    v = v * s["factor"] * (s["ids"] >= 0).unsqueeze(1)
    return v.to(s["table"].dtype if s["row_scale"] is None else torch.bfloat16)


def _embedding_gradient(s):
    ids, dout = s["ids"], s["dout"]
    out = torch.zeros((s["case"]["V"], dout.shape[1]), device=dout.device)
    there = (ids >= 0).unsqueeze(1)
    out.index_put_((ids.clamp(min=0),), dout.float() * there * s["factor"], accumulate=True)
    return out.to(dout.dtype)


_PLAIN = {"adapter": _adapter, "adapter gradient": _adapter_gradient, "logprobs": _logprobs,
          "logprobs gradient": _logprobs_gradient, "embedding": _embedding,
          "embedding gradient": _embedding_gradient}


def _own(s):
    import int8_gemm_linear_amd as q
    case = s["case"]
    kind = case["kind"]
    if kind == "adapter":
        return q.lora_mm(s["x"], s["a"], s["b"], s["ids"], scale=s["scale"], base=s["base"])
    if kind == "adapter gradient":
        dx, da, db = q.lora_mm_backward(s["dy"], s["x"], s["a"], s["b"], s["ids"], scale=s["scale"], base=s["base"])
        return {"dx": dx, "da": da, "db": db}
    if kind == "logprobs":
        logprob, entropy, lse, top, ids = q.token_logprobs(s["logits"], s["target"], top=case["top"])
        return {"logprob": logprob, "entropy": entropy, "lse": lse, "top": top, "ids": ids}
    if kind == "logprobs gradient":
        return q.token_logprobs_backward(s["dlogprob"], s["logits"], s["target"], s["lse"], entropy=s["entropy"],
                                         dentropy=s["dentropy"])
    if kind == "embedding":
        return q.embedding(s["ids"], s["table"], row_scale=s["row_scale"], scale=s["factor"])
    return q.embedding_backward(s["dout"], s["ids"], case["V"], scale=s["factor"])


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["kind"]](state)


def exact(case, seed):
    """The outputs from the definitions in fp64."""
    kind = case["kind"]
    s = prepare(case, seed)
    f64 = torch.float64
    if kind.startswith("adapter"):
        out = s["base"].double()
        da, db = (torch.zeros(s[k].shape, dtype=f64, device="cuda") for k in ("a", "b"))
        for i in range(case["L"]):
            t = torch.nonzero(s["ids"] == i).squeeze(1)
            if t.numel() == 0:
                continue
            x, a, b, scale = s["x"][t].double(), s["a"][i].double(), s["b"][i].double(), s["scale"][i].double()
            v = x @ a.t()
            if kind == "adapter":
                out[t] += scale * (v @ b.t())
                continue
            dy = s["dy"][t].double()
            u = scale * (dy @ b)
            out[t] += u @ a
            da[i] = u.t() @ x
            db[i] = scale * (dy.t() @ v)
        return out if kind == "adapter" else {"dx": out, "da": da, "db": db}
    if kind.startswith("logprobs"):
        parts = []
        step = max(1, (1 << 26) // case["V"])
        for t in range(0, case["T"], step):
            x, target = s["logits"][t:t + step].double(), s["target"][t:t + step]
            lse = torch.logsumexp(x, dim=1)
            logp = x - lse.unsqueeze(1)
            p = logp.exp()
            plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
            entropy = -plogp.sum(dim=1)
            row = torch.nonzero(target >= 0).squeeze(1)
            if kind == "logprobs":
                logprob = torch.zeros(lse.shape, dtype=f64, device="cuda")
                logprob[row] = logp[row, target[row]]
                parts.append((logprob, entropy, lse, torch.topk(logp, case["top"], dim=1).values))
                continue
            out = torch.zeros_like(p)
            out[row] -= s["dlogprob"][t:t + step].double()[row].unsqueeze(1) * p[row]
            out[row, target[row]] += s["dlogprob"][t:t + step].double()[row]
            if s["dentropy"] is not None:
                out -= s["dentropy"][t:t + step].double().unsqueeze(1) * (plogp + p * entropy.unsqueeze(1))
            parts.append(out)
        if kind == "logprobs gradient":
            return torch.cat(parts)
        return {**{k: torch.cat([p[j] for p in parts]) for j, k in enumerate(("logprob", "entropy", "lse", "top"))},
                "ids": None}
    there = torch.nonzero(s["ids"] >= 0).squeeze(1)
    ids = s["ids"][there]
    if kind == "embedding":
        out = torch.zeros((case["T"], case["H"]), dtype=f64, device="cuda")
        t = s["table"]
        v = (t.view(torch.uint8)[ids].view(t.dtype) if t.dtype == torch.float8_e4m3fn else t[ids]).double()
        if s["row_scale"] is not None:
            scale = s["row_scale"][ids].double().view(ids.numel(), -1)
            v *= scale.repeat_interleave(case["H"] // case["scales"], dim=1)
        out[there] = v * s["factor"]
        return out
    out = torch.zeros((case["V"], case["H"]), dtype=f64, device="cuda")
    out.index_add_(0, ids, s["dout"][there].double() * s["factor"])
    return out


def work(case):
    kind, T = case["kind"], case["T"]
    there = T * (1 - case["drop"])
    if kind.startswith("adapter"):
        K, N, R = case["K"], case["N"], case["R"]
        used = case["requests"] * R * (K + N)
        if kind == "adapter":
            return {"bytes": 2 * there * K + 2 * used + 4 * T * N + 4 * T, "flops": 2 * there * R * (K + N)}
        # x and dy read, base read and dx written; the gradients of all adapters
        return {"bytes": 2 * there * (K + N) + 4 * T * K + 2 * used + 4 * case["L"] * R * (K + N) + 4 * T,
                "flops": 2 * there * R * (3 * K + 2 * N)}
    if kind == "logprobs":
        # exponential, weighting and two sums for each logit
        return {"bytes": T * (case["V"] * FLOATS[case["type"]].itemsize + 20 + 8 * case["top"]),
                "flops": 5 * T * case["V"]}
    if kind == "logprobs gradient":
        return {"bytes": T * (2 * case["V"] * FLOATS[case["type"]].itemsize + 24), "flops": 6 * T * case["V"]}
    V, H, size = case["V"], case["H"], TABLES[case["type"]].itemsize
    if kind == "embedding":
        return {"bytes": there * (H * size + 4 * case["scales"]) + T * (H * (2 if case["scales"] else size) + 8),
                "flops": 2 * there * H}
    return {"bytes": there * H * size + V * H * size + 8 * T, "flops": there * H}
