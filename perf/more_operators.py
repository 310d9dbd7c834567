"""Cases of the routed-expert layer around the deltas: tokens sorted by expert and back, and the products with an epilogue.

A token t goes to the experts ``topk_ids[t, 0..k)``; pair p = t k + j.  Pairs are sorted by expert, stable in p, into rows:
``seg_start[e]`` is the first row of expert e, ``pair_row[p]`` the pair's row (-1: none), ``row_pair`` its inverse, ``row_expert`` and
``row_lora`` the row's expert and its token's adapter (-1 behind the last row).
  dispatch      rows[pair_row[t, j]] = x[t]
  combine       out[t] = residual[t] + sum_j w[t, j] rows[pair_row[t, j]]   (without w and residual: the gradient of dispatch)
  combine_grad  grad_rows[pair_row[t, j]] = w[t, j] grad_out[t],  grad_w[t, j] = grad_out[t] . rows[pair_row[t, j]]
  linear        out = act(x W^T + bias + delta) + residual; gated: act(gate) * up with W = [gate; up]
  experts       linear for the rows of each expert with its own W and bias
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one decode step of 64 requests through 64 experts, 8 a token (the MoE workloads' layer)
        {"name": "dispatch decode 64", "kind": "dispatch", "T": 64, "k": 8, "E": 64, "H": 2048, "pad": 0, "local": 0, "skew": 0.0,
         "dtype": "bf16"},
        # a prefill step of 8192 tokens, hidden size 4096, some experts twice as busy as others
        {"name": "dispatch prefill 8192", "kind": "dispatch", "T": 8192, "k": 8, "E": 64, "H": 4096, "pad": 0, "local": 0,
         "skew": 0.5, "dtype": "bf16"},
        # the way back of a decode step, padded to 64 rows
        {"name": "combine decode 64", "kind": "combine", "T": 64, "k": 8, "E": 64, "H": 2048, "pad": 3, "local": 0, "skew": 0.0,
         "dtype": "bf16", "weighted": True, "residual": True},
        # the gradient of the dispatch of a training step
        {"name": "combine 8192, no weights", "kind": "combine", "T": 8192, "k": 8, "E": 64, "H": 4096, "pad": 0, "local": 0,
         "skew": 0.5, "dtype": "bf16", "weighted": False, "residual": False},
        # the gradient of a small step, two experts a token
        {"name": "combine grad 509", "kind": "combine_grad", "T": 509, "k": 2, "E": 8, "H": 4096, "pad": 0, "local": 0, "skew": 0.5,
         "dtype": "f16"},
        # the gradient of a training step of the MoE workloads' layer
        {"name": "combine grad 8192", "kind": "combine_grad", "T": 8192, "k": 8, "E": 64, "H": 2048, "pad": 0, "local": 0,
         "skew": 0.5, "dtype": "bf16"},
        # one user's token through the decode workload's q, k and v projections: latency, and the weights' bytes
        {"name": "linear 1 row", "kind": "linear", "n": 1, "K": 4096, "N": 6144, "act": "none", "gated": False, "bias": True,
         "delta": False, "residual": False, "dtype": "bf16"},
        # the decode workload's batch
        {"name": "linear 64 rows", "kind": "linear", "n": 64, "K": 4096, "N": 6144, "act": "none", "gated": False, "bias": True,
         "delta": True, "residual": False, "dtype": "bf16"},
        # the down projection of the many-adapter workload's 1024 rows, with its residual
        {"name": "linear 1023 rows, down", "kind": "linear", "n": 1023, "K": 13824, "N": 5120, "act": "none", "gated": False,
         "bias": False, "delta": True, "residual": True, "dtype": "f16"},
        # the prefill workload's gate and up projections, with the adapters' delta and the activation
        {"name": "linear 8192 rows, gate and up", "kind": "linear", "n": 8192, "K": 4096, "N": 28672, "act": "silu", "gated": True,
         "bias": False, "delta": True, "residual": False, "dtype": "bf16"},
        # the experts' first product of a decode step
        {"name": "experts decode 64", "kind": "experts", "T": 64, "k": 8, "E": 64, "K": 2048, "N": 1536, "pad": 0, "local": 0,
         "skew": 0.0, "act": "silu", "gated": True, "bias": False, "delta": True, "residual": False, "dtype": "bf16"},
        # the experts' first product of the MoE workload's 2048 tokens
        {"name": "experts 2048 tokens", "kind": "experts", "T": 2048, "k": 8, "E": 64, "K": 2048, "N": 1536, "pad": 0, "local": 0,
         "skew": 0.5, "act": "silu", "gated": True, "bias": False, "delta": True, "residual": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        kind = rng.choice(["dispatch", "combine", "combine_grad", "linear", "linear", "experts", "experts"])
        case = {"kind": kind, "dtype": rng.choice(["bf16", "bf16", "f16"])}
        if kind != "linear":
            E = _log(rng, 2, 256)
            T, k = _log(rng, 1, 16384), rng.randint(1, min(E, 16))
            case.update(T=T, k=k, E=E, pad=rng.choice([0, 0, rng.randint(0, T - 1)]), skew=rng.choice([0.0, 0.5, 1.0]),
                        local=rng.choice([0, 0, rng.randint(1, E)]))
        if kind in ("dispatch", "combine", "combine_grad"):
            case["H"] = 8 * _log(rng, 8, 1024)
        if kind == "combine":
            case["weighted"], case["residual"] = rng.choice([True, True, False]), rng.choice([True, False])
        if kind in ("linear", "experts"):
            gated = rng.choice([True, False])
            case.update(K=8 * _log(rng, 8, 1792), N=(16 if gated else 8) * _log(rng, 4, 1792), gated=gated,
                        act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"] if gated else ["none", "none", "silu", "gelu", "gelu_tanh", "relu"]),
                        bias=rng.choice([True, False]), delta=rng.choice([True, False]), residual=rng.choice([True, False]))
        if kind == "linear":
            case["n"] = _log(rng, 1, 16384)
        if _cost(case) <= top and _memory(case) <= 6e9:
            return case


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 200)


def _memory(case):
    """Bytes of the inputs and outputs with the plain form's copies in 32 bits."""
    if case["kind"] == "linear":
        return 6 * (case["n"] * (case["K"] + 3 * case["N"]) + case["N"] * case["K"])
    P = case["T"] * case["k"]
    if case["kind"] == "experts":
        return 6 * (P * (case["K"] + 3 * case["N"]) + case["E"] * case["N"] * case["K"])
    return 6 * P * case["H"] * 2


def work(case):
    if case["kind"] in ("linear", "experts"):
        K, N = case["K"], case["N"]
        out = N // 2 if case["gated"] else N
        if case["kind"] == "linear":
            n, copies = case["n"], 1
        else:
            share = (case["local"] or case["E"]) / case["E"]
            n = int((case["T"] - case["pad"]) * case["k"] * share)
            # experts that some token reaches, for an even router
            copies = max(1, round(case["E"] * share * (1 - (1 - case["k"] / case["E"]) ** (case["T"] - case["pad"]))))
        per = 2 * (K + out + (N if case["delta"] else 0) + (out if case["residual"] else 0))
        return {"bytes": n * per + copies * 2 * N * (K + (1 if case["bias"] else 0)), "flops": 2 * n * K * N}
    T, P, H = case["T"], case["T"] * case["k"], case["H"]
    rows = int((T - case["pad"]) * case["k"] * (case["local"] or case["E"]) / case["E"])
    if case["kind"] == "dispatch":
        return {"bytes": 2 * H * (T - case["pad"] + rows) + 4 * P + 4 * T + 16 * P + 4 * (case["E"] + 1), "flops": 0}
    if case["kind"] == "combine":
        return {"bytes": 2 * H * (rows + T * (2 if case["residual"] else 1)) + P * (8 if case["weighted"] else 4),
                "flops": 2 * rows * H}
    return {"bytes": 2 * H * (2 * rows + T) + 12 * P, "flops": 3 * rows * H}


# ----------------------------------------------------------------- prepare --

def _route(case, g):
    """Router's choices [T, k], distinct for a token; padded tokens have none.  Experts' popularity differs by `skew`."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn(T, E, device="cuda", generator=g) + case["skew"] * torch.randn(E, device="cuda", generator=g)
    top, ids = torch.topk(logits, k, dim=1)
    if case["pad"]:
        ids[T - case["pad"]:] = -1
    return torch.softmax(top, 1).contiguous(), ids.int().contiguous()


def _expert_map(case, g):
    """The rank's local experts when it does not hold all: global number to local, -1 elsewhere."""
    if not case["local"]:
        return None
    m = torch.full((case["E"],), -1, dtype=torch.int32, device="cuda")
    here = torch.randperm(case["E"], device="cuda", generator=g)[:case["local"]].sort().values
    m[here] = torch.arange(case["local"], dtype=torch.int32, device="cuda")
    return m


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, kind = DTYPES[case["dtype"]], case["kind"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)

    st = {"case": case, "dtype": dtype}
    if kind != "linear":
        T, k = case["T"], case["k"]
        st["weights"], st["ids"] = _route(case, g)
        st["map"], st["E"] = _expert_map(case, g), case["local"] or case["E"]
        st["lora"] = torch.randint(-1, 8, (T,), dtype=torch.int32, device="cuda", generator=g)
        st["plan"] = _sort(st)  # (what a dispatch of this step has left)
        st["count"] = int(st["plan"][0][-1])
    if kind == "dispatch":
        st["x"], st["rows"] = normal(T, case["H"]), torch.zeros(T * k, case["H"], dtype=dtype, device="cuda")
    if kind in ("combine", "combine_grad"):
        st["rows"] = normal(T * k, case["H"])
        st["out"] = torch.zeros(T, case["H"], dtype=dtype, device="cuda")
    if kind == "combine":
        st["residual"] = normal(T, case["H"]) if case["residual"] else None
    if kind == "combine_grad":
        st["grad_out"] = normal(T, case["H"])
        st["grad_rows"] = torch.zeros(T * k, case["H"], dtype=dtype, device="cuda")
        st["grad_w"] = torch.zeros(T, k, device="cuda")
    if kind in ("linear", "experts"):
        K, N = case["K"], case["N"]
        out = N // 2 if case["gated"] else N
        n, shape = (case["n"], (N, K)) if kind == "linear" else (T * k, (st["E"], N, K))
        st["x"], st["w"] = normal(n, K), normal(*shape, std=K ** -0.5)
        st["bias"] = normal(*shape[:-1], std=0.1) if case["bias"] else None
        st["delta"] = normal(n, N, std=0.3) if case["delta"] else None
        st["residual"] = normal(n, out) if case["residual"] else None
        st["out"] = torch.zeros(n, out, dtype=dtype, device="cuda")
        st["segments"] = [0, n] if kind == "linear" else st["plan"][0].tolist()
    return st


def _sort(st):
    """seg_start, row_pair, pair_row, row_expert, row_lora of a routing."""
    case, ids, E = st["case"], st["ids"].long(), st["E"]
    key = torch.where(ids >= 0, ids if st["map"] is None else st["map"].long()[ids.clamp(min=0)], -1).flatten()
    key = torch.where(key >= 0, key, E)
    order = torch.sort(key, stable=True).indices
    seg = (key[:, None] < torch.arange(E + 1, device=key.device)).sum(0) if key.numel() * E < 1 << 24 else \
        torch.searchsorted(key[order], torch.arange(E + 1, device=key.device))
    inside = torch.arange(len(key), device=key.device) < seg[E]
    place = torch.empty_like(order)
    place[order] = torch.arange(len(key), device=key.device)
    return [seg.int(), torch.where(inside, order, -1).int(),
            torch.where(key < E, place, -1).int().view(ids.shape), torch.where(inside, key[order], -1).int(),
            torch.where(inside, st["lora"].long()[order // case["k"]], -1).int()]


# --------------------------------------------------------------------- run --

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _run_own(kind, state)
    return {"dispatch": _plain_dispatch, "combine": _plain_combine, "combine_grad": _plain_combine_grad, "linear": _plain_linear,
            "experts": _plain_linear}[kind](state)


def _run_own(kind, st):
    import lora_delta_gb300 as ld
    case = st["case"]
    if kind == "linear":
        ld.lora_linear(st["out"], st["x"], st["w"], bias=st["bias"], delta=st["delta"], residual=st["residual"],
                       activation=case["act"], gated=case["gated"])
        return st["out"]
    if "moe" not in st:  # the plan's buffers that a program keeps; all but a dispatch find them filled
        st["moe"] = ld.MoePlan(case["T"], case["k"], st["E"])
        if kind != "dispatch":
            p = st["moe"]
            for t, x in zip((p.seg_start, p.row_pair, p.pair_row, p.row_expert, p.row_lora), st["plan"]):
                t.copy_(x)
    p = st["moe"]
    if kind == "dispatch":
        ld.lora_moe_dispatch(st["rows"], st["x"], st["ids"], p, lora_ids=st["lora"], expert_map=st["map"])
        return [st["rows"], p.seg_start, p.row_pair, p.pair_row, p.row_expert, p.row_lora]
    if kind == "combine":
        ld.lora_moe_combine(st["out"], st["rows"], p, weights=st["weights"] if case["weighted"] else None, residual=st["residual"])
        return st["out"]
    if kind == "combine_grad":
        ld.lora_moe_combine_grad(st["grad_rows"], st["grad_w"], st["grad_out"], st["rows"], p, st["weights"])
        return [st["grad_rows"], st["grad_w"]]
    ld.lora_moe_linear(st["out"], st["x"], st["w"], p, bias=st["bias"], delta=st["delta"], residual=st["residual"],
                       activation=case["act"], gated=case["gated"])
    return st["out"]


def _plain_dispatch(st):
    plan = _sort(st)
    row_pair = plan[1].long()
    x = st["x"][row_pair.clamp(min=0) // st["case"]["k"]]
    st["rows"].copy_(torch.where((row_pair >= 0)[:, None], x, st["rows"]))
    return [st["rows"], *plan]


def _plain_combine(st):
    case, place = st["case"], st["plan"][2].long()
    total = torch.zeros(case["T"], case["H"], device=place.device)
    for j in range(case["k"]):
        y = st["rows"][place[:, j].clamp(min=0)].float()
        if case["weighted"]:
            y = y * st["weights"][:, j:j + 1]
        total += torch.where((place[:, j] >= 0)[:, None], y, 0.0)
    if case["residual"]:
        total = total + st["residual"].float()
    return total.to(st["dtype"])


def _plain_combine_grad(st):
    case, place = st["case"], st["plan"][2].long()
    g, grad_w = st["grad_out"].float(), torch.zeros(case["T"], case["k"], device=place.device)
    for j in range(case["k"]):
        there = place[:, j] >= 0
        y = st["rows"][place[:, j].clamp(min=0)].float()
        grad_w[:, j] = torch.where(there, (g * y).sum(1), 0.0)
    row_pair = st["plan"][1].long()
    p = row_pair.clamp(min=0)
    rows = g[p // case["k"]] * st["weights"].flatten()[p][:, None]
    st["grad_rows"].copy_(torch.where((row_pair >= 0)[:, None], rows.to(st["dtype"]), st["grad_rows"]))
    return [st["grad_rows"], grad_w]


def _activation(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_linear(st):
    case, ends = st["case"], st["segments"]
    for e in range(len(ends) - 1):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        w, bias = (st["w"], st["bias"]) if case["kind"] == "linear" else (st["w"][e], None if st["bias"] is None else st["bias"][e])
        z = st["x"][a:b].float() @ w.float().t()
        if bias is not None:
            z = z + bias.float()
        if case["delta"]:
            z = z + st["delta"][a:b].float()
        if case["gated"]:
            gate, up = z.chunk(2, 1)
            y = _activation(gate, case["act"]) * up
        else:
            y = _activation(z, case["act"])
        if case["residual"]:
            y = y + st["residual"][a:b].float()
        st["out"][a:b] = y.to(st["dtype"])
    return st["out"]


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "dispatch":
        # pair by pair on the host: the row of a pair is the number of pairs before it
        T, k = case["T"], case["k"]
        ids = st["ids"].cpu().flatten().tolist()
        local = list(range(case["E"])) if st["map"] is None else st["map"].cpu().tolist()
        lists = [[] for _ in range(st["E"])]
        for p, e in enumerate(ids):
            if e >= 0 and local[e] >= 0:
                lists[local[e]].append(p)
        pairs = [p for rows in lists for p in rows]
        rows = torch.zeros(T * k, case["H"], dtype=torch.float64, device="cuda")
        if pairs:
            rows[:len(pairs)] = st["x"].double()[torch.tensor(pairs, device="cuda") // k]
        return [rows, None, None, None, None, None]
    if case["kind"] in ("combine", "combine_grad"):
        row_pair = st["plan"][1][:st["count"]].long()
        token, w = row_pair // case["k"], st["weights"].double().flatten()[row_pair]
        y = st["rows"][:st["count"]].double()
        if case["kind"] == "combine":
            out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
            for a in range(0, case["H"], 512):  # (a part of the columns at a time)
                part = y[:, a:a + 512] * w[:, None] if case["weighted"] else y[:, a:a + 512]
                out[:, a:a + 512].index_add_(0, token, part)
            return out + st["residual"].double() if case["residual"] else out
        grad_w = torch.zeros(case["T"] * case["k"], dtype=torch.float64, device="cuda")
        grad_rows = torch.zeros(case["T"] * case["k"], case["H"], dtype=torch.float64, device="cuda")
        for a in range(0, st["count"], 8192):
            g = st["grad_out"][token[a:a + 8192]].double()
            grad_rows[a:a + len(g)] = g * w[a:a + 8192, None]
            grad_w[row_pair[a:a + 8192]] = torch.einsum("ph,ph->p", g, y[a:a + 8192])
        return [grad_rows, grad_w.view(case["T"], case["k"])]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    weights = st["w"][None] if case["kind"] == "linear" else st["w"]
    half = case["N"] // 2
    for e in range(len(weights)):
        a, b = st["segments"][e], st["segments"][e + 1]
        for r in range(a, b, 2048):
            s = min(b, r + 2048)
            z = torch.einsum("rk,nk->rn", st["x"][r:s].double(), weights[e].double())
            if case["bias"]:
                z += (st["bias"] if case["kind"] == "linear" else st["bias"][e]).double()
            if case["delta"]:
                z += st["delta"][r:s].double()
            first = z[:, :half] if case["gated"] else z
            y = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.sigmoid(v),
                 "gelu": lambda v: v * torch.special.ndtr(v),
                 "gelu_tanh": lambda v: v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}[case["act"]](first)
            if case["gated"]:
                y = y * z[:, half:]
            if case["residual"]:
                y += st["residual"][r:s].double()
            out[r:s] = y
    return out
