"""Cases of the serving-step operators: the batch plan, the 4-bit key/value cache's store and read, and attention over it.

The cache holds keys and values as 4-bit codes.  A head's D dims form groups of 64; a (token, head, group) keeps
``m = f16(min)``, ``s = f16((max - min) * (1 / 15))`` and codes ``c = clamp(rint((x - m) * (1 / s)), 0, 15)`` (0 where s is 0),
each step rounded to float32, and stands for ``s * c + m``.  Pages are [num_pages, kv_heads, page_size / 16, tile] bytes, a
tile being 16 tokens: key codes (8 D bytes) | key (s, m) pairs [16, D / 64, 2] f16 | value codes | value pairs.
Inside a plane of W = min(D, 128) dims the key codes of token t are [16 t][c 0..3][word 0..W/32): nibble i of word w is dim
64 (w / 2) + 16 c + 8 (w % 2) + i; the value codes are [h 0..1][g 0..7][c 0..3][word 0..W/32) with nibble j of a word's low and
high half being dim 64 (w / 2) + 8 g + 4 (w % 2) + j of the tokens 8 h + 2 c and 8 h + 2 c + 1.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one decode step's plan: 64 requests, a row each, as the decode qkv workload has them
        {"name": "plan decode 64", "kind": "plan", "B": 64, "ctx_lo": 1, "ctx_hi": 4096, "new_lo": 1, "new_hi": 1,
         "page": 16, "spare": 0},
        # a large mixed step: decode rows and prompt chunks of 512 requests in one padded batch
        {"name": "plan mixed 512", "kind": "plan", "B": 512, "ctx_lo": 1, "ctx_hi": 32768, "new_lo": 1, "new_hi": 1024,
         "page": 64, "spare": 37},
        # the new keys and values of a decode step (8 kv heads of 128: the 1024-wide k and v slices)
        {"name": "store decode 64", "kind": "store", "n": 64, "heads": 8, "q_heads": 32, "D": 128, "page": 16,
         "dtype": "bf16", "seq": 1},
        # a prefill step of 8192 tokens
        {"name": "store prefill 8192", "kind": "store", "n": 8192, "heads": 8, "q_heads": 32, "D": 128, "page": 64,
         "dtype": "bf16", "seq": 512},
        # cached prefixes read back, rows in any order
        {"name": "read 32765 rows", "kind": "read", "n": 32765, "heads": 8, "D": 64, "page": 32, "dtype": "f16"},
        # one user, short prompt: latency
        {"name": "attend 1 x 300", "kind": "attend", "B": 1, "ctx_lo": 299, "ctx_hi": 299, "new_lo": 1, "new_hi": 1,
         "q_heads": 32, "heads": 8, "D": 128, "page": 16, "window": 0, "dtype": "bf16"},
        # the decode qkv workload's batch over contexts of a few hundred to 8 thousand tokens
        {"name": "attend decode 64", "kind": "attend", "B": 64, "ctx_lo": 255, "ctx_hi": 8191, "new_lo": 1, "new_hi": 1,
         "q_heads": 32, "heads": 8, "D": 128, "page": 16, "window": 0, "dtype": "bf16"},
        # one long document
        {"name": "attend 1 x 131072", "kind": "attend", "B": 1, "ctx_lo": 131071, "ctx_hi": 131071, "new_lo": 1,
         "new_hi": 1, "q_heads": 32, "heads": 8, "D": 128, "page": 64, "window": 0, "dtype": "bf16"},
        # many requests of a model without shared heads (the 5120-wide projections: 40 heads of 128)
        {"name": "attend decode 256, 40 heads", "kind": "attend", "B": 256, "ctx_lo": 16, "ctx_hi": 2047, "new_lo": 1,
         "new_hi": 1, "q_heads": 40, "heads": 40, "D": 128, "page": 16, "window": 0, "dtype": "bf16"},
        # prompts of 16 to 1024 tokens, as the prefill workload's segments
        {"name": "attend prompts 32", "kind": "attend", "B": 32, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 16, "new_hi": 1024,
         "q_heads": 32, "heads": 8, "D": 128, "page": 16, "window": 0, "dtype": "bf16"},
        # one prompt of 8192 tokens
        {"name": "attend prompt 8192", "kind": "attend", "B": 1, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 8192, "new_hi": 8192,
         "q_heads": 32, "heads": 8, "D": 128, "page": 64, "window": 0, "dtype": "bf16"},
        # chunks of prompts over what is cached already, with a sliding window
        {"name": "attend chunks over 16k", "kind": "attend", "B": 4, "ctx_lo": 4096, "ctx_hi": 16384, "new_lo": 512,
         "new_hi": 1021, "q_heads": 16, "heads": 2, "D": 128, "page": 32, "window": 8192, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(max(w["bytes"], w["flops"] / 50) for w in map(work, listed()))
    while True:
        kind = rng.choice(["plan", "store", "read", "decode", "decode", "decode", "several", "prefill", "chunk"])
        if kind == "plan":
            lo, chi = rng.choice([(1, 1), (1, 4), (1, 1024), (16, 2048)]), _log(rng, 16, 65536)
            case = {"kind": "plan", "B": _log(rng, 1, 1024), "ctx_lo": rng.randint(0, 16), "ctx_hi": chi, "new_lo": lo[0],
                    "new_hi": lo[1], "page": rng.choice([16, 32, 64, 128]), "spare": rng.randint(0, 64)}
            if sum(n for _, n in _lengths(case)) > 131072 or case["B"] * (chi // case["page"] + 70) > 1 << 22:
                continue
        elif kind in ("store", "read"):
            case = {"kind": kind, "n": _log(rng, 1, 32768), "heads": rng.choice([1, 2, 4, 8, 10, 40]),
                    "D": rng.choice([64, 128, 256]), "page": rng.choice([16, 32, 64, 128]), "dtype": rng.choice(["bf16", "f16"])}
            if kind == "store":
                case["q_heads"], case["seq"] = case["heads"] * rng.choice([1, 2, 4]), _log(rng, 1, 4096)
            if case["n"] * case["heads"] * case["D"] > 1 << 26:
                continue
        else:
            heads, group = rng.choice([1, 2, 4, 8, 10, 40]), rng.choice([1, 2, 4, 5, 8, 16])
            if heads * group > 64:
                continue
            B, ctx, new = {"decode": (_log(rng, 1, 512), _log(rng, 1, 131072), (1, 1)),
                           "several": (_log(rng, 1, 128), _log(rng, 16, 32768), (1, rng.randint(2, 8))),
                           "prefill": (_log(rng, 1, 64), 0, (rng.randint(1, 64), _log(rng, 64, 8192))),
                           "chunk": (_log(rng, 1, 16), _log(rng, 64, 32768), (rng.randint(1, 32), _log(rng, 32, 2048)))}[kind]
            case = {"kind": "attend", "B": B, "ctx_lo": ctx // rng.choice([1, 4, 64]), "ctx_hi": ctx, "new_lo": new[0],
                    "new_hi": new[1], "q_heads": heads * group, "heads": heads, "D": rng.choice([64, 128, 128, 256]),
                    "page": rng.choice([16, 32, 64, 128]), "window": rng.choice([0, 0, 0, 100, 4096]),
                    "dtype": rng.choice(["bf16", "bf16", "f16"])}
            longest, most = max(c + n for c, n in _lengths(case)), max(n for _, n in _lengths(case))
            if B * most * longest * heads * group > 1.5e9 or B * longest * heads * case["D"] > 2e9:
                continue
        w = work(case)
        if max(w["bytes"], w["flops"] / 50) <= top:
            return case


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, even in their logarithm (from 1 on)."""
    a, b = math.log(max(lo, 1)), math.log(max(hi, 1))
    got = [int(round(math.exp(a + (b - a) * (i + 0.5) / n))) for i in range(n)]
    return [min(max(x, lo), hi) for x in got]


def _lengths(case):
    """(cached, new) tokens of the requests; long contexts go with short additions."""
    B = case["B"]
    return list(zip(_spread(case["ctx_lo"], case["ctx_hi"], B), reversed(_spread(case["new_lo"], case["new_hi"], B))))


def _row_bytes(D):
    return 2 * (D // 2 + 4 * (D // 64))


def work(case):
    if case["kind"] == "plan":
        lens, P = _lengths(case), case["page"]
        rows = sum(n for _, n in lens) + case["spare"]
        pages = sum(-(-(c + n) // P) - -(-c // P) for c, n in lens)
        return {"bytes": 12 * case["B"] + 8 * pages + 20 * rows + 8 * case["B"] + 4 * case["B"] + 8, "flops": 0}
    per = case["heads"] * case["D"] * 4
    if case["kind"] == "store":
        return {"bytes": case["n"] * (2 * per + 2 * case["heads"] * _row_bytes(case["D"]) + 8), "flops": 0}
    if case["kind"] == "read":
        return {"bytes": case["n"] * (per + case["heads"] * _row_bytes(case["D"]) + 8), "flops": 0}
    D, w, tokens, pairs, rows = case["D"], case["window"], 0, 0, 0
    for c, n in _lengths(case):
        span = w or c + n
        tokens += min(c + n, n - 1 + span)
        full = max(0, min(n, c + n - span))  # rows with the whole window
        pairs += full * span + sum(range(c + 1, c + n - full + 1))
        rows += n
    return {"bytes": 2 * rows * case["q_heads"] * D * 2 + tokens * case["heads"] * _row_bytes(D),
            "flops": 4 * D * case["q_heads"] * pairs}


# ------------------------------------------------------------ cache layout --

def _tile_bytes(D):
    return 16 * _row_bytes(D)


def _key_order(D):
    """The (token * D + dim) of each key nibble of a tile, in memory order."""
    W = min(D, 128)
    p, t, c, w, i = np.meshgrid(np.arange(D // W), np.arange(16), np.arange(4), np.arange(W // 32), np.arange(8), indexing="ij")
    return (t * D + p * W + 64 * (w // 2) + 16 * c + 8 * (w % 2) + i).reshape(-1)


def _value_order(D):
    W = min(D, 128)
    p, h, g, c, w, o, j = np.meshgrid(np.arange(D // W), np.arange(2), np.arange(8), np.arange(4), np.arange(W // 32),
                                      np.arange(2), np.arange(4), indexing="ij")
    return ((8 * h + 2 * c + o) * D + p * W + 64 * (w // 2) + 8 * g + 4 * (w % 2) + j).reshape(-1)


def _quantise(x):
    """Codes (uint8) and the f16 pairs of [..., D] values."""
    g = x.float().unflatten(-1, (-1, 64))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    m, s = lo.half(), ((hi - lo) * (1.0 / 15.0)).half()
    r = torch.where(s > 0, 1.0 / s.float(), torch.zeros_like(lo))
    codes = torch.clamp(torch.round((g - m.float()) * r), 0, 15).to(torch.uint8)
    return codes.flatten(-2), torch.cat([s, m], -1)


def _fill(pages, k, v, tiles):
    """Whole tiles of keys and values [tiles, 16, heads, D] put into the cache at the flat tile numbers."""
    D, H = k.shape[-1], k.shape[-2]
    page_tiles = pages.shape[2]
    for x, order, at in ((k, _key_order(D), 0), (v, _value_order(D), _tile_bytes(D) // 2)):
        codes, pairs = _quantise(x)
        order = torch.from_numpy(order).to(x.device)
        nib = codes.permute(0, 2, 1, 3).reshape(len(x), H, -1)[..., order].unflatten(-1, (-1, 2))
        both = torch.cat([nib[..., 0] | nib[..., 1] << 4, pairs.permute(0, 2, 1, 3, 4).reshape(len(x), H, -1).view(torch.uint8)], -1)
        pages[tiles // page_tiles, :, tiles % page_tiles, at:at + both.shape[-1]] = both


# ----------------------------------------------------------------- prepare --

def _random_pages(g, num_pages, heads, page, D):
    """A cache as a server's: what no request owns holds stale bytes."""
    return torch.randint(0, 256, (num_pages, heads, page // 16, _tile_bytes(D)), dtype=torch.uint8, device="cuda", generator=g)


def _keys(g, shape, dtype):
    """Keys with a few strong channels; values are plain normal."""
    strong = torch.where(torch.rand(shape[-2:], device="cuda", generator=g) < 0.04, 4.0, 0.0)
    return (torch.randn(shape, device="cuda", generator=g) + strong * torch.randn(shape[-2:], device="cuda", generator=g)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dev = "cuda"

    def ints(x, dtype=np.int32):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).to(dev)

    if case["kind"] == "plan":
        lens = np.array(_lengths(case))[rng.permutation(case["B"])]
        P, B = case["page"], case["B"]
        n = int(lens[:, 1].sum()) + case["spare"]
        held, need = -(-lens[:, 0] // P), -(-lens.sum(1) // P)
        order = rng.permutation(int(need.sum()) + 64)
        table = np.full((B, int(need.max()) + 3), -1)
        at = np.concatenate([[0], np.cumsum(held)])
        for b in range(B):
            table[b, :held[b]] = order[at[b]:at[b + 1]]
        left = order[at[-1]:]
        return {"case": case, "ctx": ints(lens[:, 0]), "new": ints(lens[:, 1]), "slot": ints(rng.integers(-1, 16, B)),
                "table": ints(table), "free": ints(left), "count": ints([len(left)]), "left": ints([0]), "n": n}
    D, H, P, dtype = case["D"], case["heads"], case["page"], DTYPES[case["dtype"]]
    if case["kind"] in ("store", "read"):
        n = case["n"]
        state = {"case": case, "n": n}
        if case["kind"] == "store":  # requests of `seq` new tokens each, begun anywhere in their pages
            per = -(-(case["seq"] + P - 1) // P) * P
            reqs = -(-n // case["seq"])
            num_pages = reqs * (per // P) + 3
            start = rng.integers(0, P, reqs)
            own_pages = rng.permutation(num_pages)[:reqs * (per // P)].reshape(reqs, -1)
            i = np.arange(n)
            pos = start[i // case["seq"]] + i % case["seq"]
            slots = own_pages[i // case["seq"], pos // P] * P + pos % P
            Q = case["q_heads"]
            state["qkv"] = torch.cat([torch.randn(n, Q, D, device=dev, generator=g).to(dtype), _keys(g, (n, H, D), dtype),
                                      torch.randn(n, H, D, device=dev, generator=g).to(dtype)], 1).view(n, -1)
            state["k"] = state["qkv"][:, Q * D:(Q + H) * D].unflatten(1, (H, D))
            state["v"] = state["qkv"][:, (Q + H) * D:].unflatten(1, (H, D))
            state["pages"] = _random_pages(g, num_pages, H, P, D)
        else:
            num_pages = -(-n // P) + 2
            slots = rng.permutation(num_pages * P)[:n]
            state["pages"] = _random_pages(g, num_pages, H, P, D)
            k, v = _keys(g, (num_pages * P, H, D), dtype), torch.randn(num_pages * P, H, D, device=dev, generator=g)
            _fill(state["pages"], k.view(-1, 16, H, D), v.view(-1, 16, H, D), torch.arange(num_pages * P // 16, device=dev))
        state["slots"] = ints(slots, np.int64)
        state["places"], state["dims"] = _byte_places(D, dev), _token_dims(D, dev)
        state["k_out"], state["v_out"] = (torch.empty(n, H, D, dtype=dtype, device=dev) for _ in range(2))
        return state
    lens = np.array(_lengths(case))[rng.permutation(case["B"])]
    seq, new = lens.sum(1), lens[:, 1]
    n, Q = int(new.sum()), case["q_heads"]
    need = -(-seq // P)
    num_pages = int(need.sum()) + 5
    order = rng.permutation(num_pages)
    at = np.concatenate([[0], np.cumsum(need)])
    table = np.full((case["B"], int(need.max()) + 1), -1)
    for b in range(case["B"]):
        table[b, :need[b]] = order[at[b]:at[b + 1]]
    pages = _random_pages(g, num_pages, H, P, D)
    for b in range(case["B"]):  # the requests' tokens; the rest of their last tiles stays stale
        tiles = -(-int(seq[b]) // 16)
        where = torch.from_numpy(table[b].repeat(P // 16) * (P // 16) + np.tile(np.arange(P // 16), table.shape[1]))[:tiles].to(dev)
        for a in range(0, tiles, 8192):
            e = min(tiles, a + 8192)
            k, v = _keys(g, ((e - a) * 16, H, D), dtype), torch.randn((e - a) * 16, H, D, device=dev, generator=g).to(dtype)
            _fill(pages, k.view(-1, 16, H, D), v.view(-1, 16, H, D), where[a:e])
    qkv = torch.randn(n, (Q + 2 * H) * D, device=dev, generator=g).to(dtype)
    return {"case": case, "n": n, "pages": pages, "table": ints(table), "seq": ints(seq),
            "dims": [ints(np.argsort(order), np.int64) for order in (_key_order(D), _value_order(D))],
            "row_start": ints(np.concatenate([[0], np.cumsum(new)])), "max_new": int(new.max()), "max_seq": int(seq.max()),
            "qkv": qkv, "q": qkv[:, :Q * D].unflatten(1, (Q, D)), "out": torch.empty(n, Q, D, dtype=dtype, device=dev)}


# --------------------------------------------------------------------- run --

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _run_own(kind, state)
    return {"plan": _plain_plan, "store": _plain_store, "read": _plain_read, "attend": _plain_attend}[kind](state)


def _run_own(kind, st):
    import lora_delta_gb300 as ld
    case = st["case"]
    if kind == "plan":
        if "plan" not in st:  # the output buffers that a program keeps
            st["plan"] = ld.BatchPlan(case["B"], st["n"], case["page"])
        p = st["plan"]
        ld.lora_batch_plan(p, st["ctx"], st["new"], st["table"], req_slot=st["slot"], free_pages=st["free"],
                           free_count=st["count"], free_left=st["left"])
        return [p.row_start, p.row_req, p.position, p.slot_map, p.seq_slot, p.seq_len, st["table"], st["left"]]
    if "cache" not in st:  # the handle of the cache's memory
        st["cache"] = ld.Kv4Cache(st["pages"], case["page"], case["D"], DTYPES[case["dtype"]])
    if kind == "attend":
        ld.lora_kv4_attention(st["out"], st["q"], st["cache"], st["table"], st["row_start"], st["seq"], st["max_new"],
                              window=case["window"])
        return st["out"]
    if kind == "store":
        ld.lora_kv4_append(st["cache"], st["k"], st["v"], st["slots"])
    ld.lora_kv4_read(st["cache"], st["k_out"], st["v_out"], st["slots"])
    return [st["k_out"], st["v_out"]]


def _plain_plan(st):
    P, n = st["case"]["page"], st["n"]
    ctx, new, table = st["ctx"].long(), st["new"].long(), st["table"]
    seq = ctx + new
    ends = torch.cumsum(new, 0)
    held, need = (ctx + P - 1) // P, (seq + P - 1) // P
    first = torch.cumsum(need - held, 0) - (need - held)
    col = torch.arange(table.shape[1], device=table.device)[None]
    fresh = (col >= held[:, None]) & (col < need[:, None])
    at = st["count"].long() - 1 - (first[:, None] + col - held[:, None])
    page = torch.where(at >= 0, st["free"][at.clamp(min=0, max=st["free"].numel() - 1)], -1)
    table.copy_(torch.where(fresh, page, table))
    row = torch.arange(n, device=table.device)
    req = torch.searchsorted(ends, row, right=True)
    real = req < len(ctx)
    r = req.clamp(max=len(ctx) - 1)
    pos = torch.where(real, ctx[r] + row - (ends - new)[r], 0)
    own_page = table[r, pos // P].long()
    slot = torch.where(real & (own_page >= 0), own_page * P + pos % P, -1)
    left = (st["count"].long() - (need - held).sum()).clamp(min=0)
    return [torch.cat([torch.zeros_like(ends[:1]), ends]).int(), torch.where(real, req, -1).int(), pos.int(), slot,
            torch.where(real, st["slot"][r], -1).int(), seq.int(), table, left.int()]


def _byte_places(D, dev):
    """For each token of a tile: the bytes of its key codes, key pairs, value codes and value pairs, [4][16, bytes]."""
    places = []
    for order, base in ((_key_order(D), 0), (_value_order(D), _tile_bytes(D) // 2)):
        token = order[::2] // D
        places.append(torch.from_numpy(base + np.argsort(token, kind="stable").reshape(16, -1)).to(dev))
        pair = np.arange(16 * 4 * (D // 64)).reshape(16, -1)
        places.append(torch.from_numpy(base + 8 * D + pair).to(dev))
    return places


def _token_dims(D, dev):
    """The dims of a token's nibbles in the order of its bytes (by token of the tile): keys, values."""
    got = []
    for order in (_key_order(D), _value_order(D)):
        o = order.reshape(-1, 2)
        o = o[np.argsort(o[:, 0] // D, kind="stable")].reshape(16, -1) % D
        got.append(torch.from_numpy(o).to(dev))
    return got


def _flat_at(pages, slots, P):
    """Byte offset of the tile of (row, head), and the token within it."""
    page, off, H = slots // P, slots % P, pages.shape[1]
    tile = (page[:, None] * H + torch.arange(H, device=pages.device)) * (P // 16) + (off // 16)[:, None]
    return tile * pages.shape[3], off % 16


def _plain_store(st):
    base, tok = _flat_at(st["pages"], st["slots"], st["case"]["page"])
    flat, places, dims = st["pages"].view(-1), st["places"], st["dims"]

    def put(x, codes_at, pairs_at, dim):
        codes, pairs = _quantise(x)
        nib = torch.gather(codes, 2, dim[tok][:, None].expand_as(codes)).unflatten(-1, (-1, 2))
        flat[base[..., None] + codes_at[tok][:, None]] = nib[..., 0] | nib[..., 1] << 4
        flat[base[..., None] + pairs_at[tok][:, None]] = pairs.reshape(*pairs.shape[:2], -1).view(torch.uint8)

    put(st["k"], places[0], places[1], dims[0])
    put(st["v"], places[2], places[3], dims[1])
    return _plain_read(st)


def _plain_read(st):
    D, P, dtype, dev = st["case"]["D"], st["case"]["page"], DTYPES[st["case"]["dtype"]], st["pages"].device
    base, tok = _flat_at(st["pages"], st["slots"], P)
    flat, places, dims = st["pages"].view(-1), st["places"], st["dims"]

    def get(codes_at, pairs_at, dim):
        b = flat[base[..., None] + codes_at[tok][:, None]]
        codes = torch.empty(*b.shape[:2], D, dtype=torch.uint8, device=dev)
        codes.scatter_(2, dim[tok][:, None].expand_as(codes), torch.stack([b & 15, b >> 4], -1).flatten(-2))
        pairs = flat[base[..., None] + pairs_at[tok][:, None]].view(torch.float16).float().unflatten(-1, (-1, 2))
        return (codes.float().unflatten(-1, (-1, 64)) * pairs[..., :1] + pairs[..., 1:]).flatten(-2).to(dtype)

    return [get(places[0], places[1], dims[0]), get(places[2], places[3], dims[1])]


def _plain_tiles(part, inverse, D):
    """float32 values [..., 16, D] of a part (keys or values) of tiles."""
    codes = part[..., :8 * D]
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., inverse].unflatten(-1, (16, D // 64, 64))
    pairs = part[..., 8 * D:].contiguous().view(torch.float16).float().unflatten(-1, (16, D // 64, 2))
    return (codes.float() * pairs[..., :1] + pairs[..., 1:]).flatten(-2)


def _plain_attend(st):
    case, dev = st["case"], st["q"].device
    D, P, H, Q, B = case["D"], case["page"], case["heads"], case["q_heads"], case["B"]
    half, L = _tile_bytes(D) // 2, -(-st["max_seq"] // P) * P
    tiles = st["pages"][st["table"][:, :L // P].clamp(min=0).long()]  # [B, pages, H, tiles, bytes]
    seq, start = st["seq"].long(), st["row_start"].long()
    t = torch.arange(L, device=dev)
    inside = (t[None] < seq[:, None])[:, None, :, None]
    k = _plain_tiles(tiles[..., :half], st["dims"][0], D).permute(0, 2, 1, 3, 4, 5).reshape(B, H, L, D)
    v = _plain_tiles(tiles[..., half:], st["dims"][1], D).permute(0, 2, 1, 3, 4, 5).reshape(B, H, L, D)
    k, v = torch.where(inside, k, 0.0), torch.where(inside, v, 0.0)
    j = torch.arange(st["max_new"], device=dev)
    new = start[1:] - start[:-1]
    q = st["q"][(start[:-1, None] + j).clamp(max=st["n"] - 1)].float()  # [B, new, Q, D]
    q = q.unflatten(2, (H, Q // H)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = torch.matmul(q, k.transpose(-1, -2)).unflatten(2, (Q // H, -1)) * D ** -0.5
    pos = (seq - new)[:, None] + j
    seen = (t <= pos[..., None]) & inside[:, 0, :, 0][:, None]
    if case["window"]:
        seen &= t > pos[..., None] - case["window"]
    s = s.masked_fill(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    s = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.flatten(2, 3), v).unflatten(2, (Q // H, -1)) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, new, Q, D]
    row = torch.arange(st["n"], device=dev)
    req = torch.searchsorted(start[1:], row, right=True)
    return o[req, row - start[req]].to(DTYPES[case["dtype"]])


# ------------------------------------------------------------------- exact --

def _exact_values(tile, which, D):
    """64-bit values [..., 16, D] of a tile's keys (which 0) or values (1), element by element from the layout."""
    t = torch.arange(16, device=tile.device)[:, None]
    d = torch.arange(D, device=tile.device)[None]
    W = min(D, 128)
    plane, e = d // W, d % W
    group, r = e // 64, e % 64
    word_bytes = W // 8  # bytes of one lane's words
    if which == 0:
        byte = plane * 8 * W + t * (W // 2) + (r // 16) * word_bytes + (2 * group + (r % 16) // 8) * 4 + (r % 8) // 2
    else:
        byte = plane * 8 * W + (t // 8) * 4 * W + (r // 8) * 4 * word_bytes + (t % 8 // 2) * word_bytes \
            + (2 * group + (r % 8) // 4) * 4 + (t % 2) * 2 + (r % 4) // 2
    half = tile[..., which * _tile_bytes(D) // 2:(which + 1) * _tile_bytes(D) // 2]
    code = torch.bitwise_right_shift(half[..., byte.expand(16, D)].int(), (4 * (d % 2)).int()).bitwise_and(15).double()
    pairs = half[..., 8 * D:].contiguous().view(torch.float16).double().unflatten(-1, (16, D // 64, 2))
    return code * pairs[..., 0].repeat_interleave(64, -1) + pairs[..., 1].repeat_interleave(64, -1)


def exact(case, seed):
    if case["kind"] == "plan":
        return None  # whole numbers, compared as they are
    st = prepare(case, seed)
    D, P = case["D"], case["page"]
    if case["kind"] == "store":
        def rounded(x, dtype):
            return x.to(dtype).double()

        def back(x):
            x = x.double().unflatten(-1, (-1, 64))
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            m = rounded(lo, torch.float16)
            s = rounded(rounded(rounded(hi - lo, torch.float32) * float(np.float32(1 / 15)), torch.float32), torch.float16)
            r = rounded(1 / s, torch.float32)
            steps = rounded(rounded(x - m, torch.float32) * r, torch.float32)
            code = torch.where(s > 0, steps.round().clamp(0, 15), torch.zeros_like(x))
            return (s * code + m).flatten(-2)
        return [back(st["k"]), back(st["v"])]
    if case["kind"] == "read":
        page, off = st["slots"] // P, st["slots"] % P
        got = []
        for which in (0, 1):
            parts = [_exact_values(st["pages"][page[a:a + 2048], :, off[a:a + 2048] // 16], which, D)
                     [torch.arange(len(page[a:a + 2048]), device=page.device), :, off[a:a + 2048] % 16]
                     for a in range(0, len(page), 2048)]
            got.append(torch.cat(parts))
        return got
    H, Q = case["heads"], case["q_heads"]
    starts, seqs, table = st["row_start"].tolist(), st["seq"].tolist(), st["table"].long()
    if sum((starts[b + 1] - starts[b]) * seqs[b] for b in range(case["B"])) * Q * D > 4e12:
        return None
    out = torch.zeros(st["n"], Q, D, dtype=torch.float64, device=st["q"].device)
    for b in range(case["B"]):
        a, e, L = starts[b], starts[b + 1], seqs[b]
        tiles = st["pages"][table[b, :-(-L // P)]]
        for h in range(H):
            head = tiles[:, h].flatten(0, 1)
            k, v = (_exact_values(head, which, D).flatten(0, 1)[:L] for which in (0, 1))
            q = st["q"][a:e, h * (Q // H):(h + 1) * (Q // H)].double()
            logits = torch.einsum("ngd,td->ngt", q, k) / math.sqrt(D)
            where = torch.arange(L - (e - a), L, device=k.device)[:, None, None]
            t = torch.arange(L, device=k.device)
            hidden = (t > where) | ((t <= where - case["window"]) if case["window"] else torch.zeros_like(t > where))
            out[a:e, h * (Q // H):(h + 1) * (Q // H)] = torch.softmax(logits.masked_fill(hidden, -math.inf), -1) @ v
    return out
