"""Plain 64-bit numpy forms of the serving-step operators, written element by element from the
header's definitions: the batch plan, the release of pages, the 4-bit cache and attention over it."""
from __future__ import annotations

import numpy as np

ERR_LENGTH, ERR_PAGE = 128, 256


# -------------------------------------------------------------------- plan --

def plan(ctx_len, new_len, req_slot, n_rows, P, table, max_pages, free=None, count=None):
    """Request by request; returns the outputs as a dict, with the table and the error bits."""
    table, B, err = table.copy(), len(ctx_len), 0
    out = {k: np.full(n_rows, -1, np.int64) for k in ("row_req", "slot_map", "seq_slot")}
    out["position"] = np.zeros(n_rows, np.int64)
    starts, seqs, row, taken = [0], [], 0, 0
    for b in range(B):
        ctx, new, cap = int(ctx_len[b]), int(new_len[b]), max_pages * P
        if ctx < 0 or new < 0 or ctx + new > cap:
            err |= ERR_LENGTH
        ctx = min(max(ctx, 0), cap)
        new = min(max(new, 0), cap - ctx)
        if row + new > n_rows:
            err |= ERR_LENGTH
            new = n_rows - row
        held = -(-ctx // P)
        for pg in range(held, -(-(ctx + new) // P)):
            if free is not None:
                at = count - 1 - taken
                table[b, pg] = free[at] if at >= 0 else -1
                taken += 1
        for j in range(new):
            page = table[b, (ctx + j) // P]
            if page < 0:
                err |= ERR_PAGE
            out["row_req"][row] = b
            out["position"][row] = ctx + j
            out["seq_slot"][row] = -1 if req_slot is None else req_slot[b]
            out["slot_map"][row] = -1 if page < 0 else int(page) * P + (ctx + j) % P
            row += 1
        starts.append(row)
        seqs.append(ctx + new)
    out.update(row_start=np.array(starts), seq_len=np.array(seqs, np.int64), table=table, err=err,
               left=None if free is None else max(0, count - taken))
    return out


def release(done, seq_len, P, table, max_pages, free, count):
    table, free, err = table.copy(), free.copy(), 0
    for b in range(len(done)):
        if not done[b]:
            continue
        pages = -(-int(seq_len[b]) // P)
        if seq_len[b] < 0 or pages > max_pages:
            err |= ERR_LENGTH
        for p in range(min(max(pages, 0), max_pages)):
            if table[b, p] < 0:
                continue
            if count >= len(free):
                err |= ERR_PAGE
                continue
            free[count] = table[b, p]
            count += 1
            table[b, p] = -1
    return table, free, count, err


# ------------------------------------------------------------------- cache --

def tile_bytes(D):
    return 2 * (8 * D + 64 * (D // 64))


def code_place(D, is_value):
    """(byte, bit shift) [16, D] of each code in a tile's half, token by token, dim by dim."""
    W, byte, shift = min(D, 128), np.zeros((16, D), int), np.zeros((16, D), int)
    for t in range(16):
        for d in range(D):
            plane, e = divmod(d, W)
            group, r = divmod(e, 64)
            if is_value:
                h, c, o = t // 8, (t % 8) // 2, t % 2
                g, w, j = r // 8, 2 * group + (r % 8) // 4, r % 4
                word = ((plane * 2 + h) * 8 + g) * 4 * (W // 32) + c * (W // 32) + w
                bit = 16 * o + 4 * j
            else:
                c, w, i = r // 16, 2 * group + (r % 16) // 8, r % 8
                word = ((plane * 16 + t) * 4 + c) * (W // 32) + w
                bit = 4 * i
            byte[t, d], shift[t, d] = 4 * word + bit // 8, bit % 8
    return byte, shift


def quantise(x):
    """[..., D] float64 values of the row type -> codes [..., D], s and m [..., D / 64] (float16)."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    f32 = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    f16 = lambda v: v.astype(np.float16).astype(np.float64)  # noqa: E731
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
        m = f16(lo)
        s = f16(f32(f32(hi - lo) * np.float64(np.float32(1 / 15))))
        r = np.where(s > 0, f32(1 / np.where(s > 0, s, 1)), 0.0)
        codes = np.rint(f32(f32(g - m) * r))
        codes = np.clip(np.nan_to_num(codes, nan=0.0), 0, 15)
    return codes.astype(np.uint8).reshape(x.shape), s[..., 0].astype(np.float16), m[..., 0].astype(np.float16)


def _tile_of(slot, P):
    return slot // P, (slot % P) // 16, slot % 16


def append(pages, k, v, slots, P):
    """``pages`` uint8 [num_pages, H, P / 16, tile], in place; k, v [n, H, D] float64."""
    H, D = k.shape[1], k.shape[2]
    half = tile_bytes(D) // 2
    for which, x in enumerate((k, v)):
        byte, shift = code_place(D, which)
        codes, s, m = quantise(x)
        for i, slot in enumerate(slots):
            if not 0 <= slot < pages.shape[0] * P:
                continue
            pg, tile, t = _tile_of(int(slot), P)
            for h in range(H):
                part = pages[pg, h, tile, which * half:(which + 1) * half]
                low = shift[t] == 0
                part[byte[t][low]] = codes[i, h][low] | codes[i, h][~low] << 4
                pair = np.stack([s[i, h], m[i, h]], -1).reshape(-1).view(np.uint8)
                n = len(pair)
                part[8 * D + t * n:8 * D + (t + 1) * n] = pair


def read(pages, slots, P, D):
    """(k, v) [n, H, D] float64: what the cache stands for."""
    H, half, got = pages.shape[1], tile_bytes(D) // 2, []
    slots = np.asarray(slots)
    pg, tile, t = _tile_of(slots, P)
    for which in (0, 1):
        byte, shift = code_place(D, which)
        part = pages[pg, :, tile, which * half:(which + 1) * half]  # [n, H, half]
        codes = np.take_along_axis(part, np.broadcast_to(byte[t][:, None], (len(slots), H, D)), 2)
        codes = (codes >> shift[t][:, None].astype(np.uint8)) & 15
        pairs = np.ascontiguousarray(part[..., 8 * D:]).view(np.float16).reshape(len(slots), H, 16, D // 64, 2)
        pairs = pairs[np.arange(len(slots)), :, t].astype(np.float64)
        got.append(codes * np.repeat(pairs[..., 0], 64, -1) + np.repeat(pairs[..., 1], 64, -1))
    return got


# --------------------------------------------------------------- attention --

def attend(q, pages, P, table, row_start, seq_len, scale, window, max_q_len=1 << 30):
    """out [n, Q, D] float64, lse [n, Q], the largest |v| that a row sees [n, Q], error bits."""
    n, Q, D = q.shape
    H, max_pages, err = pages.shape[1], table.shape[1], 0
    out, lse, big = np.zeros((n, Q, D)), np.full((n, Q), -np.inf), np.zeros((n, Q))
    for b in range(len(seq_len)):
        a, e, seq = int(row_start[b]), int(row_start[b + 1]), int(seq_len[b])
        if e - a > max_q_len:
            err |= ERR_LENGTH
            continue
        if e == a:
            continue
        if seq > max_pages * P or seq < 0:
            err |= ERR_LENGTH
        t = np.arange(max(0, min(seq, max_pages * P)))
        if window:
            t = t[t > seq - (e - a) - window]
        page = table[b, t // P]
        held = (page >= 0) & (page < pages.shape[0])
        if not held.all():
            err |= ERR_PAGE
        t, page = t[held], page[held].astype(np.int64)
        k, v = read(pages, page * P + t % P, P, D)
        for i in range(a, e):
            pos = seq - e + i
            seen = t <= pos
            if window:
                seen &= t > pos - window
            if not seen.any():
                continue
            for h in range(H):
                rows = slice(h * (Q // H), (h + 1) * (Q // H))
                s = q[i, rows] @ k[seen, h].T * scale
                top = s.max(-1, keepdims=True)
                p = np.exp(s - top)
                total = p.sum(-1, keepdims=True)
                out[i, rows] = p @ v[seen, h] / total
                lse[i, rows] = (top + np.log(total))[:, 0]
                big[i, rows] = np.abs(v[seen, h]).max()
    return out, lse, big, err
