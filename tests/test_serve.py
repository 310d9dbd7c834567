"""The serving step around the delta: the batch plan, the 4-bit key/value cache and attention over
it, against plain 64-bit numpy forms.

Tolerances.  Whole numbers, stored bytes and rows read back are equal.  Attention: the output's own
rounding, half a unit of the row type (2^-9 |out| in bf16, 2^-12 |out| in f16 to first order, doubled),
and 2^-9 of the largest |v| that the row sees, which covers weights rounded to 16 bits (2^-11 relative
in the numerator), keys and values rounded to f16 where tiles are expanded (2^-12 each, averaged over
dims and tokens) and float32 sums.  The logarithm of the denominator: 2^-9 + 2^-20 |lse|.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from tests import serve_ref as ref

NP_TYPE = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


# --------------------------------------------------------------------- CPU --

@pytest.mark.parametrize("D", [64, 128, 256])
def test_code_places_fill_a_tile_once(D):
    for which in (0, 1):
        byte, shift = ref.code_place(D, which)
        places = byte * 2 + shift // 4
        assert sorted(places.reshape(-1).tolist()) == list(range(16 * D))
        # the pairs of codes that one AND makes an operand: a word's halves hold codes 16 bits apart
        assert set(np.unique(shift)) == {0, 4}


@pytest.mark.parametrize("D", [64, 256])
def test_stored_values_are_within_half_a_step(D):
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 20, 2, D))
    k, v = k.astype(np.float16).astype(float), v.astype(np.float16).astype(float)
    pages = np.zeros((2, 2, 1, ref.tile_bytes(D)), np.uint8)
    slots = rng.permutation(32)[:20]
    ref.append(pages, k, v, slots, 16)
    for x, y in zip((k, v), ref.read(pages, slots, 16, D)):
        g = x.reshape(20, 2, -1, 64)
        step = (g.max(-1) - g.min(-1)) / 15
        # half a step, and the f16 roundings of the step (15 of them) and of the least value
        bound = 0.5 * step + 16 * step * 2.0 ** -11 + np.abs(g).max(-1) * 2.0 ** -11
        assert (np.abs(x - y).reshape(g.shape) <= bound[..., None]).all()


def test_refusals_on_the_host():
    import lora_delta_gb300 as ld
    from lora_delta_gb300.build import build
    build()
    L = ld.lib()
    f = ctypes.c_void_p(0x10000)  # never dereferenced: the checks come first
    ok, arg, shape, align, ws, unsup = 0, 1, 2, 3, 5, 6

    def plan(B=2, n=8, P=16, ld_table=4, max_pages=4, ctx=f, free=f, count=f, left=f, rows=f):
        return L.lora_batch_plan(ctx, f, None, B, n, P, f, ld_table, max_pages, free, count, left,
                                 f, f, rows, f, f, f, None, None)

    assert plan(ctx=None) == arg and plan(rows=None) == arg and plan(B=-1) == arg
    assert plan(count=None) == arg and plan(left=None) == arg and plan(free=None) == arg
    assert plan(P=24) == unsup and plan(P=0) == arg and plan(P=2048) == unsup
    assert plan(B=4097) == unsup and plan(max_pages=1 << 28, ld_table=1 << 28) == unsup
    assert plan(ld_table=3) == shape
    assert plan(rows=ctypes.c_void_p(0x10004)) == align
    assert L.lora_pages_release(f, f, 2, 16, f, 4, 4, None, 8, f, None, None) == arg
    assert L.lora_pages_release(f, f, 2, 16, f, 3, 4, f, 8, f, None, None) == shape
    assert L.lora_pages_release(None, None, 0, 16, None, 0, 4, None, 8, None, None, None) == ok

    assert ld.lora_kv4_page_bytes(16, 1, 128) == 2304 and ld.lora_kv4_page_bytes(64, 2, 64) == 9216
    assert ld.lora_kv4_page_bytes(16, 1, 96) == 0 and ld.lora_kv4_page_bytes(20, 1, 64) == 0

    for call in (L.lora_kv4_append, L.lora_kv4_read):
        def rows(pages=f, N=4, P=16, H=2, D=64, t=0, k=f, ld_k=128, ld_v=128, slots=f, n=3):
            return call(pages, N, P, H, D, t, k, ld_k, f, ld_v, slots, n, None, None)

        assert rows(pages=None) == arg and rows(k=None) == arg and rows(slots=None) == arg
        assert rows(N=0) == arg and rows(t=2) == arg and rows(n=-1) == arg and rows(n=0) == ok
        assert rows(D=96) == unsup and rows(P=40) == unsup and rows(H=1025) == unsup
        assert rows(ld_k=120) == shape and rows(ld_v=132) == align
        assert rows(pages=ctypes.c_void_p(0x10008)) == align
        assert rows(k=ctypes.c_void_p(0x10002)) == align

    def attend(out=f, ld_out=256, ld_q=256, n=3, Q=4, H=2, D=64, table=f, ld_table=4, max_pages=4,
               B=2, mq=2, window=0, work=f, wsb=1 << 30, P=16):
        return L.lora_kv4_attention(out, ld_out, f, ld_q, n, Q, f, 4, P, H, D, 0, table, ld_table,
                                    max_pages, f, f, B, mq, 1.0, window, None, work, wsb, None, None)

    assert attend(out=None) == arg and attend(table=None) == arg and attend(window=-1) == arg
    assert attend(n=-1) == arg and attend(n=0) == ok and attend(Q=0) == arg and attend(mq=-1) == arg
    assert attend(Q=3) == shape and attend(ld_out=248) == shape and attend(ld_table=3) == shape
    assert attend(ld_q=260) == align and attend(D=80) == unsup and attend(B=4097) == unsup
    assert attend(max_pages=1 << 28, ld_table=1 << 28) == unsup
    assert attend(work=None) == ws and attend(wsb=16) == ws


# --------------------------------------------------------------------- GPU --

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def ld():
    import __graft_entry__
    __graft_entry__.build()
    import lora_delta_gb300
    assert torch.cuda.is_available()
    return lora_delta_gb300


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).cuda()


def host(t):
    return t.cpu().numpy()


def check_plan(ld, ctx, new, P, n_rows, max_pages, free, count, req_slot=None, in_place=False, holes=()):
    B = len(ctx)
    table = np.full((B, max_pages + 2), -7)
    for b in range(B):
        held = -(-min(max(int(ctx[b]), 0), max_pages * P) // P)
        table[b, :held] = 100000 + 1000 * b + np.arange(held)
    for b, p in holes:
        table[b, p] = -1
    want = ref.plan(ctx, new, req_slot, n_rows, P, table, max_pages, free, count)
    d_table, err = dev(table), ld.new_error_word()
    p = ld.BatchPlan(B, n_rows, P)
    for t in (p.row_start, p.seq_len, p.row_req, p.position, p.seq_slot, p.slot_map):
        t.fill_(-99)
    kw = {}
    if free is not None:
        kw = {"free_pages": dev(free), "free_count": dev([count]), "free_left": None if in_place else dev([-5])}
    ld.lora_batch_plan(p, dev(ctx), dev(new), d_table[:, :max_pages], err=err,
                       req_slot=None if req_slot is None else dev(req_slot), **kw)
    assert ld.lora_get_error(err) == want["err"]
    for name in ("row_start", "seq_len", "row_req", "position", "seq_slot", "slot_map"):
        assert np.array_equal(host(getattr(p, name)), want[name]), name
    assert np.array_equal(host(d_table), want["table"])
    if free is not None:
        assert int((kw["free_left"] if not in_place else kw["free_count"])[0]) == want["left"]
    return want["err"]


@gpu
@pytest.mark.parametrize("seed,B,P,top,spare", [(0, 1, 16, 1, 0), (1, 7, 16, 40, 3), (2, 64, 16, 1, 0),
                                                (3, 513, 64, 9, 130), (4, 33, 128, 700, 1),
                                                (5, 4096, 32, 3, 0), (6, 2, 1024, 20000, 5)])
def test_plan_matches_the_loop(ld, seed, B, P, top, spare):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, 300, B), rng.integers(0, top + 1, B)
    ctx[rng.random(B) < 0.2] = 0
    max_pages = int(-(-(ctx + new).max() // P)) + 1
    need = int((-(-(ctx + new) // P) - -(-ctx // P)).sum())
    free = rng.permutation(need + 9)
    slots = rng.integers(-1, 16, B)
    n = int(new.sum()) + spare
    assert check_plan(ld, ctx, new, P, n, max_pages, free, need + 9, slots) == 0
    assert check_plan(ld, ctx, new, P, n, max_pages, free, need, None, in_place=True) == 0
    # every page in the tables already
    last = np.minimum(new, np.maximum((ctx + new) % P - 1, 0))
    assert check_plan(ld, ctx + new - last, last, P, n + 1, max_pages, None, None) == 0


@gpu
def test_plan_of_nothing(ld):
    assert check_plan(ld, np.zeros(0, int), np.zeros(0, int), 16, 5, 2, np.arange(3), 3) == 0
    assert check_plan(ld, np.zeros(3, int), np.zeros(3, int), 16, 0, 2, np.arange(3), 3) == 0
    assert check_plan(ld, np.full(3, 31), np.zeros(3, int), 16, 9, 2, np.arange(3), 3) == 0


@gpu
def test_plan_cuts_and_reports_what_does_not_fit(ld):
    free = np.arange(50, 90)
    # the free pages run out in the middle of a request
    assert check_plan(ld, [5, 0, 17], [40, 60, 30], 16, 130, 8, free[:4], 4) == ref.ERR_PAGE
    assert check_plan(ld, [5, 0, 17], [40, 60, 30], 16, 130, 8, free, 0, in_place=True) == ref.ERR_PAGE
    # a hole in a page that should be held
    assert check_plan(ld, [5, 20], [4, 4], 16, 8, 8, free, 40, holes=[(1, 1)]) == ref.ERR_PAGE
    # more rows than the batch has, cut in a request, at its end and before it
    for n in (100, 99, 41, 40, 39, 1, 0):
        assert check_plan(ld, [5, 0, 17], [40, 60, 30], 16, n, 8, free, 40) == ref.ERR_LENGTH
    # lengths past the table, negative ones, and ones near 2^31
    assert check_plan(ld, [120, 200, 10], [20, 4, 3], 16, 40, 8, free, 40) == ref.ERR_LENGTH
    assert check_plan(ld, [-3, 4, 9], [5, -2, 7], 16, 40, 8, free, 40) == ref.ERR_LENGTH
    big = 2 ** 31 - 1
    assert check_plan(ld, [big, 3, 0], [big, big, big], 16, 4000, 8, free, 40) & ref.ERR_LENGTH


@gpu
@pytest.mark.parametrize("seed,B,P", [(0, 5, 16), (1, 700, 32), (2, 64, 64)])
def test_release_returns_the_pages(ld, seed, B, P):
    rng = np.random.default_rng(seed)
    max_pages = 70
    seq = rng.integers(0, max_pages * P + 1, B)
    table = rng.permutation(B * max_pages).reshape(B, max_pages)
    table[rng.random(table.shape) < 0.05] = -1
    done = rng.random(B) < 0.5
    for cap, lens in ((B * max_pages + 20, seq), (B * max_pages // 6, seq), (B * max_pages, seq + rng.integers(-9, 900, B))):
        free, err = np.full(cap, -3), ld.new_error_word()
        want = ref.release(done, lens, P, table, max_pages, free, 11)
        d = dev(table), dev(free), dev([11])
        ld.lora_pages_release(dev(done), dev(lens), d[0], P, d[1], d[2], err=err)
        assert ld.lora_get_error(err) == want[3]
        assert np.array_equal(host(d[0]), want[0]) and np.array_equal(host(d[1]), want[1])
        assert int(d[2][0]) == want[2]


def to_rows(x, dtype):
    return torch.from_numpy(x).to(dtype).cuda()


def random_pages(rng, shape):
    return rng.integers(0, 256, shape, dtype=np.uint8)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,H,P,n", [(128, 8, 16, 1), (128, 2, 64, 77), (64, 3, 32, 50), (256, 1, 16, 33),
                                     (64, 1, 128, 300), (128, 5, 1024, 18)])
def test_append_and_read_bit_for_bit(ld, D, H, P, n, dtype):
    rng = np.random.default_rng(D + n)
    num_pages = -(-n // P) + 2
    slots = rng.permutation(num_pages * P)[:n].astype(np.int64)
    if n > 40:  # a run of adjacent slots, as a prompt's, beginning and ending inside a tile
        slots[:37] = np.arange(5, 42)
        slots[37:] = 42 + rng.permutation(num_pages * P - 42)[:n - 37]
        slots[n // 2] = -1
    k, v = rng.standard_normal((2, n, H, D)) * np.exp(rng.standard_normal((2, n, H, 1)) * 3)
    k[0, 0, :64] = 1.5           # a constant group
    v[0, 0, :64] = 0.0
    v[n - 1, H - 1, 64 * (D // 64 - 1):] += 1000.0  # far from zero
    pages = random_pages(rng, (num_pages, H, P // 16, ref.tile_bytes(D)))
    # rows that lie apart, as slices of a fused projection
    fused = torch.zeros(n, 3 * H * D + 8, dtype=dtype, device="cuda")
    fused[:, H * D:2 * H * D] = to_rows(k, dtype).view(n, -1)
    fused[:, 2 * H * D:3 * H * D] = to_rows(v, dtype).view(n, -1)
    dk, dv = (fused[:, a * H * D:(a + 1) * H * D].unflatten(1, (H, D)) for a in (1, 2))
    cache = ld.Kv4Cache(dev(pages, np.uint8), P, D, dtype)
    err = ld.new_error_word()
    ld.lora_kv4_append(cache, dk, dv, dev(slots, np.int64), err=err)
    assert ld.lora_get_error(err) == 0
    ref.append(pages, dk.double().cpu().numpy(), dv.double().cpu().numpy(), slots, P)
    assert np.array_equal(host(cache.pages), pages)
    gk, gv = torch.full((2, n, H, D), 7.0, dtype=dtype, device="cuda")
    ld.lora_kv4_read(cache, gk, gv, dev(slots, np.int64), err=err)
    assert ld.lora_get_error(err) == 0
    for got, want in zip((gk, gv), ref.read(pages, np.maximum(slots, 0), P, D)):
        want[slots < 0] = 0.0
        assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(dtype))


@gpu
def test_append_and_read_outside_the_cache(ld):
    D, H, P, num_pages = 64, 2, 16, 3
    rng = np.random.default_rng(1)
    pages = random_pages(rng, (num_pages, H, 1, ref.tile_bytes(D)))
    cache = ld.Kv4Cache(dev(pages, np.uint8), P, D)
    k = torch.randn(5, H, D, device="cuda").bfloat16()
    slots = np.array([-1, 48, 1 << 40, -(1 << 50), 49])
    err = ld.new_error_word()
    ld.lora_kv4_append(cache, k, k, dev(slots, np.int64), err=err)
    assert ld.lora_get_error(err) == ref.ERR_PAGE
    assert np.array_equal(host(cache.pages), pages)
    out = torch.full((2, 5, H, D), 3.0, device="cuda").bfloat16()
    ld.lora_kv4_read(cache, out[0], out[1], dev(slots, np.int64), err=err)
    assert ld.lora_get_error(err) == ref.ERR_PAGE and not out.any()


@gpu
def test_groups_with_infinities_and_nans_read_as_nan(ld):
    D, H = 128, 1
    x = torch.randn(16, H, D, device="cuda")
    x[0, 0, 3], x[1, 0, 70], x[2, 0, 127] = float("nan"), float("inf"), -float("inf")
    cache = ld.Kv4Cache.empty(1, 16, H, D, torch.float16)
    slots = torch.arange(16, device="cuda")
    k, v = torch.empty(2, 16, H, D, device="cuda", dtype=torch.float16)
    ld.lora_kv4_append(cache, x.half(), x.half(), slots)
    ld.lora_kv4_read(cache, k, v, slots)
    for got in (k, v):
        bad = torch.isnan(got).view(16, 2, 64)
        want = torch.zeros(16, 2, dtype=torch.bool, device="cuda")
        want[0, 0] = want[1, 1] = want[2, 1] = True
        assert torch.equal(bad.all(-1), want) and torch.equal(bad.any(-1), want)


def attention_case(rng, lens, D, H, group, P, dtype, spare_rows=0, num_pages=None, k_std=1.0):
    """Random pages of which the requests' tokens are stored rows; the rest is stale bytes."""
    seq = np.array([c + n for c, n in lens])
    need = -(-seq // P)
    num_pages = num_pages or int(need.sum()) + 3
    order = rng.permutation(num_pages)
    table = np.full((len(lens), int(need.max(initial=0)) + 2), -1)
    pages = random_pages(rng, (num_pages, H, P // 16, ref.tile_bytes(D)))
    at = 0
    for b, s in enumerate(seq):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        t = np.arange(s)
        k, v = rng.standard_normal((2, s, H, D))
        k = k * k_std + rng.standard_normal((H, D)) * (rng.random((H, D)) < 0.05) * 4
        k, v = (x.astype(np.float16).astype(float) for x in (k, v))
        ref.append(pages, k, v, table[b, t // P].astype(np.int64) * P + t % P, P)
    start = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(int)
    n = int(start[-1]) + spare_rows
    q = to_rows(rng.standard_normal((n, H * group, D)), dtype)
    return {"q": q, "pages": pages, "table": table, "start": start, "seq": seq, "P": P, "D": D,
            "dtype": dtype, "max_q": max([x for _, x in lens], default=0)}


def run_attention(ld, c, window=0, scale=None, max_q=None, **kw):
    cache = kw.pop("cache", None) or ld.Kv4Cache(dev(c["pages"], np.uint8), c["P"], c["D"], c["dtype"])
    out = torch.full_like(c["q"], 9.0)
    lse = torch.full(c["q"].shape[:2], 9.0, device="cuda")
    err = ld.new_error_word()
    ld.lora_kv4_attention(out, c["q"], cache, dev(c["table"]), dev(c["start"]), dev(c["seq"]),
                          c["max_q"] if max_q is None else max_q, scale=scale, window=window, lse=lse,
                          err=err, **kw)
    return out, lse, ld.lora_get_error(err)


def check_attention(ld, c, window=0, scale=None, max_q=None, want_err=0, **kw):
    out, lse, err = run_attention(ld, c, window, scale, max_q, **kw)
    want, want_lse, big, ref_err = ref.attend(
        c["q"].double().cpu().numpy(), c["pages"], c["P"], c["table"], c["start"], c["seq"],
        c["D"] ** -0.5 if scale is None else scale, window, 1 << 30 if max_q is None else max_q)
    assert err == ref_err == want_err
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bound = NP_TYPE[c["dtype"]] * np.abs(want) + 2.0 ** -9 * big[..., None]
    off = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (off <= bound).all(), (np.argwhere(off > bound)[:5], float((off - bound).max()))
    none = np.isneginf(want_lse)
    assert np.array_equal(none, np.isneginf(got_lse))
    assert (np.abs(got_lse - want_lse)[~none] <= 2.0 ** -9 + 2.0 ** -20 * np.abs(want_lse[~none])).all()
    return out


DECODE = [(0, 1), (15, 1), (16, 1), (17, 1), (300, 1), (1, 1), (95, 1), (1000, 1)]


@gpu
@pytest.mark.parametrize("D,H,group,P,dtype", [
    (128, 2, 4, 16, torch.bfloat16), (128, 1, 1, 32, torch.float16), (64, 3, 5, 64, torch.bfloat16),
    (64, 1, 8, 16, torch.float16), (256, 2, 2, 16, torch.bfloat16), (256, 1, 16, 128, torch.float16),
    (128, 1, 16, 16, torch.bfloat16), (128, 2, 9, 1024, torch.bfloat16), (64, 1, 71, 48, torch.bfloat16),
    (128, 5, 1, 16, torch.bfloat16)])
@pytest.mark.parametrize("window", [0, 33])
def test_attention_of_single_tokens(ld, D, H, group, P, dtype, window):
    rng = np.random.default_rng(D * H + group)
    check_attention(ld, attention_case(rng, DECODE, D, H, group, P, dtype), window)


SEVERAL = [(0, 3), (40, 2), (0, 0), (7, 5), (500, 8), (33, 1), (3, 0), (250, 7)]
CHUNKS = [(0, 70), (100, 33), (0, 0), (17, 129), (300, 1), (5, 12), (0, 1), (40, 200)]


@gpu
@pytest.mark.parametrize("D,H,group,P,dtype", [
    (128, 2, 4, 16, torch.bfloat16), (64, 2, 1, 32, torch.float16), (256, 1, 3, 16, torch.bfloat16),
    (128, 1, 8, 64, torch.float16), (64, 1, 20, 16, torch.bfloat16), (128, 1, 16, 16, torch.bfloat16),
    (256, 1, 8, 32, torch.float16), (128, 1, 5, 48, torch.bfloat16)])
@pytest.mark.parametrize("lens", [SEVERAL, CHUNKS], ids=["several", "chunks"])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_attention_of_several_tokens(ld, D, H, group, P, dtype, lens, window):
    rng = np.random.default_rng(D * H + group)
    check_attention(ld, attention_case(rng, lens, D, H, group, P, dtype, spare_rows=3), window)


@gpu
@pytest.mark.parametrize("lens,H,group,window", [
    ([(20000, 1)], 1, 4, 0), ([(5000, 1), (12, 1), (7000, 1)], 2, 8, 0), ([(9000, 1)], 1, 1, 5000),
    ([(6000, 4), (100, 4)], 1, 4, 0), ([(3000, 300)], 1, 2, 0), ([(4000, 150), (50, 3)], 1, 4, 1000),
    ([(0, 1500)], 1, 1, 0)])
def test_attention_over_long_contexts(ld, lens, H, group, window):
    rng = np.random.default_rng(len(lens) + H)
    check_attention(ld, attention_case(rng, lens, 128, H, group, 32, torch.bfloat16), window)


@gpu
@pytest.mark.parametrize("D,H,group,dtype,lens,window", [
    (64, 2, 4, torch.float16, [(5000, 40)], 0), (256, 1, 3, torch.bfloat16, [(3000, 90), (700, 1)], 0),
    (128, 1, 1, torch.bfloat16, [(2000, 300), (0, 1100), (1500, 33)], 900)])
def test_attention_of_few_rows_over_long_contexts(ld, D, H, group, dtype, lens, window):
    """Items that share their tokens out; twice with one workspace, and after a call that gave up."""
    c = attention_case(np.random.default_rng(D), lens, D, H, group, 32, dtype)
    first = check_attention(ld, c, window)
    prev = ld.lora_set_wait_limit_ns(0)
    try:
        run_attention(ld, c, window)
    finally:
        ld.lora_set_wait_limit_ns(prev)
    assert torch.equal(first, check_attention(ld, c, window))


@gpu
def test_attention_sums_of_long_contexts_do_not_drift(ld):
    """Requests of 8192 tokens, enough of them that a warp sums whole ones.  Three roundings to
    f16 (a weight, its product with a scale, the result), each of at most 2^-11 / sqrt(3) on the
    average, make 2^-11 of the result's norm."""
    rng = np.random.default_rng(21)
    c, B, part = attention_case(rng, [(8191, 1)], 64, 1, 1, 64, torch.float16), 4096, 64
    c["table"] = np.repeat(c["table"], B, 0)
    c["start"], c["seq"] = np.arange(B + 1), np.repeat(c["seq"], B)
    c["q"] = to_rows(rng.standard_normal((B, 1, 64)), torch.float16)
    out, _, err = run_attention(ld, c)
    assert err == 0
    want = ref.attend(c["q"][:part].double().cpu().numpy(), c["pages"], 64, c["table"][:part], c["start"][:part + 1],
                      c["seq"][:part], 64 ** -0.5, 0)[0]
    off = out[:part].double().cpu().numpy() - want
    assert np.sqrt((off ** 2).sum() / (want ** 2).sum()) <= 2.0 ** -11


@gpu
@pytest.mark.parametrize("B", [300, 4096])
def test_attention_of_many_requests(ld, B):
    rng = np.random.default_rng(B)
    lens = [(int(c), int(n)) for c, n in zip(rng.integers(0, 40, B), rng.integers(0, 3, B))]
    check_attention(ld, attention_case(rng, lens, 64, 1, 2, 16, torch.bfloat16))


@gpu
@pytest.mark.parametrize("std", [0.0, 30.0])
@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_attention_with_flat_and_sharp_weights(ld, std, lens):
    """Scores all alike, and scores of which one takes everything; values far from zero."""
    rng = np.random.default_rng(7)
    c = attention_case(rng, lens, 128, 1, 4, 16, torch.bfloat16, k_std=std)
    check_attention(ld, c, scale=None if std else 0.0)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("size", [2.0 ** -20, 1.0, 2.0 ** 12])
def test_attention_scales_of_queries_and_values(ld, dtype, size):
    """Queries and values far from 1, against the scale that brings the scores back."""
    rng = np.random.default_rng(9)
    for lens in (DECODE, CHUNKS):
        c = attention_case(rng, lens, 64, 1, 4, 16, dtype)
        q = c["q"].float() * size if dtype == torch.bfloat16 else c["q"].float() * max(size, 2.0 ** -8)
        c["q"] = q.to(dtype)
        scale = 64 ** -0.5 / (size if dtype == torch.bfloat16 else max(size, 2.0 ** -8))
        half = ref.tile_bytes(64) // 2
        pairs = c["pages"][..., half + 8 * 64:].view(np.float16)  # values' steps and least values
        pairs *= np.float16(min(max(size, 2.0 ** -6), 2.0 ** 8))
        pairs[~np.isfinite(pairs)] = 0
        check_attention(ld, c, scale=scale)


@gpu
def test_attention_does_not_see_what_lies_behind_the_lengths(ld):
    """Stale tokens, other pages and the rest of the last tile hold NaNs and infinities."""
    rng = np.random.default_rng(11)
    for lens in (DECODE, SEVERAL, CHUNKS):
        c = attention_case(rng, lens, 128, 1, 4, 32, torch.bfloat16)
        a = check_attention(ld, c, 20)
        seen = np.zeros(c["pages"].shape[0] * 32, bool)
        for b, s in enumerate(c["seq"]):
            t = np.arange(s)
            seen[c["table"][b, t // 32].astype(int) * 32 + t % 32] = True
        seen = seen.reshape(-1, 1, 2, 16)
        for at in (8 * 128, ref.tile_bytes(128) // 2 + 8 * 128):
            pairs = c["pages"][..., at:at + 128].view(np.float16).reshape(*c["pages"].shape[:3], 16, 4)
            for fill in (np.nan, np.inf, -np.inf):
                pairs = np.where(seen[..., None], pairs, np.float16(fill))
                c["pages"][..., at:at + 128] = pairs.reshape(*c["pages"].shape[:3], 64).view(np.uint8)
                b = check_attention(ld, c, 20)
                assert torch.equal(a, b)


@gpu
def test_attention_with_missing_pages_and_wrong_lengths(ld):
    rng = np.random.default_rng(13)
    for lens in (DECODE, CHUNKS):
        c = attention_case(rng, lens, 64, 2, 4, 16, torch.bfloat16)
        c["table"][4, 3], c["table"][4, 5], c["table"][0, 0] = -1, c["pages"].shape[0], 1 << 30
        check_attention(ld, c, want_err=ref.ERR_PAGE)
        check_attention(ld, c, window=30, want_err=ref.ERR_PAGE)
    # a length past the table
    c = attention_case(rng, [(40, 1), (20, 1)], 64, 1, 4, 16, torch.bfloat16)
    c["table"] = c["table"][:, :2]
    check_attention(ld, c, want_err=ref.ERR_LENGTH)
    # more rows than the host was told
    for lens, most in ((SEVERAL, 7), (CHUNKS, 128), (CHUNKS, 100)):
        c = attention_case(rng, lens, 64, 1, 4, 16, torch.bfloat16)
        check_attention(ld, c, max_q=most, want_err=ref.ERR_LENGTH)


@gpu
def test_attention_of_no_requests_and_no_rows(ld):
    rng = np.random.default_rng(15)
    c = attention_case(rng, [(0, 0), (9, 0)], 64, 1, 4, 16, torch.bfloat16, spare_rows=5)
    out, lse, err = run_attention(ld, c)
    assert err == 0 and not out.any() and torch.isneginf(lse).all()
    c["table"], c["start"], c["seq"] = c["table"][:0], c["start"][:1], c["seq"][:0]
    out, lse, err = run_attention(ld, c)
    assert err == 0 and not out.any() and torch.isneginf(lse).all()
    c["q"] = c["q"][:0]
    assert run_attention(ld, c)[2] == 0


@gpu
@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_attention_of_sliced_rows_keeps_the_rest(ld, lens):
    rng = np.random.default_rng(17)
    c = attention_case(rng, lens, 128, 2, 2, 16, torch.bfloat16)
    want = run_attention(ld, c)[0]
    n = c["q"].shape[0]
    wide = torch.full((n, 4 * 128 + 64), 5.0, device="cuda").bfloat16()
    fused = torch.randn(n, 6 * 128 + 8, device="cuda").bfloat16()
    fused[:, 128:5 * 128] = c["q"].reshape(n, -1)
    cache = ld.Kv4Cache(dev(c["pages"], np.uint8), 16, 128)
    ld.lora_kv4_attention(wide[:, 32:32 + 512].unflatten(1, (4, 128)), fused[:, 128:640].unflatten(1, (4, 128)),
                          cache, dev(c["table"]), dev(c["start"]), dev(c["seq"]), c["max_q"])
    assert torch.equal(wide[:, 32:544].reshape(n, 4, 128), want)
    assert (wide[:, :32] == 5).all() and (wide[:, 544:] == 5).all()


@gpu
def test_attention_offsets_past_32_bits(ld):
    """A cache of more than 4 GiB, its high pages in use."""
    D, H, P = 128, 2, 16
    num_pages = (5 << 30) // ld.lora_kv4_page_bytes(P, H, D)
    rng = np.random.default_rng(19)
    for lens in ([(100, 1), (37, 1)], [(60, 90)]):
        c = attention_case(rng, lens, D, H, 4, P, torch.bfloat16)
        big = torch.zeros(num_pages, H, 1, ref.tile_bytes(D), dtype=torch.uint8, device="cuda")
        small = len(c["pages"])
        big[-small:] = dev(c["pages"], np.uint8)
        want = run_attention(ld, c)[0]
        c["table"] = np.where(c["table"] >= 0, c["table"] + num_pages - small, -1)
        cache = ld.Kv4Cache(big, P, D)
        assert torch.equal(run_attention(ld, c, cache=cache)[0], want)
        # and the same rows stored and read there
        slots = dev(num_pages * P - 1 - np.arange(50), np.int64)
        k, v = torch.randn(2, 50, H, D, device="cuda").bfloat16()
        got = torch.empty(2, 50, H, D, device="cuda", dtype=torch.bfloat16)
        ld.lora_kv4_append(cache, k, v, slots)
        ld.lora_kv4_read(cache, got[0], got[1], slots)
        assert (got[0] - k).abs().max() < 0.5 and (got[1] - v).abs().max() < 0.5


@gpu
@pytest.mark.parametrize("lens", [DECODE, [(3000, 1), (10, 1)], CHUNKS], ids=["decode", "split", "chunks"])
def test_attention_repeats_bit_for_bit_on_any_stream_and_in_a_graph(ld, lens):
    rng = np.random.default_rng(21)
    c = attention_case(rng, lens, 128, 2, 4, 16, torch.bfloat16)
    want = run_attention(ld, c)[0]
    for _ in range(3):
        assert torch.equal(run_attention(ld, c)[0], want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(run_attention(ld, c)[0], want)
    cache = ld.Kv4Cache(dev(c["pages"], np.uint8), 16, 128)
    args = dev(c["table"]), dev(c["start"]), dev(c["seq"]), c["max_q"]
    q, out, ws = torch.zeros_like(c["q"]), torch.empty_like(c["q"]), ld.lora_kv4_attention_workspace()
    torch.cuda.synchronize()
    ld.lora_kv4_attention(out, c["q"], cache, *args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for workspace in (ws, None):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ld.lora_kv4_attention(out, q, cache, *args, workspace=workspace)
        for _ in range(3):
            q.copy_(c["q"])
            out.fill_(3.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


@gpu
def test_binding_refuses_wrong_tensors(ld):
    cache = ld.Kv4Cache.empty(4, 16, 2, 64)
    x = torch.zeros(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        ld.lora_kv4_append(cache, x.half(), x, slots)
    with pytest.raises(ValueError):
        ld.lora_kv4_append(cache, x, x, slots.int())
    with pytest.raises(ValueError):
        ld.lora_kv4_append(cache, x, x[:2], slots)
    with pytest.raises(ValueError):
        ld.lora_kv4_append(cache, x.transpose(1, 2).contiguous().transpose(1, 2), x, slots)
    with pytest.raises(ValueError):
        ld.Kv4Cache(cache.pages, 16, 128)
    with pytest.raises(ValueError):
        ld.Kv4Cache(cache.pages, 16, 64, torch.float32)
    with pytest.raises(ValueError):
        ld.Kv4Cache.empty(4, 16, 2, 80)
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    one = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 3, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ld.LoraError) as e:  # 3 query heads on 2 heads of the cache
        ld.lora_kv4_attention(torch.empty_like(q), q, cache, table, one, one[:1], 1)
    assert e.value.code == 2
    with pytest.raises(ValueError):
        ld.lora_kv4_attention(q.cpu(), q, cache, table, one, one[:1], 1)
    with pytest.raises(ValueError):
        ld.lora_kv4_attention(q, q, cache, table.long(), one, one[:1], 1)


@gpu
@pytest.mark.parametrize("lens", [DECODE, [(3000, 1), (10, 1)], CHUNKS], ids=["decode", "split", "chunks"])
def test_attention_that_gives_up_waiting_reports_it_and_leaves_all_usable(ld, lens):
    """With a wait limit of 0 a wait gives up at its first poll that finds its phase incomplete: the call
    sets the time-out bit (or no poll did, and the result is right), and the workspace and the device
    serve the next call as before."""
    rng = np.random.default_rng(23)
    c = attention_case(rng, lens, 128, 2, 4, 16, torch.bfloat16)
    ws = ld.lora_kv4_attention_workspace()
    want = run_attention(ld, c, workspace=ws)[0]
    prev = ld.lora_set_wait_limit_ns(0)
    try:
        out, _, err = run_attention(ld, c, workspace=ws)
    finally:
        ld.lora_set_wait_limit_ns(prev)
    assert err == 8 or (err == 0 and torch.equal(out, want))
    torch.cuda.synchronize()
    assert not ws[:int(ld.lib().lora_kv4_attention_zeroed_bytes())].any()
    for _ in range(2):
        out, _, err = run_attention(ld, c, workspace=ws)
        assert err == 0 and torch.equal(out, want)


@gpu
def test_example_steps_match_the_plain_forms(ld, oracle):
    """The example's steps: plan, projections with adapters, store and attention together."""
    from examples.serve_step import D, HIDDEN, KV_HEADS, PAGE, Q_HEADS, WIDTHS, Server
    slots = [0, 2, -1, 1, 1]
    server = Server(slots, max_tokens=128, num_pages=40)
    cache = server.cache
    cache.pages.zero_()
    pages = host(cache.pages)
    g = torch.Generator(device="cuda").manual_seed(5)
    A, Bm = [[t.double().cpu().numpy() for t in x] for x in (server.pool.A, server.pool.B)]
    scale = server.pool.scale_table.double().cpu().numpy()
    table, free, count, ctx = host(server.table), host(server.free), 40, np.zeros(5, int)
    for new in ([37, 5, 64, 1, 0], [1, 1, 1, 1, 1], [1, 3, 1, 0, 2]):
        n, new = sum(new) + 2, np.array(new)  # two padding rows
        x = torch.randn(n, HIDDEN, device="cuda", generator=g).bfloat16()
        out, plan, qkv = server.step(x, dev(new), int(new.max()))
        want = ref.plan(ctx, new, slots, n, PAGE, table, table.shape[1], free, count)
        assert want["err"] == 0
        table, count, ctx = want["table"], want["left"], want["seq_len"]
        for name in ("row_req", "position", "slot_map", "seq_slot", "seq_len", "row_start"):
            assert np.array_equal(host(getattr(plan, name)), want[name]), name
        assert np.array_equal(host(server.table), table) and int(server.free_count[0]) == count
        # the delta on the rows' adapters
        base = (x @ server.weight).double().cpu().numpy()
        xs, s = x.double().cpu().numpy(), want["seq_slot"]
        at = 0
        for j, w in enumerate(WIDTHS):
            for i in np.nonzero(s >= 0)[0]:
                base[i, at:at + w] += scale[s[i]] * (xs[i] @ A[j][s[i]].T) @ Bm[j][s[i]].T
            at += w
        got = qkv.double().cpu().numpy()
        assert (np.abs(got - base) <= 2.0 ** -7 * np.abs(base) + 2.0 ** -7).all()
        # what was stored, from the projections as they are
        k, v = (got[:, a:a + KV_HEADS * D].reshape(n, KV_HEADS, D) for a in (WIDTHS[0], WIDTHS[0] + WIDTHS[1]))
        ref.append(pages, k, v, want["slot_map"], PAGE)
        assert np.array_equal(host(cache.pages), pages)
        q = got[:, :WIDTHS[0]].reshape(n, Q_HEADS, D)
        exact, _, big, err = ref.attend(q, pages, PAGE, table, want["row_start"], want["seq_len"], D ** -0.5, 0)
        off = np.abs(out.double().cpu().numpy() - exact)
        assert err == 0 and (off <= 2.0 ** -8 * np.abs(exact) + 2.0 ** -9 * big[..., None]).all()
    server.release(dev([1, 0, 1, 0, 0]))
    freed = ref.release([1, 0, 1, 0, 0], ctx, PAGE, table, table.shape[1], free, count)
    assert np.array_equal(host(server.table), freed[0]) and int(server.free_count[0]) == freed[2]
    assert ld.lora_get_error(server.err) == 0
