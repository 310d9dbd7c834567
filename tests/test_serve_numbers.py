"""Attention over the 4-bit cache where numbers are large, not finite or badly spread, against plain
64-bit numpy forms.

Tolerance of an output: as in ``tests/test_serve.py``, two roundings of the row type and 2^-9 of the largest
|v| that the row sees; and what the float32 sum of a score can move.  A score is off by at most
e = 2^-20 scale sum_d |q_d k_d| (products of up to 22 bits, sums of at most 256 of them in float32, a few
roundings after them), so weights change by factors of at most exp(2 e), and where 1 - r is the weight of the
row's largest score (and of tokens with the same key), the result moves by at most
2 max|v| min(1, r (exp(2 e) - 1)) and the logarithm of the denominator by e.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import serve_ref as ref
from tests.test_serve import NP_TYPE, attention_case, dev, host, ld, run_attention  # noqa: F401

gpu = pytest.mark.gpu


def rows_of(c, b):
    """Of a request: its rows, the positions they stand at and what its pages hold."""
    a, e, seq = int(c["start"][b]), int(c["start"][b + 1]), int(c["seq"][b])
    t = np.arange(seq)
    page = c["table"][b, t // c["P"]].astype(np.int64)
    k, v = ref.read(c["pages"], page * c["P"] + t % c["P"], c["P"], c["D"])
    return a, e, seq - (e - a) + np.arange(e - a), k, v


def score_room(c, scale, window=0):
    """For each row and head [n, Q]: min(1, r (exp(2 e) - 1)), and e."""
    q = c["q"].double().cpu().numpy()
    room, off = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    for b in range(len(c["seq"])):
        a, e, pos, k, _ = rows_of(c, b)
        t = np.arange(len(k))
        for h in range(k.shape[1]):
            g = q.shape[1] // k.shape[1]
            rows = q[a:e, h * g:(h + 1) * g]
            s = np.einsum("ngd,td->ngt", rows, k[:, h]) * scale
            err = 2.0 ** -20 * abs(scale) * np.einsum("ngd,td->ngt", np.abs(rows), np.abs(k[:, h]))
            seen = (t <= pos[:, None]) & ((t > pos[:, None] - window) if window else True)
            s = np.where(seen[:, None], s, -np.inf)
            most = np.where(seen[:, None], err, 0).max(-1)
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            tied = s > top - 1e-10 * np.abs(top)  # (the same key, so the same error)
            rest = np.where(tied, 0, p).sum(-1) / p.sum(-1)
            with np.errstate(over="ignore", invalid="ignore"):
                grown = np.where(rest > 0, np.exp(np.log(np.maximum(rest, 1e-300)) + 2 * most) - rest, 0)
            room[a:e, h * g:(h + 1) * g], off[a:e, h * g:(h + 1) * g] = np.minimum(1, grown), most
    return room, off


def check_large(ld, c, scale, window=0):  # noqa: F811
    out, lse, err = run_attention(ld, c, window, scale)
    want, want_lse, big, _ = ref.attend(c["q"].double().cpu().numpy(), c["pages"], c["P"], c["table"], c["start"],
                                        c["seq"], scale, window)
    assert err == 0
    got, (room, off) = out.double().cpu().numpy(), score_room(c, scale, window)
    bound = NP_TYPE[c["dtype"]] * np.abs(want) + (2.0 ** -9 + 2 * room[..., None]) * big[..., None]
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) - bound).max())
    got_lse = lse.double().cpu().numpy()
    assert (np.abs(got_lse - want_lse) <= 2.0 ** -9 + off + 2.0 ** -20 * np.abs(want_lse)).all()
    return room


MANY_ROWS = [(0, 70), (100, 33), (17, 129), (40, 200)]
# (type, size of q, of k, scale): scores of 2^12 to 2^40
LARGE = [(torch.bfloat16, 1.0, 1.0, 2.0 ** 12), (torch.bfloat16, 2.0 ** 18, 1000.0, None),
         (torch.bfloat16, 1.0, 1.0, -2.0 ** 27), (torch.float16, 1.0, 1.0, 2.0 ** 29),
         (torch.float16, 3000.0, 3000.0, 2.0 ** 17), (torch.bfloat16, 2.0 ** -30, 1.0, 2.0 ** 56)]


def large_case(seed, lens, D, group, kind):
    dtype, q_size, k_size, scale = kind
    c = attention_case(np.random.default_rng(seed), lens, D, 1, group, 32, dtype, k_std=k_size)
    c["q"] = (c["q"].float() * q_size).to(dtype)
    return c, D ** -0.5 if scale is None else scale


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", LARGE)
def test_large_scores_of_many_rows(ld, D, kind):  # noqa: F811
    """The largest score takes all but a few rows whole, at any size."""
    c, scale = large_case(D, MANY_ROWS, D, 4, kind)
    room = check_large(ld, c, scale)
    assert (room < 2.0 ** -9).mean() > 0.75
    check_large(ld, c, scale, window=40)


@gpu
@pytest.mark.parametrize("kind", LARGE)
def test_large_scores_of_a_split_item(ld, kind):  # noqa: F811
    c, scale = large_case(3, [(5000, 40)], 128, 2, kind)
    check_large(ld, c, scale)


@gpu
@pytest.mark.parametrize("scale", [2.0 ** 5, 2.0 ** 15, 2.0 ** 30])
def test_equal_large_scores_of_many_rows_share_the_weight(ld, scale):  # noqa: F811
    """Tokens 16 to 31 have the keys of 0 to 15: a row that sees both gives them the same weights."""
    c = attention_case(np.random.default_rng(5), [(16, 64), (16, 200)], 128, 1, 4, 32, torch.bfloat16)
    half = ref.tile_bytes(128) // 2
    for b in range(2):
        page = c["pages"][c["table"][b, 0]]
        page[:, 1, :half] = page[:, 0, :half]
    c["seq"] = np.array([32, 32])       # rows 16 to 31 of the positions; the rows before them see less
    c["start"] = np.array([0, 16, 32])
    c["q"] = c["q"][:32].contiguous()
    c["max_q"] = 16
    check_large(ld, c, scale)


FEW_ROWS = [(0, 1), (16, 1), (17, 1), (300, 1), (95, 1), (1000, 1)]


@gpu
@pytest.mark.parametrize("D,group", [(64, 1), (64, 20), (128, 4), (128, 16), (256, 5), (256, 16)])
@pytest.mark.parametrize("kind", LARGE)
def test_large_scores_of_few_rows(ld, D, group, kind):  # noqa: F811
    c, scale = large_case(D + group, FEW_ROWS, D, group, kind)
    check_large(ld, c, scale)
    check_large(ld, c, scale, window=40)


@gpu
@pytest.mark.parametrize("kind", LARGE)
def test_large_scores_of_few_rows_over_a_long_context(ld, kind):  # noqa: F811
    """Parts of many CTAs, each with a largest score of its own."""
    c, scale = large_case(7, [(9000, 2), (400, 1)], 128, 4, kind)
    check_large(ld, c, scale)


@gpu
@pytest.mark.parametrize("scale", [2.0 ** 5, 2.0 ** 15, 2.0 ** 30])
def test_equal_large_scores_of_few_rows_share_the_weight(ld, scale):  # noqa: F811
    c = attention_case(np.random.default_rng(5), [(31, 1), (40, 1)], 128, 1, 4, 32, torch.bfloat16)
    half = ref.tile_bytes(128) // 2
    for b in range(2):
        page = c["pages"][c["table"][b, 0]]
        page[:, 1, :half] = page[:, 0, :half]
    check_large(ld, c, scale)


@gpu
@pytest.mark.parametrize("lens", [FEW_ROWS, MANY_ROWS], ids=["few", "many"])
def test_scores_grow_and_fall_across_the_limit_along_a_context(ld, lens):  # noqa: F811
    """Keys that grow from 2^-4 to 2^10 along the tokens, and ones that fall: the largest score moves from
    ordinary sizes to large ones, and a row's first large one stays."""
    for flip in (False, True):
        c = attention_case(np.random.default_rng(9), lens, 128, 1, 4, 32, torch.bfloat16)
        half = ref.tile_bytes(128) // 2
        for b, s in enumerate(c["seq"]):
            size = 2.0 ** np.linspace(-4, 10, s)[::-1 if flip else 1]
            for t in range(s):
                pair = c["pages"][c["table"][b, t // 32], 0, t % 32 // 16, 8 * 128:half].view(np.float16).reshape(16, 4)
                pair[t % 16] = pair[t % 16] * size[t]
        check_large(ld, c, 16.0)
        check_large(ld, c, -16.0)


def spoil_value(c, b, t, group, fill):
    """A token's value pair of one group becomes (fill, fill)."""
    D, half = c["D"], ref.tile_bytes(c["D"]) // 2
    tile = c["pages"][c["table"][b, t // c["P"]], :, t % c["P"] // 16, half + 8 * D:]
    pairs = np.ascontiguousarray(tile).view(np.float16).reshape(len(tile), 16, D // 64, 2)
    pairs[:, t % 16, group] = fill
    tile[:] = pairs.reshape(len(tile), -1).view(np.uint8)


def spoiled(c, places, window, fill):
    """The case with values that are not finite, which outputs [n, Q, D] see them, and what the rest should be."""
    q, scale = c["q"].double().cpu().numpy(), c["D"] ** -0.5
    want, want_lse, big, _ = ref.attend(q, c["pages"], c["P"], c["table"], c["start"], c["seq"], scale, window)
    hit = np.zeros(want.shape, bool)
    for b, t, group in places:
        spoil_value(c, b, t, group, fill)
        a, e, seq = int(c["start"][b]), int(c["start"][b + 1]), int(c["seq"][b])
        pos = seq - (e - a) + np.arange(e - a)
        sees = (t <= pos) & ((t > pos - window) if window else True)
        hit[a:e, :, 64 * group:64 * (group + 1)] |= sees[:, None, None]
    return hit, want, want_lse, big


@gpu
@pytest.mark.parametrize("fill", [np.nan, np.inf])
@pytest.mark.parametrize("D,group,lens,window,places", [
    (128, 1, [(0, 256)], 0, [(0, 5, 0)]), (64, 1, [(0, 300), (0, 256)], 0, [(0, 130, 0), (1, 100, 0)]),
    (128, 1, [(0, 256)], 60, [(0, 5, 1), (0, 140, 0)]), (128, 4, [(10, 64), (0, 40)], 0, [(0, 20, 1), (1, 0, 0)]),
    (256, 2, [(3, 130)], 0, [(0, 40, 3), (0, 70, 1)]), (128, 1, [(3000, 256)], 0, [(0, 2990, 1), (0, 3100, 0), (0, 100, 0)]),
    (128, 1, [(0, 256)], 130, [(0, 0, 0), (0, 255, 1)])])
def test_many_rows_that_see_a_value_that_is_not_finite_show_it(ld, D, group, lens, window, places, fill):  # noqa: F811
    """A tile may be hidden from some rows of one half of an item's rows and seen by all of the other."""
    c = attention_case(np.random.default_rng(D + window), lens, D, 1, group, 32, torch.bfloat16)
    hit = spoiled(c, places, window, fill)[0]
    got = run_attention(ld, c, window)[0].float().cpu().numpy()
    # (steps and least values that are infinities stand for inf * code + inf, an infinity or a NaN)
    assert not np.isfinite(got[hit]).any() and (np.isinf(fill) or np.isnan(got[hit]).all())
    sees = hit.any(-1)
    assert np.isfinite(got[~sees]).all()


@gpu
@pytest.mark.parametrize("D,group,lens,window,places", [
    (128, 1, [(0, 256)], 60, [(0, 5, 1), (0, 140, 0)]), (128, 4, [(10, 64), (0, 40)], 0, [(0, 20, 1), (1, 0, 0)]),
    (256, 2, [(3, 130)], 0, [(0, 40, 3), (0, 70, 1)]), (128, 1, [(3000, 256)], 0, [(0, 2990, 1), (0, 3100, 0), (0, 100, 0)]),
    (128, 4, [(30, 1), (64, 1), (40, 1)], 0, [(0, 29, 0), (1, 3, 1), (2, 40, 1)]), (256, 2, [(50, 8)], 20, [(0, 40, 2), (0, 55, 0)]),
    (64, 1, [(90, 5)], 0, [(0, 92, 0)]), (128, 8, [(5000, 1)], 0, [(0, 5000, 1), (0, 77, 0)])])
def test_a_value_that_is_not_finite_shows_in_its_group_only(ld, D, group, lens, window, places):  # noqa: F811
    """The result's dims of other groups, and the logarithm of the denominator, do not depend on it."""
    c = attention_case(np.random.default_rng(D + group), lens, D, 1, group, 32, torch.bfloat16)
    hit, want, want_lse, big = spoiled(c, places, window, np.nan)
    out, lse, err = run_attention(ld, c, window)
    assert err == 0
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), hit)
    # (a row's weights are its own, so the rest is as it was before)
    bound = NP_TYPE[c["dtype"]] * np.abs(want) + 2.0 ** -9 * big[..., None]
    assert (np.abs(got - want) <= bound)[~hit].all()
    assert (np.abs(got_lse - want_lse) <= 2.0 ** -9 + 2.0 ** -20 * np.abs(want_lse)).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_groups_beyond_f16_read_as_nan_and_ones_up_to_it_do_not(ld, dtype):  # noqa: F811
    D, n = 128, 16
    x = torch.randn(n, 1, D, device="cuda").to(dtype)
    limit = 65280.0 if dtype == torch.bfloat16 else 65440.0  # (65280 is the last of bfloat16)
    x[0, 0, 3], x[1, 0, 70], x[2, 0, :64] = limit, -limit, limit
    x[3, 0, 64], x[3, 0, 65] = limit, -limit
    held = torch.ones(n, 2, dtype=torch.bool, device="cuda")
    if dtype == torch.bfloat16:
        x[5, 0, 3], x[6, 0, 127], x[7, 0, :64], x[8, 0, 64:] = 65536.0, -70000.0, 1e5, -1e30
        x[9, 0, :64], x[10, 0, 0], x[10, 0, 1] = torch.linspace(0, 5e5, 64, device="cuda").to(dtype), 3e38, -3e38
        held[5, 0] = held[6, 1] = held[7, 0] = held[8, 1] = held[9, 0] = held[10, 0] = False
    x[11, 0, :64], x[12, 0, 64:], x[13, 0, 9] = float("inf"), -float("inf"), float("nan")
    held[11, 0] = held[12, 1] = held[13, 0] = False
    cache, err = ld.Kv4Cache.empty(1, 16, 1, D, dtype), ld.new_error_word()
    slots = torch.arange(n, device="cuda")
    k, v = torch.empty(2, n, 1, D, device="cuda", dtype=dtype)
    ld.lora_kv4_append(cache, x, x, slots, err=err)
    ld.lora_kv4_read(cache, k, v, slots, err=err)
    assert ld.lora_get_error(err) == 0
    for got in (k, v):
        g, w = got.float().view(n, 2, 64), x.float().view(n, 2, 64)
        assert torch.equal(torch.isnan(g).all(-1), ~held) and torch.equal(torch.isfinite(g).all(-1), held)
        # half a step, the step's rounding 15 times over, and the row type's
        step = (w.amax(-1) - w.amin(-1)) / 15
        bound = 0.5 * step + 16 * step * 2.0 ** -11 + w.abs().amax(-1) * (2.0 ** -10 + NP_TYPE[dtype])
        assert ((g - w).abs() <= bound[..., None])[held].all()


@gpu
@pytest.mark.parametrize("lens", [FEW_ROWS, MANY_ROWS], ids=["few", "many"])
def test_attention_over_groups_beyond_f16(ld, lens):  # noqa: F811
    """Rows that see a key or value which the cache does not hold are NaN, be it read by either kernel."""
    c = attention_case(np.random.default_rng(4), lens, 64, 1, 4, 32, torch.bfloat16)
    cache = ld.Kv4Cache(dev(c["pages"], np.uint8), 32, 64)
    b = 1
    at = int(c["seq"][b]) - 1
    slot = dev([int(c["table"][b, at // 32]) * 32 + at % 32], np.int64)
    x = torch.zeros(1, 1, 64, device="cuda").bfloat16()
    x[0, 0, 5] = 1e5
    for k, v in ((torch.zeros_like(x), x), (x, torch.zeros_like(x))):
        ld.lora_kv4_append(cache, k, v, slot)
        out = run_attention(ld, c, cache=cache)[0].float()
        last = int(c["start"][b + 1]) - 1
        assert torch.isnan(out[last]).all() and torch.isfinite(out[:last]).all() and torch.isfinite(out[last + 1:]).all()


def keys_case(seed, lens, D, group, dtype, key_of, q_of):
    """A case whose keys and queries are changed before they are stored: key_of(k [s, D]), q_of(q [n, Q, D])."""
    rng = np.random.default_rng(seed)
    c = attention_case(rng, lens, D, 1, group, 32, dtype)
    for b, s in enumerate(c["seq"]):
        t = np.arange(s)
        k, v = rng.standard_normal((2, s, 1, D))
        k = key_of(k[:, 0])[:, None]
        k, v = (torch.from_numpy(x).to(dtype).double().numpy() for x in (k, v))
        ref.append(c["pages"], k, v, c["table"][b, t // 32].astype(np.int64) * 32 + t % 32, 32)
    c["q"] = torch.from_numpy(q_of(rng.standard_normal(c["q"].shape))).to(dtype).cuda()
    return c


def check_scores(ld, c):  # noqa: F811
    """The logarithm of the denominator is as exact as the scores: e, and 2^-9 for weights rounded to 16 bits."""
    out, lse, err = run_attention(ld, c)
    want, want_lse, big, _ = ref.attend(c["q"].double().cpu().numpy(), c["pages"], c["P"], c["table"], c["start"],
                                        c["seq"], c["D"] ** -0.5, 0)
    assert err == 0
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    room, off = score_room(c, c["D"] ** -0.5)
    assert (np.abs(got_lse - want_lse) <= 2.0 ** -9 + off).all(), float((np.abs(got_lse - want_lse) - off).max())
    bound = NP_TYPE[c["dtype"]] * np.abs(want) + (2.0 ** -9 + 2 * room[..., None]) * big[..., None]
    assert (np.abs(got - want) <= bound).all()


def times(x, at, by):
    x = x.copy()
    x[at] *= by
    return x


@gpu
@pytest.mark.parametrize("D,group,head", [(128, 4, 3), (128, 4, 1), (64, 8, 5), (256, 2, 1)])
def test_scores_of_a_head_with_large_queries(ld, D, group, head):  # noqa: F811
    """One query head of a group is 30 times the others."""
    c = keys_case(D, [(0, 300), (200, 90)], D, group, torch.bfloat16, lambda k: k, lambda q: times(q, np.s_[:, head], 30.0))
    check_scores(ld, c)


@gpu
def test_scores_of_one_row_with_a_large_query(ld):  # noqa: F811
    for row in (0, 1, 77, 128, 255, 299):
        c = keys_case(row, [(0, 300)], 128, 4, torch.bfloat16, lambda k: k, lambda q: times(q, np.s_[row, 2], 100.0))
        check_scores(ld, c)


@gpu
@pytest.mark.parametrize("at", range(16))
def test_scores_of_one_large_key_in_each_place_of_a_block(ld, at):  # noqa: F811
    """One token in 300 has a key 60 times the others' size."""
    c = keys_case(at, [(0, 300), (100, 60)], 128, 2, torch.bfloat16, lambda k: times(k, 64 + at, 60.0), lambda q: q)
    check_scores(ld, c)


@gpu
@pytest.mark.parametrize("D,size", [(128, 10.0), (64, 8.0), (256, 12.0), (128, 30.0)])
def test_scores_of_a_dim_that_is_strong_in_queries_and_keys(ld, D, size):  # noqa: F811
    for dim in (0, 13, D - 1):
        c = keys_case(dim, [(0, 300), (500, 70)], D, 4, torch.bfloat16, lambda k: times(k, np.s_[:, dim], size),
                      lambda q: times(q, np.s_[..., dim], size))
        check_scores(ld, c)


@gpu
def test_requests_of_many_rows_do_not_depend_on_their_neighbours(ld):  # noqa: F811
    """The same requests in another order, with keys about the size from which two operands are taken."""
    rng = np.random.default_rng(17)
    lens = [(int(a), int(b)) for a, b in zip(rng.integers(0, 300, 40), rng.integers(33, 200, 40))]
    c = keys_case(1, lens, 128, 4, torch.bfloat16, lambda k: k * np.exp(rng.standard_normal((len(k), 1)) * 0.5), lambda q: q * 2.5)
    out, lse, _ = run_attention(ld, c)
    order = rng.permutation(40)
    rows = np.concatenate([np.arange(c["start"][b], c["start"][b + 1]) for b in order])
    d = dict(c, table=c["table"][order], seq=c["seq"][order], q=c["q"][torch.from_numpy(rows).cuda()].contiguous(),
             start=np.concatenate([[0], np.cumsum([lens[b][1] for b in order])]))
    out2, lse2, _ = run_attention(ld, d)
    at = torch.from_numpy(rows).cuda()
    assert torch.equal(out[at], out2) and torch.equal(lse[at], lse2)
