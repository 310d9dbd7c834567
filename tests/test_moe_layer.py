"""The routed-expert layer around the deltas: tokens sorted by expert and back, their gradients, and the products with an
epilogue, against plain 64-bit numpy forms.

Tolerances.  Plans and rows moved are equal.  Other results are off by the rounding of the result, half a step of its type
(2^-9 |y| to 2^-8 |y| in bf16: 2^-8; f16: 2^-11), plus what float32 sums may add: for combine k additions of products
rounded to 2^-24 each of the sum of magnitudes; for dots 2^-24 of it for each of H additions, in practice far less; for
products as ``moe_ref.linear`` derives it.  Below the normal range a step is absolute: 2^-25 in f16.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

from tests import moe_ref as ref

STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.bfloat16, torch.float16]
gpu = pytest.mark.gpu


# --------------------------------------------------------------------- CPU --

def test_plan_form_is_a_stable_sort():
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, 5, (40, 3))
    p = ref.plan(ids, 5)
    key = ids.reshape(-1)
    order = [i for i in np.argsort(np.where(key < 0, 99, key), kind="stable") if key[i] >= 0]
    assert np.array_equal(p["row_pair"][:len(order)], order) and (p["row_pair"][len(order):] == -1).all()
    assert p["err"] == 0 and p["seg_start"][-1] == len(order)


def test_forms_are_each_others_gradients():
    """Differences of a loss through combine, and through dispatch, against the gradient forms."""
    rng = np.random.default_rng(1)
    T, k, E, H = 7, 2, 3, 4
    p = ref.plan(rng.integers(-1, E, (T, k)), E)
    rows, w, g = rng.standard_normal((T * k, H)), rng.standard_normal((T, k)), rng.standard_normal((T, H))
    grad_rows, grad_w, _ = ref.combine_grad(g, rows, p["pair_row"], w)

    def loss(rows, w):
        return (ref.combine(rows, p["pair_row"], w)[0] * g).sum()

    step = 1e-5
    for i in np.ndindex(*rows.shape):
        d = np.zeros_like(rows)
        d[i] = step
        got = (loss(rows + d, w) - loss(rows - d, w)) / (2 * step)
        assert abs(got - (0 if np.isnan(grad_rows[i]) else grad_rows[i])) < 1e-8
    for i in np.ndindex(*w.shape):
        d = np.zeros_like(w)
        d[i] = step
        assert abs((loss(rows, w + d) - loss(rows, w - d)) / (2 * step) - grad_w[i]) < 1e-8
    # dispatch is linear: its transpose is combine without weights
    x, y = rng.standard_normal((T, H)), rng.standard_normal((T * k, H))
    moved = np.where(p["row_pair"][:, None] >= 0, x[p["row_pair"] // k], 0)
    assert abs((moved * y).sum() - (ref.combine(y, p["pair_row"])[0] * x).sum()) < 1e-10


def test_refusals_on_the_host():
    import lora_delta_gb300 as ld
    from lora_delta_gb300.build import build
    build()
    L = ld.lib()
    at = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(12)]  # never dereferenced: the checks come first
    odd = ctypes.c_void_p(0x10000008)
    ok, arg, shape, align, unsup = 0, 1, 2, 3, 6

    def dispatch(rows=at[0], ld_rows=64, seg=at[1], pair=at[2], x=at[3], ld_x=64, ids=at[4], lora=at[5], m=None, nm=0, T=8, k=2,
                 E=4, H=64, row_pair=at[6]):
        return L.lora_moe_dispatch(rows, ld_rows, seg, row_pair, pair, at[7], at[8], x, ld_x, ids, lora, m, nm, T, k, E, H, None, None)

    assert dispatch(rows=None) == arg and dispatch(seg=None) == arg and dispatch(pair=None) == arg and dispatch(x=None) == arg
    assert dispatch(ids=None) == arg and dispatch(T=-1) == arg and dispatch(k=0) == arg and dispatch(E=0) == arg
    assert dispatch(H=0) == arg and dispatch(m=at[9], nm=0) == arg
    assert dispatch(H=60) == align and dispatch(ld_x=68) == align and dispatch(rows=odd) == align
    assert dispatch(ids=ctypes.c_void_p(0x50000002)) == align
    assert dispatch(ld_rows=56) == shape and dispatch(ld_x=56) == shape
    assert dispatch(E=1025) == unsup and dispatch(k=65) == unsup and dispatch(T=1 << 30) == unsup
    assert dispatch(x=at[0]) == arg and dispatch(x=ctypes.c_void_p(0x10000000 + 2 * 64 * 15)) == arg
    assert dispatch(ids=at[2]) == arg and dispatch(seg=at[2]) == arg and dispatch(pair=at[0]) == arg and dispatch(row_pair=at[3]) == arg

    def combine(out=at[0], ld_out=64, rows=at[1], ld_rows=64, pair=at[2], w=at[3], res=at[4], ld_res=64, T=8, k=2, H=64, t=0):
        return L.lora_moe_combine(out, ld_out, rows, ld_rows, pair, w, res, ld_res, T, k, H, t, None)

    assert combine(T=0, out=None) == ok
    assert combine(out=None) == arg and combine(rows=None) == arg and combine(pair=None) == arg and combine(t=2) == arg
    assert combine(rows=at[0]) == arg and combine(w=at[0]) == arg and combine(res=at[0], ld_res=72) == arg
    assert combine(res=ctypes.c_void_p(0x10000000 + 128)) == arg
    assert combine(ld_out=60) == shape and combine(ld_rows=68) == align and combine(res=odd) == align and combine(k=65) == unsup

    def grad(gr=at[0], ld_gr=64, gw=at[1], go=at[2], rows=at[3], pair=at[4], w=at[5], T=8, k=2, H=64, t=0):
        return L.lora_moe_combine_grad(gr, ld_gr, gw, go, 64, rows, 64, pair, w, T, k, H, t, None)

    assert grad(T=0) == ok and grad(gr=None) == arg and grad(go=None) == arg and grad(rows=None) == arg and grad(pair=None) == arg
    assert grad(rows=at[0]) == arg and grad(go=at[0]) == arg and grad(gw=at[5]) == arg and grad(gw=at[0]) == arg
    assert grad(H=4) == align and grad(ld_gr=56) == shape and grad(t=-1) == arg

    def linear(out=at[0], ld_out=48, x=at[1], ld_x=64, n=5, K=64, w=at[2], ld_w=64, N=48, bias=at[3], delta=at[4], ld_delta=48,
               res=at[5], ld_res=48, act=0, gated=0, t=0, E=0, seg=at[6], stride=48 * 64, work=None, wsb=0):
        if E:
            return L.lora_moe_linear(out, ld_out, x, ld_x, n, K, seg, E, w, ld_w, stride, N, bias, delta, ld_delta, res, ld_res,
                                     act, gated, t, work, wsb, None, None)
        return L.lora_linear(out, ld_out, x, ld_x, n, K, w, ld_w, N, bias, delta, ld_delta, res, ld_res, act, gated, t, work, wsb, None, None)

    for E in (0, 3):
        assert linear(E=E, n=0, out=None) == ok
        assert linear(E=E, out=None) == arg and linear(E=E, x=None) == arg and linear(E=E, w=None) == arg
        assert linear(E=E, n=-1) == arg and linear(E=E, K=0) == arg and linear(E=E, N=0) == arg
        assert linear(E=E, act=5) == arg and linear(E=E, act=-1) == arg and linear(E=E, gated=2) == arg and linear(E=E, t=2) == arg
        assert linear(E=E, K=60) == align and linear(E=E, N=44) == align and linear(E=E, N=40, gated=1) == align
        assert linear(E=E, x=odd) == align and linear(E=E, ld_w=68) == align and linear(E=E, bias=odd) == align
        assert linear(E=E, ld_out=40) == shape and linear(E=E, ld_x=56) == shape and linear(E=E, ld_delta=40) == shape
        assert linear(E=E, x=at[0]) == arg and linear(E=E, w=at[0]) == arg and linear(E=E, delta=at[0]) == arg
        assert linear(E=E, bias=at[0]) == arg and linear(E=E, res=at[0], ld_res=56) == arg
        assert linear(E=E, res=ctypes.c_void_p(0x10000000 + 96)) == arg
        assert linear(E=E, n=1000, work=at[7], wsb=1000) == 5 and linear(E=E, work=odd, wsb=1 << 30) == align
    assert linear(E=3, seg=None) == arg and linear(E=3, stride=47 * 64) == shape and linear(E=3, stride=48 * 64 + 8) == shape
    assert linear(n=2 ** 30 + 1) == unsup and linear(E=1025) == unsup and linear(E=3, seg=at[0]) == arg


def test_refusals_of_shared_workspaces_and_error_words():
    """The workspace and the error word are written too: no argument may lie in them."""
    import lora_delta_gb300 as ld
    from lora_delta_gb300.build import build
    build()
    L = ld.lib()
    base, n, E = 1 << 40, 1000, 3
    at = {name: base + i * (1 << 30) for i, name in enumerate(("out", "x", "w", "bias", "delta", "res", "seg", "err", "work"))}
    size = int(L.lora_linear_workspace_size(n, E))
    assert size == int(L.lora_linear_workspace_size(n, 1)) > 1 << 20

    def linear(experts, **other):
        p = {k: ctypes.c_void_p(v) for k, v in {**at, **other}.items()}
        if experts:
            return L.lora_moe_linear(p["out"], 48, p["x"], 64, n, 64, p["seg"], E, p["w"], 64, 48 * 64, 48, p["bias"], p["delta"], 48,
                                     p["res"], 48, 0, 0, 0, p["work"], size, p["err"], None)
        return L.lora_linear(p["out"], 48, p["x"], 64, n, 64, p["w"], 64, 48, p["bias"], p["delta"], 48, p["res"], 48, 0, 0, 0, p["work"],
                             size, p["err"], None)

    last = {"out": 2 * n * 48, "x": 2 * n * 64, "delta": 2 * n * 48, "res": 2 * n * 48}
    for experts in (False, True):
        last.update(w=2 * (E if experts else 1) * 48 * 64, bias=2 * (E if experts else 1) * 48, seg=4 * (E + 1), err=4)
        for name in at:
            if name == "work" or (name == "seg" and not experts):
                continue
            # inside the workspace, and with its last bytes in the first of it
            assert linear(experts, **{name: at["work"] + size - 256}) == 1, name
            end = (last[name] - 4) // 256 * 256 if name != "err" else 0
            assert linear(experts, work=at[name] + end) == 1, name
            if name != "err":
                assert linear(experts, err=at[name]) == 1 and linear(experts, err=at[name] + last[name] - 4) == 1, name
        # the residual's excuse is its own
        assert linear(experts, res=at["out"], x=at["out"]) == 1 and linear(experts, res=at["out"], err=at["out"] + 4) == 1

    def dispatch(err):
        p = [ctypes.c_void_p(base + i * (1 << 30)) for i in range(9)]
        return L.lora_moe_dispatch(p[0], 64, p[1], p[2], p[3], p[4], p[5], p[6], 64, p[7], p[8], None, 0, 8, 2, 4, 64, ctypes.c_void_p(err), None)

    for i in range(9):
        assert dispatch(base + i * (1 << 30)) == 1, i


def test_plans_are_made_on_the_gpu():
    import lora_delta_gb300 as ld
    with pytest.raises(ValueError):
        ld.MoePlan(4, 2, 8, device="cpu")
    for T, k, E in ((-1, 2, 8), (4, 0, 8), (4, 2, 0)):
        with pytest.raises(ValueError):
            ld.MoePlan(T, k, E)


# --------------------------------------------------------------------- GPU --

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
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def normal(rng, dtype, *shape, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * std).to(dtype).cuda()


def close(got, want, bound, dtype):
    """`got` within half a step of its type of `want`, and `bound` besides."""
    tiny = 2.0 ** -25 if dtype is torch.float16 else 2.0 ** -134
    off = np.abs(got - want)
    limit = bound + STEP[dtype] * (np.abs(want) + bound) + tiny
    assert np.isfinite(got).all() and (off <= limit).all(), (off - limit).max()


def route(rng, T, k, E, none=0.0, skew=False):
    """Distinct experts of each token, some tokens without any."""
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k), int)
    if skew:
        ids = np.minimum(ids, rng.integers(0, E, ids.shape))
    ids[rng.random(T) < none] = -1
    return ids


def dispatched(ld, ids, E, x, lora=None, m=None, rows=None):
    T, k = ids.shape
    plan, err = ld.MoePlan(T, k, E), ld.new_error_word()
    if rows is None:
        rows = torch.zeros(T * k, x.shape[1], dtype=x.dtype, device="cuda")
    ld.lora_moe_dispatch(rows, x, dev(ids), plan, lora_ids=None if lora is None else dev(lora),
                         expert_map=None if m is None else dev(m), err=err)
    return plan, rows, ld.lora_get_error(err)


def check_plan(plan, want):
    for name in ("seg_start", "row_pair", "pair_row", "row_expert", "row_lora"):
        assert np.array_equal(host(getattr(plan, name)), want[name]), name


@gpu
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 8), (1, 8, 64, 72), (64, 8, 64, 2048), (63, 3, 7, 264), (130, 16, 256, 4104), (300, 7, 1024, 16),
                                     (2500, 8, 64, 136), (9000, 4, 40, 8), (70001, 2, 33, 8), (20000, 16, 300, 24)])
def test_dispatch(ld, T, k, E, H):
    rng = np.random.default_rng(T + k)
    ids, lora = route(rng, T, k, max(E, k), none=0.1, skew=T % 2 == 0), rng.integers(-1, 9, T)
    ids = np.minimum(ids, E - 1)
    x = normal(rng, TYPES[T % 2], T, H)
    mark = torch.full((T * k, H), 7.0, dtype=x.dtype, device="cuda")
    plan, rows, err = dispatched(ld, ids, E, x, lora, rows=mark)
    want = ref.plan(ids, E, lora)
    assert err == 0
    check_plan(plan, want)
    count = want["seg_start"][-1]
    pairs = torch.from_numpy(want["row_pair"][:count] // k).cuda()
    assert torch.equal(rows[:count], x[pairs]) and (rows[count:] == 7).all()


@gpu
@pytest.mark.parametrize("T", [5, 3000])
def test_dispatch_of_ids_that_have_no_expert_here(ld, T):
    """Maps, padded tokens, ids out of range with and without a map, and a token that names an expert twice."""
    rng, E, k = np.random.default_rng(T), 5, 4
    x = normal(rng, torch.bfloat16, T, 16)
    m = np.array([3, -1, 0, 4, -1, 1, 2, -1, 9])  # (the last is no number of this rank)
    for ids, mp in ((rng.integers(-1, E, (T, k)), None), (rng.integers(-3, E + 2, (T, k)), None), (rng.integers(-1, 8, (T, k)), m),
                    (rng.integers(-2, 12, (T, k)), m), (np.full((T, k), -1), None), (np.full((T, k), 2), None)):
        plan, rows, err = dispatched(ld, ids, E, x, m=mp)
        want = ref.plan(ids, E, expert_map=mp)
        check_plan(plan, want)
        assert err == want["err"]
        count = want["seg_start"][-1]
        assert torch.equal(rows[:count], x[torch.from_numpy(want["row_pair"][:count] // k).cuda()]) and not rows[count:].any()


@gpu
def test_dispatch_of_no_tokens(ld):
    plan = ld.MoePlan(0, 4, 6)
    plan.seg_start.fill_(5)
    ld.lora_moe_dispatch(torch.empty(0, 8, device="cuda").bfloat16(), torch.empty(0, 8, device="cuda").bfloat16(),
                         torch.empty(0, 4, dtype=torch.int32, device="cuda"), plan)
    assert not plan.seg_start.any()
    ld.lora_moe_combine(torch.empty(0, 8, device="cuda").bfloat16(), torch.empty(0, 8, device="cuda").bfloat16(), plan)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H,weighted,residual", [(1, 1, 8, True, False), (1, 8, 2048, True, True), (63, 8, 2056, True, True), (200, 3, 72, False, False),
                                                     (17, 16, 4104, True, False), (5, 64, 264, False, True), (1000, 2, 520, True, True)])
def test_combine_and_its_gradient(ld, dtype, T, k, H, weighted, residual):
    rng, E = np.random.default_rng(T * k), max(k, 9)
    plan, _, _ = dispatched(ld, route(rng, T, k, E, none=0.15), E, normal(rng, dtype, T, 8))
    pair_row, count = host(plan.pair_row), int(plan.seg_start[-1])
    rows, g = normal(rng, dtype, T * k, H), normal(rng, dtype, T, H)
    rows[count:] = float("nan")  # what no pair leads to is not read
    w = dev(rng.standard_normal((T, k)), np.float32) if weighted else None
    w64 = host(w) if weighted else None
    res = normal(rng, dtype, T, H) if residual else None
    out = torch.full((T, H), float("nan"), dtype=dtype, device="cuda")
    ld.lora_moe_combine(out, rows, plan, weights=w, residual=res)
    want, size = ref.combine(host(rows), pair_row, w64, host(res) if residual else None)
    close(host(out), want, size * (k + 2) * 2.0 ** -23, dtype)
    if residual:  # in place
        ld.lora_moe_combine(res, rows, plan, weights=w, residual=res)
        assert torch.equal(res, out)
    grad_rows, grad_w = torch.full_like(rows, 3.0), torch.full((T, k), 3.0, device="cuda")
    ld.lora_moe_combine_grad(grad_rows, grad_w, g, rows, plan, weights=w)
    want_rows, want_w, size = ref.combine_grad(host(g), host(rows), pair_row, w64)
    assert (grad_rows[count:] == 3).all()
    close(host(grad_rows)[:count], want_rows[:count], 0.0, dtype)
    # (at most H / 8 + 16 float32 additions of the sums of 8 follow one another)
    assert (np.abs(host(grad_w) - want_w) <= size * (H / 8 + 24) * 2.0 ** -24).all()
    only = torch.full_like(rows, 3.0)
    ld.lora_moe_combine_grad(only, None, g, rows, plan, weights=w)
    assert torch.equal(only, grad_rows)


@gpu
def test_combine_skips_rows_that_are_none(ld):
    """A plan that a caller has written: entries outside the rows are no rows."""
    plan = ld.MoePlan(3, 2, 4)
    plan.pair_row.copy_(dev([[0, 6], [-5, 2 ** 31 - 1], [5, -2 ** 31]]))
    rows = torch.arange(48, device="cuda").view(6, 8).bfloat16()
    out = torch.empty(3, 8, device="cuda").bfloat16()
    ld.lora_moe_combine(out, rows, plan)
    assert torch.equal(out, torch.stack([rows[0], torch.zeros_like(rows[0]), rows[5]]))
    grad, gw = torch.full_like(rows, 9.0), torch.empty(3, 2, device="cuda")
    ld.lora_moe_combine_grad(grad, gw, out, rows, plan)
    assert torch.equal(grad[0], out[0]) and torch.equal(grad[5], out[2]) and (grad[1:5] == 9).all()
    assert gw[0, 1] == 0 and not gw[1].any() and gw[2, 1] == 0


LINEAR = [  # n, K, N, act, gated, bias, delta, residual
    (1, 8, 8, "none", False, False, False, False), (1, 4096, 520, "none", False, True, False, False),
    (3, 72, 16, "silu", True, True, True, True), (16, 2048, 1536, "silu", True, False, True, False),
    (17, 136, 264, "relu", False, True, False, True), (64, 1000, 392, "gelu", False, True, True, True),
    (65, 64, 128, "gelu_tanh", False, False, True, False), (100, 520, 48, "gelu", True, True, False, True),
    (129, 256, 640, "gelu_tanh", True, False, False, False), (200, 1032, 1000, "none", False, False, True, True),
    (255, 392, 272, "relu", True, True, True, False), (257, 128, 512, "silu", False, True, True, True),
    (700, 328, 1296, "silu", True, False, True, True), (1500, 904, 776, "none", False, True, False, True),
    # tiles shared along K by two pairs of CTAs and by more, whole rounds of tiles, no rows but one past a tile's
    (300, 8192, 512, "none", False, True, True, True), (1090, 4096, 1296, "silu", True, False, True, False),
    (5000, 72, 2064, "relu", False, False, False, True), (257, 5000, 272, "gelu", True, True, False, True)]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,K,N,act,gated,bias,delta,residual", LINEAR)
def test_linear(ld, dtype, n, K, N, act, gated, bias, delta, residual):
    rng = np.random.default_rng(n + K)
    width = N // 2 if gated else N
    x, w = normal(rng, dtype, n, K), normal(rng, dtype, N, K, std=K ** -0.5)
    b = normal(rng, dtype, N) if bias else None
    d = normal(rng, dtype, n, N) if delta else None
    r = normal(rng, dtype, n, width) if residual else None
    out, err = torch.full((n, width), float("nan"), dtype=dtype, device="cuda"), ld.new_error_word()
    ld.lora_linear(out, x, w, bias=b, delta=d, residual=r, activation=act, gated=gated, err=err)
    want, bound = ref.linear(*(None if t is None else host(t) for t in (x, w, b, d, r)), act=act, gated=gated)
    assert ld.lora_get_error(err) == 0
    close(host(out), want, bound, dtype)
    if residual:  # in place
        ld.lora_linear(r, x, w, bias=b, delta=d, residual=r, activation=act, gated=gated)
        assert torch.equal(r, out)


@gpu
def test_linear_on_columns_of_larger_tensors(ld):
    """Row strides, slices of a fused buffer on both sides, and what lies beside the result stays."""
    rng = np.random.default_rng(5)
    buf = normal(rng, torch.bfloat16, 90, 512)
    before, w = buf.clone(), normal(rng, torch.bfloat16, 200, 144)[:, 8:136]
    ld.lora_linear(buf[:, 200:400], buf[:, 64:192], w, residual=buf[:, 200:400], activation="relu")
    want, bound = ref.linear(host(before[:, 64:192]), host(w), residual=host(before[:, 200:400]), act="relu")
    close(host(buf[:, 200:400]), want, bound, torch.bfloat16)
    assert torch.equal(buf[:, :200], before[:, :200]) and torch.equal(buf[:, 400:], before[:, 400:])
    with pytest.raises(ld.LoraError) as e:
        ld.lora_linear(buf[:, 184:384], buf[:, 64:192], w)
    assert e.value.code == 1


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,K,N,act,gated,bias,delta,residual", [
    (1, 1, 1, 64, 16, "none", False, True, False, True), (1, 8, 64, 256, 160, "silu", True, False, True, False),
    (64, 8, 64, 512, 272, "silu", True, True, True, True), (40, 2, 3, 72, 392, "gelu", False, True, True, False),
    (200, 4, 8, 264, 128, "relu", False, False, False, True), (300, 8, 16, 136, 528, "gelu_tanh", True, True, False, False),
    (700, 3, 5, 128, 264, "none", False, False, True, True), (30, 2, 600, 64, 24, "silu", False, True, True, True),
    (2000, 4, 64, 64, 528, "silu", True, False, True, False), (400, 2, 3, 4096, 128, "none", False, True, False, True)])
def test_experts(ld, dtype, T, k, E, K, N, act, gated, bias, delta, residual):
    rng = np.random.default_rng(T + E)
    width, P = N // 2 if gated else N, T * k
    plan, x, _ = dispatched(ld, route(rng, T, k, max(E, k), none=0.1, skew=True) % E, E, normal(rng, dtype, T, K))
    seg = host(plan.seg_start)
    count = seg[-1]
    x[count:] = float("nan")
    w, b = normal(rng, dtype, E, N, K, std=K ** -0.5), normal(rng, dtype, E, N) if bias else None
    d, r = normal(rng, dtype, P, N) if delta else None, normal(rng, dtype, P, width) if residual else None
    out, err = torch.full((P, width), 5.0, dtype=dtype, device="cuda"), ld.new_error_word()
    ld.lora_moe_linear(out, x, w, plan, bias=b, delta=d, residual=r, activation=act, gated=gated, err=err)
    assert ld.lora_get_error(err) == 0 and (out[count:] == 5).all()
    got = host(out)
    for e in range(E):
        a, z = seg[e], seg[e + 1]
        if a < z:
            want, bound = ref.linear(host(x[a:z]), host(w[e]), host(b[e]) if bias else None, host(d[a:z]) if delta else None,
                                     host(r[a:z]) if residual else None, act, gated)
            close(got[a:z], want, bound, dtype)


@gpu
def test_experts_of_all_rows_at_one(ld):
    rng, T, E = np.random.default_rng(8), 600, 16
    plan, x, _ = dispatched(ld, np.full((T, 1), 11), E, normal(rng, torch.bfloat16, T, 64))
    w, out = normal(rng, torch.bfloat16, E, 80, 64), torch.zeros(T, 80, device="cuda").bfloat16()
    ld.lora_moe_linear(out, x, w, plan)
    want, bound = ref.linear(host(x), host(w[11]))
    close(host(out), want, bound, torch.bfloat16)


@gpu
def test_experts_report_segments_outside_the_rows(ld):
    rng = np.random.default_rng(9)
    for n in (40, 400):  # few rows an expert, and many
        for seg in ([0, 50, 30, 90], [-4, 10, 20, 40], [0, 10, 20, 2 ** 31 - 1], [70, 80, 90, 100], [0, n, 0, n], [2 ** 31 - 1, -1, n, 0]):
            if all(0 <= a <= b <= n for a, b in zip(seg, seg[1:])):
                continue
            plan, err = ld.MoePlan(n, 1, 3), ld.new_error_word()
            plan.seg_start.copy_(dev(seg))
            big = torch.full((n + 20, 24), 5.0, device="cuda").bfloat16()
            ld.lora_moe_linear(big[10:n + 10], normal(rng, torch.bfloat16, n, 64), normal(rng, torch.bfloat16, 3, 24, 64), plan, err=err)
            assert ld.lora_get_error(err) == 64
            assert (big[:10] == 5).all() and (big[n + 10:] == 5).all()


@gpu
def test_numbers_that_are_not_finite_stay_in_their_rows(ld):
    """A row's NaN or infinity, and one behind the experts' rows, reaches no other row."""
    rng = np.random.default_rng(10)
    for n, K, N in ((5, 64, 40), (70, 128, 264), (300, 192, 520)):
        x, w = normal(rng, torch.bfloat16, n, K), normal(rng, torch.bfloat16, N, K)
        clean, out = torch.empty(2, n, N, device="cuda").bfloat16()
        ld.lora_linear(clean, x, w)
        x[2, 3], x[4, K - 1] = float("nan"), float("inf")
        ld.lora_linear(out, x, w)
        rest = [i for i in range(n) if i not in (2, 4)]
        assert torch.equal(out[rest], clean[rest]) and out[2].isnan().all() and not out[4].isfinite().any()


@gpu
def test_activations_at_their_ends(ld):
    """Large and not finite arguments: z itself, 0, or what the formula gives."""
    z = torch.tensor([-60000.0, -300, -100, -88, -20, -1, -0.0, 0, 1, 20, 88, 100, 300, 60000, float("inf"), float("nan")], device="cuda").half()
    x, w = torch.zeros(1, 8, device="cuda").half(), torch.zeros(16, 8, device="cuda").half()
    out = torch.empty(1, 16, device="cuda").half()
    for act in ("none", "relu", "silu", "gelu", "gelu_tanh"):
        ld.lora_linear(out, x, w, bias=z, activation=act)
        want = {"none": z, "relu": torch.relu(z), "silu": z.double() * torch.sigmoid(z.double()),
                "gelu": torch.nn.functional.gelu(z.double()), "gelu_tanh": torch.nn.functional.gelu(z.double(), approximate="tanh")}[act]
        assert torch.allclose(out[0].double(), want.double(), rtol=2.0 ** -10, atol=2.0 ** -24, equal_nan=True), act


@gpu
def test_binding_refuses(ld):
    rng = np.random.default_rng(11)
    x, w, out = normal(rng, torch.bfloat16, 6, 64), normal(rng, torch.bfloat16, 32, 64), torch.empty(6, 32, device="cuda").bfloat16()
    plan, ids = ld.MoePlan(3, 2, 4), dev(np.zeros((3, 2)))
    bad = [lambda: ld.lora_linear(out, x.float(), w), lambda: ld.lora_linear(out, x.cpu(), w), lambda: ld.lora_linear(out, x, w.half()),
           lambda: ld.lora_linear(out[:5], x, w), lambda: ld.lora_linear(out, x, w[:, :32]), lambda: ld.lora_linear(out, x, w.t()),
           lambda: ld.lora_linear(out, x, w, gated=True), lambda: ld.lora_linear(out, x, w, activation="tanh"),
           lambda: ld.lora_linear(out, x, w, bias=w[0]), lambda: ld.lora_linear(out, x, w, delta=out[:, :16]),
           lambda: ld.lora_linear(out, x, w, residual=out.float()), lambda: ld.lora_linear(out, x, w, err=torch.zeros(1, device="cuda")),
           lambda: ld.lora_moe_linear(out, x, w, plan), lambda: ld.lora_moe_linear(out, x, w.expand(3, 32, 64), plan),
           lambda: ld.lora_moe_dispatch(x, x[:3], ids.long(), plan), lambda: ld.lora_moe_dispatch(x, x[:3], ids[:2], plan),
           lambda: ld.lora_moe_dispatch(x[:5], x[:3], ids, plan), lambda: ld.lora_moe_dispatch(x.half(), x[:3], ids, plan),
           lambda: ld.lora_moe_combine(out[:3], x, plan), lambda: ld.lora_moe_combine(out[:3], out, plan, weights=out[:3, :2]),
           lambda: ld.lora_moe_combine_grad(x, None, x[:3], out, plan),
           lambda: ld.lora_moe_combine_grad(x, ids, x[:3].clone(), x.clone(), plan), lambda: setattr(plan, "seg_start", plan.seg_start)]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, AttributeError)):
            call()
            raise RuntimeError(f"call {i} was taken")
    # a weight shared by all experts has no stride
    with pytest.raises(ld.LoraError):
        ld.lora_moe_linear(out, x, w[None].expand(4, 32, 64), plan)


def layer_case(ld, seed, T=90, k=3, E=6, H=256, I=128, rank=16, L=3, dtype=torch.bfloat16):
    rng = np.random.default_rng(seed)

    def bank(*shape, std):
        return normal(rng, dtype, E, L, *shape, std=std)

    c = {"ids": route(rng, T, k, E, none=0.1), "lora": rng.integers(-1, L, T), "x": normal(rng, dtype, T, H),
         "w": dev(rng.random((T, k)), np.float32), "w13": normal(rng, dtype, E, 2 * I, H, std=H ** -0.5),
         "w2": normal(rng, dtype, E, H, I, std=I ** -0.5), "a13": [bank(rank, H, std=H ** -0.5) for _ in range(2)],
         "b13": [bank(I, rank, std=rank ** -0.5) for _ in range(2)], "a2": bank(rank, I, std=I ** -0.5), "b2": bank(H, rank, std=rank ** -0.5)}
    c.update(E=E, I=I, rank=rank, L=L, H=H, k=k, T=T)
    return c


def pointers(banks):
    return torch.tensor([[b[e].data_ptr() for e in range(b.shape[0])] for b in banks], dtype=torch.int64, device="cuda")


def run_layer(ld, c, plan=None, stream=None):
    """dispatch, gate and up with the adapters' delta, down, its delta, combine: the calls' results in a dict."""
    P, dtype = c["T"] * c["k"], c["x"].dtype
    plan = plan or ld.MoePlan(c["T"], c["k"], c["E"])
    rows = torch.zeros(P, c["H"], dtype=dtype, device="cuda")
    d13, act = torch.zeros(P, 1, 2 * c["I"], dtype=dtype, device="cuda"), torch.zeros(P, c["I"], dtype=dtype, device="cuda")
    y, out = torch.zeros(P, c["H"], dtype=dtype, device="cuda"), torch.zeros_like(c["x"])
    if "ptr" not in c:
        c["ptr"] = pointers(c["a13"]), pointers(c["b13"]), pointers([c["a2"]])[0].contiguous(), pointers([c["b2"]])[0].contiguous()
        c["d_ids"], c["d_lora"] = dev(c["ids"]), dev(c["lora"])
    a13, b13, a2, b2 = c["ptr"]
    R, H, I = c["rank"], c["H"], c["I"]
    kw = {"stream": stream}
    ld.lora_moe_dispatch(rows, c["x"], c["d_ids"], plan, lora_ids=c["d_lora"], **kw)
    ids = plan.row_expert.view(P, 1)
    ld.lora_moe_fc1_delta(d13, rows, a13, R * H, b13, I * R, False, ids, plan.row_lora, c["E"], I, R, c["L"], 2.0, **kw)
    ld.lora_moe_linear(act, rows, c["w13"], plan, delta=d13.view(P, -1), activation="silu", gated=True, **kw)
    ld.lora_moe_linear(y, act, c["w2"], plan, **kw)
    ld.lora_moe_w2_delta(y.view(P, 1, H), act, a2, R * I, b2, H * R, ids, plan.row_lora, c["E"], H, R, c["L"], 2.0, **kw)
    ld.lora_moe_combine(out, y, plan, weights=c["w"], residual=c["x"], **kw)
    return {"plan": plan, "rows": rows, "d13": d13, "act": act, "y": y, "out": out}


@gpu
def test_a_layer_of_experts_with_adapters(ld):
    """The calls one after another as a layer, against the layer's formula in 64 bits from its inputs.

    Each of the five intermediate roundings (d13, act, y twice, out) is half a bf16 step of its value; carried through
    the products they grow with the root of the sum: the norm of a token's error stays below 6 * 2^-9 of the norm of what
    is rounded, and the test takes twice that, 2^-5.4 of out's norm less the residual's part."""
    c = layer_case(ld, 21)
    got = run_layer(ld, c)
    x, out = host(c["x"]), host(got["out"])
    w13, w2, w = host(c["w13"]), host(c["w2"]), host(c["w"])
    (ag, au), (bg, bu), a2, b2 = [host(b) for b in c["a13"]], [host(b) for b in c["b13"]], host(c["a2"]), host(c["b2"])
    for t in range(c["T"]):
        total, l = np.zeros(c["H"]), c["lora"][t]
        for j in range(c["k"]):
            e = c["ids"][t, j]
            if e < 0:
                continue
            z = w13[e] @ x[t]
            if l >= 0:
                z = z + 2.0 * np.concatenate([bg[e, l] @ (ag[e, l] @ x[t]), bu[e, l] @ (au[e, l] @ x[t])])
            h = ref.activation(z[:c["I"]], "silu") * z[c["I"]:]
            y = w2[e] @ h
            if l >= 0:
                y = y + 2.0 * b2[e, l] @ (a2[e, l] @ h)
            total += w[t, j] * y
        # (the sum's own error, and the rounding of the result)
        off = np.linalg.norm(out[t] - x[t] - total)
        assert off <= 12 * 2.0 ** -9 * np.linalg.norm(total) + 2.0 ** -8 * np.linalg.norm(x[t] + total)
    assert ld.lora_get_error(ld.new_error_word()) == 0


@gpu
def test_a_captured_layer_replays_on_new_inputs(ld):
    """A layer's calls in a graph, replayed with other tokens and routes on a stream of its own, beside eager calls."""
    cases = [layer_case(ld, 30 + i) for i in range(3)]
    want = [run_layer(ld, c)["out"].clone() for c in cases]
    base = layer_case(ld, 30)
    run_layer(ld, base)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        got = run_layer(ld, base)
    names = ("x", "w", "w13", "w2", "a2", "b2")
    for c, y in zip(cases, want):
        for n in names:
            base[n].copy_(c[n])
        for n in ("a13", "b13"):
            for t, u in zip(base[n], c[n]):
                t.copy_(u)
        base["d_ids"].copy_(dev(c["ids"]))
        base["d_lora"].copy_(dev(c["lora"]))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        assert torch.equal(run_layer(ld, c)["out"], y)
        torch.cuda.synchronize()
        assert torch.equal(got["out"], y)


@gpu
def test_calls_on_two_streams_at_once(ld):
    cases = [layer_case(ld, 40 + i, T=400) for i in range(2)]
    want = [run_layer(ld, c)["out"].clone() for c in cases]
    streams, got = [torch.cuda.Stream() for _ in cases], [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run_layer(ld, cases[i])["out"])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


@gpu
def test_results_repeat_and_do_not_depend_on_neighbours(ld):
    """Bit for bit: a call again, a token's combine alone, and a row of a product beside other rows."""
    rng = np.random.default_rng(50)
    x, w = normal(rng, torch.bfloat16, 64, 1024), normal(rng, torch.bfloat16, 512, 1024, std=1 / 32)
    a, b = torch.empty(2, 64, 512, device="cuda").bfloat16()
    ld.lora_linear(a, x, w)
    for _ in range(5):
        ld.lora_linear(b, x, w)
        assert torch.equal(a, b)
    y = x.clone()
    y[32:] = 0
    ld.lora_linear(b, y, w)
    assert torch.equal(a[:32], b[:32])


@gpu
@pytest.mark.parametrize("n,gated", [(5, False), (64, True), (300, False), (700, True)])
def test_a_wait_that_gives_up_is_reported(ld, n, gated):
    """With a limit of 0 a wait gives up at its first look, which may itself block for a while: the call reports it, or no
    wait was too long and it is whole.  The next call is whole, its workspace's counters at zero."""
    rng = np.random.default_rng(60)
    x, w = normal(rng, torch.bfloat16, n, 2048), normal(rng, torch.bfloat16, 512, 2048)
    want, out = torch.empty(2, n, 256 if gated else 512, device="cuda").bfloat16()
    ld.lora_linear(want, x, w, gated=gated)
    err = ld.new_error_word()
    torch.cuda.synchronize()
    old = ld.lora_set_wait_limit_ns(0)
    try:
        ld.lora_linear(out, x, w, gated=gated, err=err)
        bits = ld.lora_get_error(err)
        assert bits == 8 or (bits == 0 and torch.equal(out, want))
    finally:
        ld.lora_set_wait_limit_ns(old)
    for _ in range(2):
        out.fill_(3)
        ld.lora_linear(out, x, w, gated=gated, err=err)
        assert ld.lora_get_error(err) == 0 and torch.equal(out, want)


@gpu
def test_workspaces_of_products(ld):
    """One's own or none given: the same result; left ready; refused where it cannot be used."""
    rng = np.random.default_rng(70)
    x, w = normal(rng, torch.bfloat16, 300, 8192), normal(rng, torch.bfloat16, 512, 8192, std=1 / 90)
    want, out, ws = *torch.empty(2, 300, 512, device="cuda").bfloat16(), ld.lora_linear_workspace()
    ld.lora_linear(want, x, w)
    for _ in range(3):
        ld.lora_linear(out, x, w, workspace=ws)
        assert torch.equal(out, want)
    assert not ws[:int(ld.lib().lora_linear_zeroed_bytes())].any()
    for bad in (ws.cpu(), ws[::2]):
        with pytest.raises(ValueError):
            ld.lora_linear(out, x, w, workspace=bad)
    with pytest.raises(ld.LoraError) as e:
        ld.lora_linear(out, x, w, workspace=ws[:-256])
    assert e.value.code == 5
    assert int(ld.lib().lora_linear_workspace_size(1, 1)) == 0 and int(ld.lib().lora_linear_workspace_size(2000, 64)) == 0
    # none at all, by the C call: whole tiles only
    import ctypes
    p = [ctypes.c_void_p(t.data_ptr()) for t in (out, x, w)]
    out.zero_()
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert ld.lib().lora_linear(p[0], 512, p[1], 8192, 300, 8192, p[2], 8192, 512, None, None, 0, None, 0, 0, 0, 0, None, 0, None, s) == 0
    reference, bound = ref.linear(host(x), host(w))
    close(host(out), reference, bound, torch.bfloat16)


@gpu
def test_graphs_of_products_have_workspaces_of_their_own(ld):
    """Two graphs and eager calls of shared tiles, side by side on three streams."""
    rng = np.random.default_rng(71)
    x, w = normal(rng, torch.bfloat16, 300, 8192), normal(rng, torch.bfloat16, 512, 8192, std=1 / 90)
    outs, graphs, streams = [torch.empty(300, 512, device="cuda").bfloat16() for _ in range(3)], [], [torch.cuda.Stream() for _ in range(3)]
    want = torch.empty_like(outs[0])
    ld.lora_linear(want, x, w)
    torch.cuda.synchronize()
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=streams[i]):
            ld.lora_linear(outs[i], x, w)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        ld.lora_linear(outs[2], x, w, stream=streams[2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@gpu
@pytest.mark.parametrize("T", [1, 50])
def test_example_of_a_layer(ld, T):
    from examples.moe_layer import MoeLayer
    layer, rng = MoeLayer(), np.random.default_rng(T)
    x, lora = normal(rng, torch.bfloat16, T, layer.H), dev(rng.integers(-1, layer.L, T))
    weights, ids = layer.route(x)
    out, plan = layer.forward(x, weights, ids, lora)
    c = {"ids": host(ids), "lora": host(lora), "x": x, "w": weights, "w13": layer.w13, "w2": layer.w2, "a13": layer.a13, "b13": layer.b13,
         "a2": layer.a2, "b2": layer.b2, "E": layer.E, "I": layer.I, "rank": layer.rank, "L": layer.L, "H": layer.H, "k": layer.top_k, "T": T}
    assert ld.lora_get_error(layer.err) == 0 and torch.equal(out, run_layer(ld, c)["out"])
    check_plan(plan, ref.plan(c["ids"], layer.E, c["lora"]))


@gpu
def test_gradients_of_a_loss_through_dispatch_and_combine(ld):
    """The calls' gradients of sum(combine(c * dispatch(x)) * g) against differences of the 64-bit form."""
    rng, T, k, E, H = np.random.default_rng(80), 20, 3, 5, 16
    ids = route(rng, T, k, E, none=0.1)
    x, c, g = normal(rng, torch.bfloat16, T, H), normal(rng, torch.bfloat16, T * k, H), normal(rng, torch.bfloat16, T, H)
    w = dev(rng.random((T, k)), np.float32)
    plan, rows, _ = dispatched(ld, ids, E, x)
    y = (rows.float() * c.float()).bfloat16()
    grad_y, grad_w = torch.zeros_like(y), torch.empty(T, k, device="cuda")
    ld.lora_moe_combine_grad(grad_y, grad_w, g, y, plan, weights=w)
    grad_rows, grad_x = (grad_y.float() * c.float()).bfloat16(), torch.empty_like(x)
    ld.lora_moe_combine(grad_x, grad_rows, plan)
    p, c64, g64, w64 = ref.plan(ids, E), host(c), host(g), host(w)

    def loss(x, w):
        moved = np.where(p["row_pair"][:, None] >= 0, x[p["row_pair"] // k], 0.0)
        return (ref.combine(moved * c64, p["pair_row"], w)[0] * g64).sum()

    x64, step = host(x), 1e-4
    for i in [(0, 0), (3, 7), (11, 15), (19, 2)]:
        d = np.zeros_like(x64)
        d[i] = step
        size = sum(abs(w64[i[0], j] * g64[i] * c64[r, i[1]]) for j, r in enumerate(p["pair_row"][i[0]]) if r >= 0)
        # three roundings to bf16 (grad_y, grad_rows, grad_x), half a step each, of terms and of their sum
        assert abs((loss(x64 + d, w64) - loss(x64 - d, w64)) / (2 * step) - host(grad_x)[i]) <= 3.1 * 2.0 ** -8 * size + 1e-6
    for i in [(0, 0), (5, 2), (17, 1)]:
        d = np.zeros_like(w64)
        d[i] = step
        r = p["pair_row"][i]
        size = np.abs(g64[i[0]] * x64[i[0]] * c64[r]).sum() if r >= 0 else 0.0
        # one rounding to bf16, of y
        assert abs((loss(x64, w64 + d) - loss(x64, w64 - d)) / (2 * step) - host(grad_w)[i]) <= 1.1 * 2.0 ** -8 * size + 1e-6


@gpu
@pytest.mark.parametrize("n,K,gated", [(1, 64, False), (16, 128, True), (128, 64, False)])
def test_products_are_awaited_after_a_wait_that_gave_up(ld, n, K, gated):
    """Sums so short that the wait for the last products is the likeliest to give up: it is reported, they are awaited all the
    same before their tensor memory is freed, and the calls that take it next are whole."""
    rng = np.random.default_rng(61)
    x, w = normal(rng, torch.bfloat16, n, K), normal(rng, torch.bfloat16, 2048, K)
    want, out = torch.empty(2, n, 1024 if gated else 2048, device="cuda").bfloat16()
    ld.lora_linear(want, x, w, gated=gated)
    reference, bound = ref.linear(host(x), host(w), gated=gated)
    close(host(want), reference, bound, torch.bfloat16)
    err = ld.new_error_word()
    for limit in (0, 0, 0, 1, 1000, 5000):
        old = ld.lora_set_wait_limit_ns(limit)
        try:
            ld.lora_linear(out, x, w, gated=gated, err=err)
        finally:
            ld.lora_set_wait_limit_ns(old)
        bits = ld.lora_get_error(err)
        assert bits == 8 or (bits == 0 and torch.equal(out, want))
        for _ in range(3):
            out.fill_(3)
            ld.lora_linear(out, x, w, gated=gated, err=err)
        assert ld.lora_get_error(err) == 0 and torch.equal(out, want)


@gpu
@pytest.mark.parametrize("n,K,N,gated", [(300, 8192, 512, False), (1090, 4096, 1296, True), (5000, 72, 2064, False), (3000, 1024, 4096, True)])
def test_counters_end_at_zero_after_waits_that_gave_up(ld, n, K, N, gated):
    """Limits so short that any wait of a product may give up, those for the next item of work among them: the call ends, reports
    it or is whole, leaves the counters of shared tiles at zero, and the next call with the same workspace is whole."""
    rng = np.random.default_rng(62)
    x, w, ws = normal(rng, torch.bfloat16, n, K), normal(rng, torch.bfloat16, N, K), ld.lora_linear_workspace()
    want, out = torch.empty(2, n, N // 2 if gated else N, device="cuda").bfloat16()
    ld.lora_linear(want, x, w, gated=gated, workspace=ws)
    counters, err = ws[:int(ld.lib().lora_linear_zeroed_bytes())], ld.new_error_word()
    for limit in (0, 0, 1, 2000, 5000, 20000, 50000):
        old = ld.lora_set_wait_limit_ns(limit)
        try:
            ld.lora_linear(out, x, w, gated=gated, workspace=ws, err=err)
        finally:
            ld.lora_set_wait_limit_ns(old)
        bits = ld.lora_get_error(err)
        assert bits == 8 or (bits == 0 and torch.equal(out, want))
        assert not counters.any()
        out.fill_(3)
        ld.lora_linear(out, x, w, gated=gated, workspace=ws, err=err)
        assert ld.lora_get_error(err) == 0 and torch.equal(out, want)


@gpu
def test_experts_after_waits_that_gave_up(ld):
    """The same over experts of uneven sizes."""
    rng, T, k, E, K, N = np.random.default_rng(63), 900, 4, 12, 1024, 784
    plan, x, _ = dispatched(ld, route(rng, T, k, E, none=0.1, skew=True), E, normal(rng, torch.bfloat16, T, K))
    w, ws, err = normal(rng, torch.bfloat16, E, N, K), ld.lora_linear_workspace(), ld.new_error_word()
    want, out = torch.zeros(2, T * k, N, device="cuda").bfloat16()
    ld.lora_moe_linear(want, x, w, plan, workspace=ws, err=err)
    for limit in (0, 0, 1, 2000, 5000, 20000):
        old = ld.lora_set_wait_limit_ns(limit)
        try:
            ld.lora_moe_linear(out, x, w, plan, workspace=ws, err=err)
        finally:
            ld.lora_set_wait_limit_ns(old)
        bits = ld.lora_get_error(err)
        assert bits == 8 or (bits == 0 and torch.equal(out, want))
        assert not ws[:int(ld.lib().lora_linear_zeroed_bytes())].any()
        out.zero_()
        ld.lora_moe_linear(out, x, w, plan, workspace=ws, err=err)
        assert ld.lora_get_error(err) == 0 and torch.equal(out, want)


@gpu
@pytest.mark.parametrize("n,K,N", [(300, 8192, 512), (1023, 6144, 2560), (256, 16384, 512), (8192, 4096, 4096)])
def test_waits_for_parts_of_shared_tiles_follow_the_limit(ld, n, K, N):
    """Tiles shared by two pairs of CTAs, by a few and by many, and behind whole rounds of tiles, with limits down to none: a
    call that does not report a wait is whole, one that does leaves the counters at zero."""
    rng = np.random.default_rng(64)
    x, w, ws = normal(rng, torch.float16, n, K), normal(rng, torch.float16, N, K, std=K ** -0.5), ld.lora_linear_workspace()
    want, out = torch.empty(2, n, N, device="cuda").half()
    err = ld.new_error_word()
    ld.lora_linear(want, x, w, workspace=ws, err=err)
    assert ld.lora_get_error(err) == 0
    if n < 2000:
        reference, bound = ref.linear(host(x), host(w))
        close(host(want), reference, bound, torch.float16)
    for limit in [0] + [300 * 2 ** (i / 2) for i in range(20)]:
        out.fill_(3)
        old = ld.lora_set_wait_limit_ns(int(limit))
        try:
            ld.lora_linear(out, x, w, workspace=ws, err=err)
        finally:
            ld.lora_set_wait_limit_ns(old)
        bits = ld.lora_get_error(err)
        assert bits == 8 or (bits == 0 and torch.equal(out, want))
        assert not ws[:int(ld.lib().lora_linear_zeroed_bytes())].any()
    ld.lora_linear(out, x, w, workspace=ws, err=err)
    assert ld.lora_get_error(err) == 0 and torch.equal(out, want)


def activation_alone(z, act):
    """An activation in 64 bits with nothing that cancels, and how far float32 may be from it relative to it.

    Of 2^-19: two powers 2^-22 each, a reciprocal 2^-23, a polynomial's fit and some ten roundings 2^-24 each.  The power's
    exponent is rounded 2^-24 relative, twice and in its constant, so that its value is off by the exponent times 2^-23 at most."""
    if act == "gelu":
        return 0.5 * z * np.vectorize(math.erfc)(-z / math.sqrt(2)), 2.0 ** -19 + z * z * 2.0 ** -23
    # z / (1 + e^-t), t for gelu_tanh of four roundings 2^-24 and constants' 2^-24 more, which the exponent takes whole
    t = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    e = np.exp(-np.abs(t))
    return np.where(t < 0, z * e, z) / (1 + e), 2.0 ** -19 + np.abs(t) * (2.0 ** -23 if act == "silu" else 2.0 ** -21)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["gelu", "silu", "gelu_tanh"])
@pytest.mark.parametrize("n", [1, 130])
@pytest.mark.parametrize("gated", [False, True])
def test_activations_of_every_number(ld, dtype, act, n, gated):
    """An activation of each 16-bit number, brought by the bias, to its own rounding: in the tails too, down to where the result
    leaves its type."""
    z = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32, device="cuda").to(torch.int16).view(dtype)
    bias = torch.cat([z, torch.ones_like(z)]) if gated else z
    x, w = torch.zeros(n, 8, device="cuda", dtype=dtype), torch.zeros(len(bias), 8, device="cuda", dtype=dtype)
    out, err = torch.empty(n, len(z), device="cuda", dtype=dtype), ld.new_error_word()
    ld.lora_linear(out, x, w, bias=bias, activation=act, gated=gated, err=err)
    assert ld.lora_get_error(err) == 0
    assert torch.equal(out.view(torch.int16), out[:1].view(torch.int16).expand_as(out))
    got, z = host(out[0]), host(z)
    assert np.isnan(got[np.isnan(z)]).all() and (got[z == np.inf] == np.inf).all()
    there = np.isfinite(z)
    want, off = activation_alone(z[there], act)
    # (what float32 itself may be off by below its normal range is less than a tenth of a step of bf16 there)
    tiny = 2.0 ** -25 if dtype is torch.float16 else 1.1 * 2.0 ** -134
    worst = np.abs(got[there] - want) - (STEP[dtype] * (1 + off) + off) * np.abs(want) - tiny
    assert (worst <= 0).all(), (z[there][worst.argmax()], got[there][worst.argmax()], want[worst.argmax()])


def layer_buffers(c):
    P, dtype = c["T"] * c["k"], c["x"].dtype
    names = {"rows": (P, c["H"]), "d13": (P, 1, 2 * c["I"]), "act": (P, c["I"]), "y": (P, c["H"]), "out": (c["T"], c["H"])}
    c["ptr"] = pointers(c["a13"]), pointers(c["b13"]), pointers([c["a2"]])[0].contiguous(), pointers([c["b2"]])[0].contiguous()
    c["d_ids"], c["d_lora"] = dev(c["ids"]), dev(c["lora"])
    return {n: torch.zeros(*shape, dtype=dtype, device="cuda") for n, shape in names.items()}


def run_layer_with_word(ld, c, b, plan, err):
    """The layer's calls into buffers ``b``, each with the error word."""
    P, R, H, I, kw = c["T"] * c["k"], c["rank"], c["H"], c["I"], {"err": err}
    a13, b13, a2, b2 = c["ptr"]
    ld.lora_moe_dispatch(b["rows"], c["x"], c["d_ids"], plan, lora_ids=c["d_lora"], **kw)
    ids = plan.row_expert.view(P, 1)
    ld.lora_moe_fc1_delta(b["d13"], b["rows"], a13, R * H, b13, I * R, False, ids, plan.row_lora, c["E"], I, R, c["L"], 2.0, **kw)
    ld.lora_moe_linear(b["act"], b["rows"], c["w13"], plan, delta=b["d13"].view(P, -1), activation="silu", gated=True, **kw)
    ld.lora_moe_linear(b["y"], b["act"], c["w2"], plan, **kw)
    ld.lora_moe_w2_delta(b["y"].view(P, 1, H), b["act"], a2, R * I, b2, H * R, ids, plan.row_lora, c["E"], H, R, c["L"], 2.0, **kw)
    ld.lora_moe_combine(b["out"], b["y"], plan, weights=c["w"], residual=c["x"])


@gpu
@pytest.mark.parametrize("T", [90, 400])
def test_a_layer_reports_into_one_error_word(ld, T):
    """No call of a layer reports anything, eager, on two streams at once or replayed; one that meets a bad expert does."""
    cases = [layer_case(ld, 90 + i, T=T) for i in range(2)]
    want = [run_layer(ld, c)["out"].clone() for c in cases]
    buffers, plans = [layer_buffers(c) for c in cases], [ld.MoePlan(T, c["k"], c["E"]) for c in cases]
    words, streams = [ld.new_error_word() for _ in cases], [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, b, plan, err, s in zip(cases, buffers, plans, words, streams):
            with torch.cuda.stream(s):
                run_layer_with_word(ld, c, b, plan, err)
    torch.cuda.synchronize()
    for b, y, err in zip(buffers, want, words):
        assert ld.lora_get_error(err) == 0 and torch.equal(b["out"], y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        run_layer_with_word(ld, cases[0], buffers[0], plans[0], words[0])
    for name in ("x", "w", "d_ids", "d_lora", "w13", "w2", "a2", "b2"):
        cases[0][name].copy_(cases[1][name])
    for name in ("a13", "b13"):
        for t, u in zip(cases[0][name], cases[1][name]):
            t.copy_(u)
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert ld.lora_get_error(words[0]) == 0 and torch.equal(buffers[0]["out"], want[1])
    cases[0]["d_ids"][T // 2, 0] = cases[0]["E"]
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert ld.lora_get_error(words[0]) == ref.ERR_EXPERT
    rest = [t for t in range(T) if t != T // 2]
    assert torch.equal(buffers[0]["out"][rest], want[1][rest])


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_a_tokens_combine_and_gradient_alone(ld, dtype):
    """Bit for bit what they are among other tokens."""
    rng, T, k, E, H = np.random.default_rng(91), 37, 5, 9, 1032
    plan, _, _ = dispatched(ld, route(rng, T, k, E, none=0.2), E, normal(rng, dtype, T, 8))
    rows, g, res, w = normal(rng, dtype, T * k, H), normal(rng, dtype, T, H), normal(rng, dtype, T, H), dev(rng.standard_normal((T, k)), np.float32)
    out, grad_rows, grad_w = torch.empty_like(g), torch.zeros_like(rows), torch.empty(T, k, device="cuda")
    ld.lora_moe_combine(out, rows, plan, weights=w, residual=res)
    ld.lora_moe_combine_grad(grad_rows, grad_w, g, rows, plan, weights=w)
    for t in range(T):
        # the token's rows first, in a plan of its own
        there = plan.pair_row[t] >= 0
        mine = torch.zeros(k, H, dtype=dtype, device="cuda")
        mine[there] = rows[plan.pair_row[t][there].long()]
        one = ld.MoePlan(1, k, E)
        one.pair_row.copy_(torch.where(there, torch.arange(k, device="cuda"), -1).view(1, k))
        y, gr, gw = torch.empty(1, H, dtype=dtype, device="cuda"), torch.zeros_like(mine), torch.empty(1, k, device="cuda")
        ld.lora_moe_combine(y, mine, one, weights=w[t:t + 1], residual=res[t:t + 1])
        ld.lora_moe_combine_grad(gr, gw, g[t:t + 1], mine, one, weights=w[t:t + 1])
        assert torch.equal(y, out[t:t + 1]) and torch.equal(gw, grad_w[t:t + 1])
        assert torch.equal(gr[there], grad_rows[plan.pair_row[t][there].long()])


@gpu
@pytest.mark.parametrize("T,k,E,K,N,gated", [(64, 8, 64, 512, 272, True), (400, 2, 3, 4096, 128, False), (2000, 4, 16, 64, 528, True)])
def test_products_of_experts_repeat(ld, T, k, E, K, N, gated):
    """Bit for bit the same again, with others between that leave their parts in the same workspace: few rows, tiles shared by
    many pairs, whole rounds of tiles."""
    rng = np.random.default_rng(92)
    plan, x, _ = dispatched(ld, route(rng, T, k, max(E, k), none=0.1, skew=True) % E, E, normal(rng, torch.bfloat16, T, K))
    w, other = normal(rng, torch.bfloat16, E, N, K, std=K ** -0.5), normal(rng, torch.bfloat16, 700, 2048)
    wo, oo = normal(rng, torch.bfloat16, 512, 2048), torch.empty(700, 512, device="cuda").bfloat16()
    want, out = torch.zeros(2, T * k, N // 2 if gated else N, device="cuda").bfloat16()
    err = ld.new_error_word()
    ld.lora_moe_linear(want, x, w, plan, gated=gated, err=err)
    for i in range(12):
        if i % 2:
            ld.lora_linear(oo, other, wo, err=err)
        out.fill_(0)
        ld.lora_moe_linear(out, x, w, plan, gated=gated, err=err)
        assert torch.equal(out, want)
    assert ld.lora_get_error(err) == 0


@gpu
def test_offsets_beyond_32_bits(ld):
    """Rows whose elements lie past 2^31: a dispatch, its way back with weights, its gradient, and products of them."""
    T, k, E, H = 34000, 8, 16, 8192
    rng = np.random.default_rng(95)
    ids = dev(rng.permuted(np.tile(np.arange(E), (T, 1)), axis=1)[:, :k])
    g = torch.Generator(device="cuda").manual_seed(95)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    w = torch.rand(T, k, device="cuda", generator=g)
    plan, rows, err = ld.MoePlan(T, k, E), torch.zeros(T * k, H, device="cuda").bfloat16(), ld.new_error_word()
    assert rows.numel() > 2 ** 31
    ld.lora_moe_dispatch(rows, x, ids, plan, err=err)
    token = torch.div(plan.row_pair, k, rounding_mode="floor").long()
    for a in range(0, T * k, 16384):
        assert torch.equal(rows[a:a + 16384], x[token[a:a + 16384]])
    out = torch.empty_like(x)
    ld.lora_moe_combine(out, rows, plan, weights=w)
    want = x[-500:].double() * w[-500:].double().sum(1, keepdim=True)
    # (k additions in float32 of terms of one sign)
    assert ((out[-500:].double() - want).abs() <= (2.0 ** -8 + (k + 2) * 2.0 ** -23) * want.abs() + 2.0 ** -134).all()
    grad, grad_w = torch.zeros_like(rows), torch.empty(T, k, device="cuda")
    ld.lora_moe_combine_grad(grad, grad_w, x, rows, plan, weights=w)
    for a in (0, T * k - 16384):
        t, p = token[a:a + 16384], plan.row_pair[a:a + 16384].long()
        assert torch.equal(grad[a:a + 16384], (x[t].float() * w.view(-1)[p][:, None]).bfloat16())
    # products: the many-rows kernel over all rows, in narrow columns of a wide result and to 8192 columns of it
    weight = torch.randn(E, 256, H, device="cuda", generator=g).bfloat16() * H ** -0.5
    y = torch.empty(T * k, 256, device="cuda").bfloat16()
    ld.lora_moe_linear(y, rows, weight, plan, err=err)
    ld.lora_linear(grad[:, -256:], rows, weight[3], delta=y, residual=y, err=err)
    wide = torch.randn(H, 64, device="cuda", generator=g).bfloat16() / 8
    ld.lora_linear(rows, y[:, :64], wide, err=err)
    assert ld.lora_get_error(err) == 0
    last, seg = slice(T * k - 300, T * k), host(plan.seg_start)
    assert seg[E - 1] < T * k - 300
    x64 = host(x[token[last]])
    want, bound = ref.linear(x64, host(weight[E - 1]))
    close(host(y[last]), want, bound, torch.bfloat16)
    want, bound = ref.linear(x64, host(weight[3]), delta=host(y[last]), residual=host(y[last]))
    close(host(grad[last, -256:]), want, bound, torch.bfloat16)
    want, bound = ref.linear(host(y[last, :64]), host(wide))
    close(host(rows[last]), want, bound, torch.bfloat16)
